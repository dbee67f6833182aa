"""Work of the operators of a decoder layer that checks drafted tokens with 8-bit projections, for timing and
comparing them.

quantize8 (16-bit values to e4m3 with a scale per row, per 128 values or per 128 x 128), Matmul8 (product of e4m3
activations and weights with those scales), tree_plan (positions and ancestor masks of each request's drafted tree),
PagedAttention with such a mask, and tree_accept (the path that the model's own tokens take through the tree, its keys
and values moved to where the next step expects them).

`run` computes a case either in plain form (elementary torch operations in 32 bits, rounded once at the end) or, where
`own` is true, through this package's kernels. `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
_handles = {}  # the handles (workspaces) of products and attention, kept as a serving program keeps them


def listed():
    return [
        # one token: the projection of 96 heads of 128 back to the layer's hidden size, latency and weights' bytes
        dict(name="matmul_T1", op="matmul", T=1, N=7168, K=12288, row_scale=False, dtype="bf16"),
        # q, k and v of a decode batch at the serving concurrency of 53: streaming the weights
        dict(name="matmul_T53", op="matmul", T=53, N=14336, K=7168, row_scale=False, dtype="bf16"),
        # a ragged chunk through a narrow projection whose sizes divide nothing, a scale per token
        dict(name="matmul_T517_odd", op="matmul", T=517, N=1811, K=7152, row_scale=True, dtype="f16"),
        # a full prefill chunk: tensor-core bound
        dict(name="matmul_T8192", op="matmul", T=8192, N=14336, K=7168, row_scale=False, dtype="bf16"),
        # attention's output of a decode batch, before its projection
        dict(name="quantize_T53", op="quantize", T=53, H=12288, group=128, rows=1, dtype="bf16"),
        # the same of a prefill chunk
        dict(name="quantize_T8192", op="quantize", T=8192, H=12288, group=128, rows=1, dtype="bf16"),
        # 16 requests with a window of 4 drafted positions each
        dict(name="plan_B16_window", op="plan", B=16, tree="chain", new="equal", new_max=4, W=1),
        # a thousand requests with trees of up to 64 nodes, some with a prompt chunk instead
        dict(name="plan_B1021_trees", op="plan", B=1021, tree="wide", new="mixed", new_max=64, W=2),
        # the window of 4 over some thousand cached tokens: streaming the cache
        dict(name="attn_B16_window", op="attention", B=16, tree="chain", new="equal", new_max=4, W=1, ctx_min=500,
             ctx_max=7500, Hq=96, Hkv=8, D=128, P=64, dtype="bf16", layout="token"),
        # trees of 1 to 60 nodes for the serving concurrency of 53
        dict(name="attn_B53_trees", op="attention", B=53, tree="wide", new="mixed", new_max=60, W=2, ctx_min=0,
             ctx_max=4000, Hq=96, Hkv=8, D=128, P=64, dtype="bf16", layout="token"),
        # one user's tree of 25 nodes, one layer's cache: latency
        dict(name="accept_B1", op="accept", B=1, tree="wide", new="equal", new_max=25, ctx_max=500, layers=1, Hkv=8, D=128,
             P=64, depth=6, certain=False, dtype="bf16"),
        # 53 users' trees of up to 60 nodes, the caches of 24 layers in one call
        dict(name="accept_B53_layers", op="accept", B=53, tree="wide", new="mixed", new_max=60, ctx_max=100, layers=24,
             Hkv=8, D=128, P=16, depth=8, certain=True, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "quantize", "plan", "attention", "attention", "accept"])
    dt = rng.choice(["bf16", "bf16", "f16"])
    if op == "matmul":
        T = _log_int(rng, 1, 8192)
        N = rng.choice([_log_int(rng, 16, 14336), 128 * _log_int(rng, 1, 112), 14336, 7168])
        K = rng.choice([16 * _log_int(rng, 1, 768), 128 * _log_int(rng, 1, 96), 7168, 12288])
        while T * N * K > 8192 * 14336 * 7168:
            T = T // 2
        return dict(op=op, T=T, N=N, K=K, row_scale=rng.random() < 0.25, dtype=dt)
    if op == "quantize":
        rows = rng.choice([1, 1, 128])
        return dict(op=op, T=_log_int(rng, 1, 8192), H=rng.choice([_log_int(rng, 1, 12288), 128 * _log_int(rng, 1, 96)]),
                    group=128 if rows == 128 else rng.choice([0, 128]), rows=rows, dtype=dt)
    tree, new = rng.choice(["wide", "wide", "chain", "deep"]), rng.choice(["equal", "mixed"])
    if op == "plan":
        B, W = _log_int(rng, 1, 1500), rng.randint(1, 8)
        return dict(op=op, B=B, tree=tree, new=new, new_max=_log_int(rng, 1, 32 * W), W=W)
    if op == "accept":
        layers, Hkv, D = _log_int(rng, 1, 60), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        B = _log_int(rng, 1, max(1, min(256, 16_000_000 // (layers * Hkv * D * 160))))
        return dict(op=op, B=B, tree=tree, new=new, new_max=_log_int(rng, 1, 120), ctx_max=_log_int(rng, 1, 100),
                    layers=layers, Hkv=Hkv, D=D, P=rng.choice([16, 32, 64]), depth=rng.randint(1, 12),
                    certain=rng.random() < 0.5, dtype=dt)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 6, 8, 12])
    D, P, ctx = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128]), _log_int(rng, 1, 12000)
    n = _log_int(rng, 1, 256)
    B = _log_int(rng, 1, max(1, min(128, 400000 // (ctx + n), 12_000_000 // (n * (ctx + n)))))
    W = rng.randint(-(-n // 32), 8)
    return dict(op=op, B=B, tree=tree, new=new, new_max=n, W=W, ctx_min=rng.choice([0, ctx // 8, ctx]), ctx_max=ctx,
                Hq=G * Hkv, Hkv=Hkv, D=D, P=P, dtype=dt, layout=rng.choice(["token", "head"]))


def _requests(case):
    """(context, parents) of each request: a function of the case's numbers alone, so `work` knows them too.
    Parents stand before their children; node 0 is the root. chain: drafts in a row; deep: two drafts a level on
    average; wide: four. mixed: every size up to the largest, one request in twelve without drafts, and with a mask of W words
    one in sixteen has a prompt chunk, longer than the mask, in the place of a tree."""
    r = random.Random(f"{case['B']},{case['tree']},{case['new']},{case['new_max']},{case.get('ctx_max', 0)}")
    ctx, parents = [], []
    for b in range(case["B"]):
        ctx.append(r.randint(case.get("ctx_min", 0), case.get("ctx_max", 9000)))
        n, chain = case["new_max"], case["tree"] == "chain"
        if case["new"] == "mixed" and b:
            kind = r.random()
            n = 1 if kind < 1 / 12 else r.randint(1, n)
            if "W" in case and kind > 15 / 16:
                n, chain = 32 * case["W"] + r.randint(1, 40), True
        p, up = [-1], 0
        step = {"wide": 0.25, "deep": 0.5}.get(case["tree"])
        for j in range(1, n):
            while not chain and up < j - 1 and r.random() < step:
                up += 1
            p.append(j - 1 if chain else up)
        parents.append(p)
    return ctx, parents


def _path(r, parents, certain, depth):
    """The drafted nodes that the case's targets accept after the `certain` first ones: a random walk down the tree,
    such that no accepted node lies where another is moved to (so a repeated call finds the same keys and values)."""
    kids = {}
    for j, p in enumerate(parents):
        kids.setdefault(p, []).append(j)
    best = []
    for _ in range(8):
        path, cur = [], certain - 1
        while len(path) < depth and kids.get(cur) and r.random() < 0.85:
            cur = r.choice(kids[cur])
            path.append(cur)
        end = certain + len(path)
        if all(j == certain + i or j >= end for i, j in enumerate(path)) and len(path) > len(best):
            best = path
    return best


def _drafts(case):
    """Of each request: tokens, the model's tokens after each node, and how many first nodes are certain."""
    r = random.Random(f"drafts {case['B']},{case['tree']},{case['new_max']},{case['depth']}")
    ctx, parents = _requests(case)
    out = []
    for p in parents:
        certain = 1
        if case["certain"] and r.random() < 0.2:  # a prompt: a chain whose tokens are all known
            p[:] = list(range(-1, len(p) - 1))
            certain = len(p)
        path = _path(r, p, certain, case["depth"])
        tokens = r.sample(range(150000), len(p))
        targets = [r.randrange(150000, 160000) for _ in p]  # tokens that no draft has
        for a, b in zip([certain - 1] + path, path):
            targets[a] = tokens[b]
        out.append((tokens, targets, certain, path))
    return ctx, parents, out


def _quantized(x, group, rows):
    """x as e4m3 values and fp32 scales: blocks of `group` columns (0: the row) and `rows` rows."""
    T, H = x.shape
    group = group or H
    f = torch.nn.functional.pad(x.float(), (0, -H % group, 0, -T % rows))
    blocks = f.view(-1, rows, f.shape[1] // group, group)
    scales = blocks.abs().amax(dim=(1, 3)) / 448.0
    q = blocks / torch.where(scales > 0, scales, torch.ones_like(scales))[:, None, :, None]
    return q.reshape(f.shape)[:T, :H].to(E4M3), scales


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape, dtype, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * scale).to(dtype)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    s = dict(case=case)
    dt = DTYPES[case["dtype"]] if "dtype" in case else None
    if case["op"] == "matmul":
        T, N, K = case["T"], case["N"], case["K"]
        # activations of a norm: some channels of every token are several times larger than the others
        x = randn(T, K, dtype=torch.float32) * (1.0 + 3.0 * (torch.rand(K, generator=g, device=dev) < 0.02))
        s["a8"], s["a_scales"] = _quantized(x, 0 if case["row_scale"] else 128, 1)
        s["w8"], s["w_scales"] = _quantized(randn(N, K, dtype=torch.float32, scale=K ** -0.5), 128, 128)
        s["out"] = torch.empty(T, N, dtype=dt, device=dev)
        return s
    if case["op"] == "quantize":
        T, H = case["T"], case["H"]
        s["x"] = randn(T, H, dtype=dt, scale=0.3)
        s["out8"] = torch.empty(T, H, dtype=E4M3, device=dev)
        s["scales"] = torch.empty(-(-T // case["rows"]), -(-H // (case["group"] or H)), dtype=torch.float32, device=dev)
        return s
    if case["op"] == "accept":
        ctx, parents, drafts = _drafts(case)
    else:
        ctx, parents = _requests(case)
    if case["op"] == "plan":
        ctx = [c + seed % 5 for c in ctx]
    new = [len(p) for p in parents]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["q_start"], s["ctx_lens"] = i32(starts), i32(ctx)
    s["parents"] = i32([p for q in parents for p in q])
    N, B = starts[-1], case["B"]
    if case["op"] == "plan":
        s["positions"], s["mask"] = i32([0] * N), torch.zeros(N, case["W"], dtype=torch.int32, device=dev)
        return s
    P, Hkv, D = case["P"], case["Hkv"], case["D"]
    kv = [c + n for c, n in zip(ctx, new)]
    W = -(-max(kv) // P) + 1
    have = i32([-(-t // P) for t in kv])
    pages = int(sum(-(-t // P) for t in kv)) + 5
    used = torch.arange(W, device=dev)[None, :] < have[:, None]
    rank = (torch.cumsum(used.flatten().to(torch.int64), 0) - 1).reshape(B, W)
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    s["block_table"] = torch.where(used, perm[rank.clamp(min=0)], torch.full((), -1, dtype=torch.int32, device=dev))
    if case["op"] == "accept":
        shape = (case["layers"], pages, P, Hkv, D)
        s["k_cache"], s["v_cache"] = randn(*shape, dtype=dt), randn(*shape, dtype=dt)
        s["tokens"], s["targets"] = (i32([t + seed % 1009 for d in drafts for t in d[i]]) for i in (0, 1))
        s["certain"] = i32([d[2] for d in drafts]) if case["certain"] else None
        s["path"] = torch.zeros(B, case["depth"], dtype=torch.int32, device=dev)
        s["accepted"], s["ctx_out"], s["next_tokens"] = i32([0] * B), i32([0] * B), i32([0] * B)
        return s
    shape = (pages, P, Hkv, D) if case["layout"] == "token" else (pages, Hkv, P, D)
    s["k_cache"], s["v_cache"] = randn(*shape, dtype=dt), randn(*shape, dtype=dt)
    if case["layout"] == "head":
        s["k_cache"], s["v_cache"] = s["k_cache"].transpose(1, 2), s["v_cache"].transpose(1, 2)
    s["q"] = randn(N, case["Hq"], D, dtype=dt, scale=1.5)
    s["kv_lens"], s["max_new"], s["scale"] = i32(kv), max(new), D ** -0.5
    # what tree_plan writes once for all layers of a step
    words = []
    for p in parents:
        bits = []
        for j, up in enumerate(p):
            bits.append((1 << j) | (bits[up] if up >= 0 else 0))
        for m in bits:
            m = m if len(p) <= 32 * case["W"] else 0
            words.append([((m >> (32 * w)) & 0xFFFFFFFF ^ 0x80000000) - 0x80000000 for w in range(case["W"])])
    s["mask"] = i32(words)
    s["out"] = torch.empty_like(s["q"])
    return s


def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


# ---- this package's kernels ------------------------------------------------------------------


def _handle(name):
    if name not in _handles:
        import routed_expert_layer_gb300 as rel
        _handles[name] = getattr(rel, name)(device=0)
    return _handles[name]


def _own_matmul(s):
    _handle("Matmul8").forward(s["a8"], s["a_scales"], s["w8"], s["w_scales"], s["out"])
    return {"out": s["out"]}


def _own_quantize(s):
    import routed_expert_layer_gb300 as rel
    rel.quantize8(s["x"], s["out8"], s["scales"], group=s["case"]["group"], rows=s["case"]["rows"])
    return {"out8": s["out8"], "scales": s["scales"]}


def _own_plan(s):
    import routed_expert_layer_gb300 as rel
    rel.tree_plan(s["parents"], s["q_start"], s["ctx_lens"], positions=s["positions"], mask=s["mask"])
    return {"positions": s["positions"], "mask": s["mask"]}


def _own_attention(s):
    _handle("PagedAttention").forward(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["q_start"], s["kv_lens"],
                                      s["out"], scale=s["scale"], max_new=s["max_new"], tree=s["mask"])
    return {"out": s["out"]}


def _own_accept(s):
    import routed_expert_layer_gb300 as rel
    rel.tree_accept(s["parents"], s["tokens"], s["targets"], s["q_start"], s["ctx_lens"], s["block_table"], s["k_cache"],
                    s["v_cache"], path=s["path"], accepted=s["accepted"], ctx_out=s["ctx_out"],
                    next_tokens=s["next_tokens"], certain=s["certain"])
    return {k: s[k] for k in ("path", "accepted", "ctx_out", "next_tokens", "k_cache", "v_cache")}


_run_own = {"matmul": _own_matmul, "quantize": _own_quantize, "plan": _own_plan, "attention": _own_attention,
            "accept": _own_accept}


# ---- plain forms -----------------------------------------------------------------------------


def _spread(scales, rows, K):
    """A scale per element of a row of K: [rows][K] from [rows or ceil(rows / 128)][blocks or 1]."""
    if scales.shape[0] != rows:
        scales = scales.repeat_interleave(128, dim=0)[:rows]
    if scales.shape[1] == 1:
        return scales
    return scales.repeat_interleave(128, dim=1)[:, :K]


def _plain_matmul(s):
    (T, K), N = s["a8"].shape, s["w8"].shape[0]
    a = s["a8"].float() * _spread(s["a_scales"], T, K)
    w = s["w8"].float() * _spread(s["w_scales"], N, K)
    return {"out": (a @ w.t()).to(s["out"].dtype)}


def _plain_quantize(s):
    out8, scales = _quantized(s["x"], s["case"]["group"], s["case"]["rows"])
    return {"out8": out8, "scales": scales}


def _rows(s, N):
    """Of every row: its request, its place in the request, and the request's number of new tokens."""
    n = torch.arange(N, device=s["q_start"].device)
    b = torch.searchsorted(s["q_start"].long(), n, right=True) - 1
    start = s["q_start"].long()
    return b, n - start[b], (start[1:] - start[:-1])[b]


def _plain_plan(s):
    N, W = s["mask"].shape
    b, t, new = _rows(s, N)
    chunk = new > 32 * W  # a prompt chunk: a chain, its mask is not written
    up = s["parents"].long()
    first = torch.arange(N, device=up.device) - t
    word = torch.arange(W, device=up.device)[None, :]
    mask = torch.zeros(N, W, dtype=torch.int64, device=up.device)
    depth = torch.zeros(N, dtype=torch.int64, device=up.device)
    node = t
    for _ in range(s["case"]["new_max"]):  # one level up per turn
        live = node >= 0
        mask += torch.where(live[:, None] & (word == node[:, None] // 32), 1 << (node[:, None] % 32), 0)
        node = torch.where(live, up[first + node.clamp(min=0)], node)
        depth += (node >= 0).long()
    mask = torch.where(chunk[:, None], s["mask"].long(), mask)
    positions = s["ctx_lens"].long()[b] + torch.where(chunk, t, depth)
    return {"positions": positions.int(), "mask": mask.int()}


def _plain_attention(s):
    q, P = s["q"], s["case"]["P"]
    N, Hq, D = q.shape
    Hkv, W = s["k_cache"].shape[2], s["mask"].shape[1]
    B, M = s["kv_lens"].numel(), s["max_new"]
    L = s["block_table"].shape[1] * P
    dev = q.device
    kpos = torch.arange(L, device=dev)
    start = s["q_start"].long()
    new = start[1:] - start[:-1]
    ctx = s["kv_lens"].long() - new
    t = torch.arange(M, device=dev)
    out = torch.zeros(N, Hq, D, dtype=torch.float32, device=dev)
    piece = max(1, 2_000_000_000 // (M * Hq * L))  # requests whose scores are in memory at a time
    for b0 in range(0, B, piece):
        some = slice(b0, min(B, b0 + piece))
        page = s["block_table"][some][:, kpos // P].clamp(min=0)
        k = s["k_cache"][page, kpos % P].float().permute(0, 2, 3, 1)  # [b, Hkv, D, L]
        v = s["v_cache"][page, kpos % P].float().permute(0, 2, 1, 3)  # [b, Hkv, L, D]
        at = (start[:-1][some, None] + t).clamp(max=N - 1)
        rows = q[at].float().view(-1, M, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(-1, Hkv, Hq // Hkv * M, D)
        scores = (rows * s["scale"]) @ k                              # [b, Hkv, G M, L]
        rel = kpos[None, :] - ctx[some, None]                         # the new token at each key
        inside = rel.clamp(0, 32 * W - 1)
        bits = s["mask"][at].gather(2, (inside // 32)[:, None, :].expand(-1, M, -1)) >> (inside % 32)[:, None, :]
        tree = (rel < 0)[:, None, :] | (((bits & 1) == 1) & (rel < new[some, None])[:, None, :])
        causal = rel[:, None, :] <= t[None, :, None]
        seen = torch.where((new[some] > 32 * W)[:, None, None], causal, tree)
        scores.view(-1, Hkv, Hq // Hkv, M, L).masked_fill_(~seen[:, None, None], float("-inf"))
        scores -= scores.amax(dim=-1, keepdim=True)
        p = scores.exp_()
        o = ((p @ v) / p.sum(dim=-1, keepdim=True)).view(-1, Hkv, Hq // Hkv, M, D).permute(0, 3, 1, 2, 4).reshape(-1, M, Hq, D)
        live = t[None, :] < new[some, None]
        out[at[live]] = o[live]
    return {"out": out.to(q.dtype)}


def _plain_accept(s):
    B, depth = s["path"].shape
    N, P = s["parents"].numel(), s["case"]["P"]
    dev = s["parents"].device
    b, t, _ = _rows(s, N)
    start = s["q_start"].long()
    first = torch.ones(B, dtype=torch.int64, device=dev) if s["certain"] is None else s["certain"].long()
    cur, count = first - 1, torch.zeros(B, dtype=torch.int64, device=dev)
    path = torch.full((B, depth), -1, dtype=torch.int64, device=dev)
    none = torch.full((B,), N, dtype=torch.int64, device=dev)
    for i in range(depth):
        target = s["targets"][start[:-1] + cur]
        hit = (s["parents"] == cur[b]) & (s["tokens"] == target[b]) & (t >= first[b]) & (count[b] == i)
        child = none.scatter_reduce(0, b, torch.where(hit, t, N), "amin")
        found = child < N
        cur = torch.where(found, child, cur)
        count += found.long()
        path[:, i] = torch.where(found, child, path[:, i])
    step = torch.arange(depth, device=dev)[None, :]
    ctx = s["ctx_lens"].long()[:, None]
    # places past the path move the last certain token's row to itself
    still = (first - 1)[:, None].expand(-1, depth)
    src = ctx + torch.where(path >= 0, path, still)
    dst = ctx + torch.where(path >= 0, first[:, None] + step, still)
    table = s["block_table"].long()
    for cache in (s["k_cache"], s["v_cache"]):
        rows = cache[:, table.gather(1, src // P), src % P]
        cache[:, table.gather(1, dst // P), dst % P] = rows
    accepted = (first + count).int()
    return {"path": path.int(), "accepted": accepted, "ctx_out": s["ctx_lens"] + accepted,
            "next_tokens": s["targets"][start[:-1] + cur], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


_run_plain = {"matmul": _plain_matmul, "quantize": _plain_quantize, "plan": _plain_plan, "attention": _plain_attention,
              "accept": _plain_accept}


# ---- what a pass cannot do without -------------------------------------------------------------


def work(case):
    if case["op"] == "matmul":
        T, N, K = case["T"], case["N"], case["K"]
        blocks = -(-K // 128)
        return {"bytes": T * K + N * K + 2 * T * N + 4 * (T * (1 if case["row_scale"] else blocks) + -(-N // 128) * blocks),
                "flops": 2 * T * N * K}
    if case["op"] == "quantize":
        T, H = case["T"], case["H"]
        return {"bytes": 3 * T * H + 4 * -(-T // case["rows"]) * -(-H // (case["group"] or H)), "flops": 3 * T * H}
    if case["op"] == "accept":
        ctx, parents, drafts = _drafts(case)
        new = sum(len(p) for p in parents)
        moved = sum(1 for d in drafts for i, j in enumerate(d[3]) if j != d[2] + i)
        return {"bytes": 4 * 3 * new + 4 * case["B"] * (5 + case["depth"]) +
                2 * 2 * 2 * moved * case["layers"] * case["Hkv"] * case["D"], "flops": 0}
    ctx, parents = _requests(case)
    new = [len(p) for p in parents]
    masked = sum(n for n in new if n <= 32 * case["W"])
    if case["op"] == "plan":
        return {"bytes": 4 * (2 * sum(new) + masked * case["W"] + 2 * case["B"] + 1), "flops": 0}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    kv, pairs = sum(ctx) + sum(new), 0
    for c, p in zip(ctx, parents):
        depth = []
        for up in p:
            depth.append(1 + (depth[up] if up >= 0 else 0))
        pairs += c * len(p) + sum(depth)
    pages = sum(-(-(c + n) // case["P"]) for c, n in zip(ctx, new))
    return {"bytes": 2 * 2 * kv * Hkv * D + 2 * 2 * sum(new) * Hq * D + 4 * masked * case["W"] + 4 * pages + 8 * case["B"],
            "flops": 4 * pairs * Hq * D}


# ---- the definition in 64 bits -----------------------------------------------------------------


def exact(case, seed):
    if case["op"] in ("plan", "accept"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "matmul":
        K, N = case["K"], case["N"]
        out = torch.zeros(case["T"], N, dtype=f64, device="cuda")
        w_scale = torch.repeat_interleave(s["w_scales"].to(f64), 128, dim=0)[:N]
        for i, k in enumerate(range(0, K, 128)):
            block = torch.einsum("tk,nk->tn", s["a8"][:, k:k + 128].to(f64), s["w8"][:, k:k + 128].to(f64))
            out += block * s["a_scales"].to(f64)[:, i if s["a_scales"].shape[1] > 1 else 0, None] * w_scale[:, i]
        return {"out": out}
    if case["op"] == "quantize":
        T, H = case["T"], case["H"]
        group, x = case["group"] or H, s["x"].to(f64)
        scales = torch.zeros(s["scales"].shape, dtype=f64, device="cuda")
        out8 = torch.zeros_like(x)
        if case["rows"] == 1:
            for i, k in enumerate(range(0, H, group)):
                part = x[:, k:k + group]
                scales[:, i] = part.abs().max(dim=1).values / 448.0
                out8[:, k:k + group] = part / scales[:, i, None].clamp(min=1e-300)
            return {"out8": out8, "scales": scales}
        for r in range(scales.shape[0]):
            rows = slice(128 * r, 128 * (r + 1))
            tops = [p.abs().max() / 448.0 for p in torch.split(x[rows], 128, dim=1)]
            scales[r] = torch.stack(tops)
            out8[rows] = x[rows] / torch.repeat_interleave(scales[r].clamp(min=1e-300), 128)[:H]
        return {"out8": out8, "scales": scales}
    ctx, parents = _requests(case)
    if sum(len(p) * (c + len(p)) for c, p in zip(ctx, parents)) * case["Hq"] * case["D"] > 4e12:
        return None
    out = torch.empty(s["q"].shape, dtype=f64, device="cuda")
    G, at = case["Hq"] // case["Hkv"], 0
    for b, (c, p) in enumerate(zip(ctx, parents)):
        n = len(p)
        seen = torch.zeros(n, c + n, dtype=torch.bool)
        seen[:, :c] = True
        for j, up in enumerate(p):
            if up >= 0:
                seen[j, c:] = seen[up, c:]
            seen[j, c + j] = True
        seen = seen.cuda()
        pages = s["block_table"][b, :-(-(c + n) // case["P"])].long()
        k = s["k_cache"][pages].reshape(-1, case["Hkv"], case["D"])[:c + n].to(f64)
        v = s["v_cache"][pages].reshape(-1, case["Hkv"], case["D"])[:c + n].to(f64)
        q = s["q"][at:at + n].to(f64).view(n, case["Hkv"], G, case["D"])
        w = torch.einsum("nhgd,lhd->hgnl", q, k) * s["scale"]
        w = torch.softmax(w.masked_fill(~seen, -math.inf), dim=3)
        out[at:at + n] = torch.einsum("hgnl,lhd->nhgd", w, v).reshape(n, case["Hq"], case["D"])
        at += n
    return {"out": out}
