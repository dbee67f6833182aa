"""Work of the operators around the expert layer, for timing and comparing them.

The four operators are the attention half of a decoder layer whose other half is the routed
expert layer: add_rmsnorm (the norm before attention and before the router), paged_plan (a
serving step's positions, page tables and cache slots from request lengths), rotary_append
(rotary positions on q and k, k and v into the paged cache) and PagedAttention (a chunk of
new tokens, or one token, of each request over its pages).

`run` computes a case either in plain form (elementary torch operations in 32 bits, rounded
once at the end) or, where `own` is true, through this package's kernels. `exact` is the
definition in 64 bits, written per request.
"""
import math
import random

import torch

own = False
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_handle = None  # the attention handle (workspace), kept as a serving program keeps it


def listed():
    return [
        # one token of one user: norm before attention, latency only (7,168 is the layer's hidden size)
        dict(name="norm_T1", op="norm", T=1, H=7168, dtype="bf16", residual=True, quant="none"),
        # a decode batch at the serving concurrency of 53, with an 8-bit copy for an 8-bit projection
        dict(name="norm_T53_row8", op="norm", T=53, H=7168, dtype="bf16", residual=True, quant="row"),
        # a prefill chunk of the largest bench size, 8-bit output in blocks of 128
        dict(name="norm_T8192_block8", op="norm", T=8192, H=7168, dtype="bf16", residual=True, quant="block"),
        # a decode step of 53 requests: every request gets one slot, some a new page
        dict(name="plan_B53", op="plan", B=53, new="one", new_max=1, ctx_max=8000, P=64, W=160),
        # a large step: prompts of up to a few hundred tokens joining a thousand running requests
        dict(name="plan_B1021_mixed", op="plan", B=1021, new="mixed", new_max=701, ctx_max=16000, P=16, W=1056),
        # decode: one token of 53 requests, 96 query heads over 8 key heads
        dict(name="rotary_T53", op="rotary", N=53, Hq=96, Hkv=8, D=128, rot=128, inter=False, scaled=True, P=64,
             dtype="bf16", pos_max=60000),
        # a chunk with rotary on half of each head, interleaved pairs, f16, ragged size
        dict(name="rotary_T1531_part", op="rotary", N=1531, Hq=24, Hkv=4, D=64, rot=32, inter=True, scaled=False,
             P=16, dtype="f16", pos_max=8000),
        # a full prefill chunk
        dict(name="rotary_T8192", op="rotary", N=8192, Hq=96, Hkv=8, D=128, rot=128, inter=False, scaled=True, P=64,
             dtype="bf16", pos_max=120000),
        # decode of a few short requests: latency
        dict(name="attn_decode_B5_short", op="attention", B=5, new="one", new_max=1, ctx_min=20, ctx_max=700, Hq=24,
             Hkv=4, D=64, P=16, dtype="f16", layout="token"),
        # decode of 128 requests of some thousand tokens each: streaming the cache
        dict(name="attn_decode_B128", op="attention", B=128, new="one", new_max=1, ctx_min=500, ctx_max=7500, Hq=96,
             Hkv=8, D=128, P=64, dtype="bf16", layout="token"),
        # a serving step that mixes prompt chunks of odd lengths with decoding requests
        dict(name="attn_mixed_B33", op="attention", B=33, new="mixed", new_max=517, ctx_min=0, ctx_max=5000, Hq=20,
             Hkv=4, D=128, P=32, dtype="bf16", layout="head"),
        # one chunk of a long prompt over the chunks before it: tensor-core bound
        dict(name="attn_chunk_4096", op="attention", B=1, new="equal", new_max=4096, ctx_min=12288, ctx_max=12288,
             Hq=96, Hkv=8, D=128, P=64, dtype="bf16", layout="token"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "plan", "rotary", "attention", "attention"])
    dt = rng.choice(["bf16", "bf16", "f16"])
    if op == "norm":
        H = rng.choice([_log_int(rng, 64, 14336), 8 * _log_int(rng, 16, 1792), 7168])
        return dict(op=op, T=_log_int(rng, 1, 8192), H=H, dtype=dt, residual=rng.random() < 0.75,
                    quant=rng.choice(["none", "row", "block"]))
    if op == "plan":
        P = rng.choice([16, 32, 64, 128])
        new = rng.choice(["one", "mixed", "equal"])
        B, ctx = _log_int(rng, 1, 1500), _log_int(rng, 10, 16000)
        n = 1 if new == "one" else _log_int(rng, 2, max(3, min(2000, 60000 // B)))
        return dict(op=op, B=B, new=new, new_max=n, ctx_max=ctx, P=P, W=(ctx + n) // P + 1 + rng.randrange(40))
    if op == "rotary":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, N=_log_int(rng, 1, 8192), Hq=Hkv * rng.choice([1, 3, 4, 6, 8, 12]), Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2, D - 24]), inter=rng.random() < 0.5, scaled=rng.random() < 0.5,
                    P=rng.choice([16, 32, 64, 128]), dtype=dt, pos_max=_log_int(rng, 100, 120000))
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 6, 8, 12])
    kind = rng.choice(["one", "one", "few", "mixed", "equal"])
    D, P = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    ctx = _log_int(rng, 30, 16000)
    if kind == "one":
        B, n = _log_int(rng, 1, max(2, min(256, 900000 // ctx))), 1
    elif kind == "few":  # a few draft tokens of each request checked at once
        B, n = _log_int(rng, 1, max(2, min(128, 400000 // ctx))), rng.randrange(2, 9)
    else:
        n = _log_int(rng, 9, 4000)
        B = _log_int(rng, 1, max(2, min(32, 60_000_000 // (n * (ctx + n)))))
        while B * G * Hkv * n * (ctx + n) > 96 * 4096 * 16384:
            n = n // 2 + 1
    return dict(op=op, B=B, new="equal" if kind == "few" else kind, new_max=n, ctx_min=rng.choice([0, ctx // 8, ctx]),
                ctx_max=ctx, Hq=G * Hkv, Hkv=Hkv, D=D, P=P, dtype=dt, layout=rng.choice(["token", "head"]))


def _lengths(case):
    """(context, new) tokens of each request: a function of the case's numbers alone, so `work` knows them too."""
    r = random.Random(f"{case['B']},{case['new']},{case['new_max']},{case['ctx_max']},{case['P']}")
    ctx = [r.randint(case.get("ctx_min", 0), case["ctx_max"]) for _ in range(case["B"])]
    kind, top = case["new"], case["new_max"]
    if kind == "one":
        new = [1] * case["B"]
    elif kind == "equal":
        new = [top] * case["B"]
    else:  # one request in eight brings a prompt chunk, the rest decode one token; the first always brings the longest
        new = [top if b == 0 else (r.randint(1, top) if r.random() < 0.125 else 1) for b in range(case["B"])]
    return ctx, new


def _inv_freq(case, dev):
    """Radians per position of each rotary pair, 64 bits. scaled: pairs that turn fewer than once in 4,096 positions are
    slowed 32 times for a 32 times longer context, those that turn over 32 times are kept, the ones between are blended."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / case["rot"])
    if case["scaled"]:
        keep = ((4096.0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / 32.0)
    return f.to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape, dtype, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * scale).to(dtype)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    s = dict(case=case)
    if case["op"] == "norm":
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        s["x"] = randn(T, H, dtype=dt)
        s["residual"] = randn(T, H, dtype=dt, scale=3.0) if case["residual"] else None
        s["weight"] = (1.0 + randn(H, dtype=torch.float32, scale=0.2)).to(dt)
        s["out"] = torch.empty(T, H, dtype=dt, device=dev)
        s["residual_out"] = torch.empty(T, H, dtype=dt, device=dev) if case["residual"] else None
        group = {"none": None, "row": 0, "block": 128}[case["quant"]]
        s["group"] = group or 0
        s["out8"] = None if group is None else torch.empty(T, H, dtype=torch.float8_e4m3fn, device=dev)
        s["scales"] = None if group is None else torch.empty(T, -(-H // (group or H)), dtype=torch.float32, device=dev)
        return s
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        B, P, W = case["B"], case["P"], case["W"]
        have = [-(-c // P) for c in ctx]
        need = sum(-(-(c + n) // P) - h for c, n, h in zip(ctx, new, have))
        pages = sum(have) + need + 100
        perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        s["ctx_lens"], s["new_lens"] = i32(ctx), i32(new)
        used = torch.arange(W, device=dev)[None, :] < i32(have)[:, None]
        rank = (torch.cumsum(used.flatten().to(torch.int64), 0) - 1).reshape(B, W)
        s["block_table"] = torch.where(used, perm[rank.clamp(min=0)], torch.full((), -1, dtype=torch.int32, device=dev))
        s["free_pages"] = perm[sum(have):].contiguous()
        s["free_head"] = i32([seed % 7])
        s["free_head_out"] = i32([0])
        N = sum(new)
        s["q_start"], s["kv_lens"] = i32([0] * (B + 1)), i32([0] * B)
        s["positions"], s["slots"] = i32([0] * N), i32([0] * N)
        return s
    if case["op"] == "rotary":
        N, Hq, Hkv, D, P, dt = (case[k] for k in ("N", "Hq", "Hkv", "D", "P", "dtype"))
        dt = DTYPES[dt]
        qkv = randn(N, (Hq + 2 * Hkv) * D, dtype=dt)  # one projection's output, q, k and v side by side
        s["q"] = qkv[:, :Hq * D].view(N, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(N, Hkv, D)
        s["v"] = qkv[:, (Hq + Hkv) * D:].view(N, Hkv, D)
        s["positions"] = torch.randint(0, case["pos_max"], (N,), generator=g, device=dev, dtype=torch.int32)
        pages = -(-N // P) + 3
        s["slots"] = torch.randperm(pages * P, generator=g, device=dev)[:N].to(torch.int32)
        s["inv_freq"] = _inv_freq(case, dev)
        s["mscale"] = 0.1 * math.log(32.0) + 1.0 if case["scaled"] else 1.0
        s["k_cache"] = torch.zeros(pages, P, Hkv, D, dtype=dt, device=dev)
        s["v_cache"] = torch.zeros(pages, P, Hkv, D, dtype=dt, device=dev)
        s["q_out"] = torch.empty(N, Hq, D, dtype=dt, device=dev)
        return s
    ctx, new = _lengths(case)
    B, P, Hq, Hkv, D, dt = (case[k] for k in ("B", "P", "Hq", "Hkv", "D", "dtype"))
    dt = DTYPES[dt]
    kv = [c + n for c, n in zip(ctx, new)]
    W = -(-max(kv) // P) + 1
    have = i32([-(-t // P) for t in kv])
    pages = int(sum(-(-t // P) for t in kv)) + 5
    used = torch.arange(W, device=dev)[None, :] < have[:, None]
    rank = (torch.cumsum(used.flatten().to(torch.int64), 0) - 1).reshape(B, W)
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    s["block_table"] = torch.where(used, perm[rank.clamp(min=0)], torch.full((), -1, dtype=torch.int32, device=dev))
    shape = (pages, P, Hkv, D) if case["layout"] == "token" else (pages, Hkv, P, D)
    s["k_cache"], s["v_cache"] = randn(*shape, dtype=dt), randn(*shape, dtype=dt)
    if case["layout"] == "head":
        s["k_cache"], s["v_cache"] = s["k_cache"].transpose(1, 2), s["v_cache"].transpose(1, 2)
    N = sum(new)
    s["q"] = randn(N, Hq, D, dtype=dt, scale=1.5)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["q_start"], s["kv_lens"] = i32(starts), i32(kv)
    s["max_new"] = max(new)
    s["scale"] = D ** -0.5
    s["out"] = torch.empty_like(s["q"])
    return s


def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


# ---- this package's kernels ------------------------------------------------------------------


def _own_norm(s):
    import routed_expert_layer_gb300 as rel
    rel.add_rmsnorm(s["x"], s["weight"], 1e-6, out=s["out"], residual=s["residual"], residual_out=s["residual_out"],
                    out8=s["out8"], scales=s["scales"], group=s["group"])
    return {k: s[k] for k in ("out", "residual_out", "out8", "scales")}


def _own_plan(s):
    import routed_expert_layer_gb300 as rel
    rel.paged_plan(s["ctx_lens"], s["new_lens"], s["block_table"], s["free_pages"], s["free_head"], s["case"]["P"],
                   q_start=s["q_start"], kv_lens=s["kv_lens"], positions=s["positions"], slots=s["slots"],
                   free_head_out=s["free_head_out"])
    return {k: s[k] for k in ("block_table", "q_start", "kv_lens", "positions", "slots", "free_head_out")}


def _own_rotary(s):
    import routed_expert_layer_gb300 as rel
    rel.rotary_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["k_cache"], s["v_cache"],
                      q_out=s["q_out"], interleaved=s["case"]["inter"], mscale=s["mscale"])
    return {k: s[k] for k in ("q_out", "k_cache", "v_cache")}


def _own_attention(s):
    global _handle
    if _handle is None:
        import routed_expert_layer_gb300 as rel
        _handle = rel.PagedAttention(device=0)
    _handle.forward(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["q_start"], s["kv_lens"], s["out"],
                    scale=s["scale"], max_new=s["max_new"])
    return {"out": s["out"]}


_run_own = {"norm": _own_norm, "plan": _own_plan, "rotary": _own_rotary, "attention": _own_attention}


# ---- plain forms -----------------------------------------------------------------------------


def _plain_norm(s):
    dt = s["x"].dtype
    t = s["x"].float()
    if s["residual"] is not None:
        t = t + s["residual"].float()
    y = t * torch.rsqrt((t * t).mean(dim=1, keepdim=True) + 1e-6) * s["weight"].float()
    out8 = scales = None
    if s["out8"] is not None:
        T, H = y.shape
        group = s["group"] or H
        blocks = torch.nn.functional.pad(y, (0, -H % group)).view(T, -1, group)
        scales = blocks.abs().amax(dim=2) / 448.0
        q = blocks / torch.where(scales > 0, scales, torch.ones_like(scales))[:, :, None]
        out8 = q.reshape(T, -1)[:, :H].to(torch.float8_e4m3fn)
    return {"out": y.to(dt), "residual_out": None if s["residual"] is None else t.to(dt), "out8": out8,
            "scales": scales}


def _plain_plan(s):
    P, table, ctx, new = s["case"]["P"], s["block_table"], s["ctx_lens"], s["new_lens"]
    B, W = table.shape
    N = s["positions"].numel()
    kv = ctx + new
    q_start = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0, dtype=torch.int32)])
    have, end = (ctx + P - 1) // P, (kv + P - 1) // P
    need = end - have
    first = torch.cumsum(need, 0, dtype=torch.int32) - need + s["free_head"]
    col = torch.arange(W, device=ctx.device, dtype=torch.int32)[None, :]
    fresh = (col >= have[:, None]) & (col < end[:, None])
    at = torch.where(fresh, first[:, None] + col - have[:, None], torch.zeros_like(col))
    table = torch.where(fresh, s["free_pages"][at], table)
    n = torch.arange(N, device=ctx.device, dtype=torch.int32)
    b = torch.searchsorted(q_start, n, right=True) - 1
    pos = ctx[b] + n - q_start[b]
    slots = table[b, pos // P] * P + pos % P
    return {"block_table": table, "q_start": q_start, "kv_lens": kv, "positions": pos, "slots": slots,
            "free_head_out": s["free_head"] + need.sum(dtype=torch.int32)}


def _rotate(t, cos, sin, rot, inter):
    r = t[..., :rot].float()
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :rot // 2], r[..., rot // 2:])
    x, y = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((x, y), dim=-1).flatten(-2) if inter else torch.cat((x, y), dim=-1)
    return torch.cat((turned, t[..., rot:].float()), dim=-1).to(t.dtype)


def _plain_rotary(s):
    angle = s["positions"].float()[:, None] * s["inv_freq"].float()[None, :]
    cos, sin = (torch.cos(angle) * s["mscale"])[:, None, :], (torch.sin(angle) * s["mscale"])[:, None, :]
    rot, inter = s["case"]["rot"], s["case"]["inter"]
    q_out = _rotate(s["q"], cos, sin, rot, inter)
    page, at = s["slots"] // s["case"]["P"], s["slots"] % s["case"]["P"]
    s["k_cache"][page, at] = _rotate(s["k"], cos, sin, rot, inter)
    s["v_cache"][page, at] = s["v"]
    return {"q_out": q_out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    q, P = s["q"], s["case"]["P"]
    N, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    B, M = s["kv_lens"].numel(), s["max_new"]
    L = s["block_table"].shape[1] * P
    dev = q.device
    kpos = torch.arange(L, device=dev)
    page = s["block_table"][:, kpos // P].clamp(min=0)
    k = s["k_cache"][page, kpos % P].float().permute(0, 2, 3, 1)  # [B, Hkv, D, L]
    v = s["v_cache"][page, kpos % P].float().permute(0, 2, 1, 3)  # [B, Hkv, L, D]
    start = s["q_start"].long()
    t = torch.arange(M, device=dev)
    rows = q[(start[:-1, None] + t).clamp(max=N - 1)].float()     # [B, M, Hq, D]
    rows = rows.view(B, M, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    scores = (rows * s["scale"]) @ k                              # [B, Hkv, G M, L]
    last = (s["kv_lens"] - (s["q_start"][1:] - s["q_start"][:-1])).long()[:, None] + t  # last key of each new token
    hidden = kpos[None, None, :] > last[:, :, None]
    scores.view(B, Hkv, Hq // Hkv, M, L).masked_fill_(hidden[:, None, None], float("-inf"))
    scores -= scores.amax(dim=-1, keepdim=True)
    p = scores.exp_()
    o = (p @ v) / p.sum(dim=-1, keepdim=True)
    o = o.view(B, Hkv, Hq // Hkv, M, D).permute(0, 3, 1, 2, 4)
    n = torch.arange(N, device=dev)
    b = torch.searchsorted(start, n, right=True) - 1
    return {"out": o[b, n - start[b]].reshape(N, Hq, D).to(q.dtype)}


_run_plain = {"norm": _plain_norm, "plan": _plain_plan, "rotary": _plain_rotary, "attention": _plain_attention}


# ---- what a pass cannot do without -------------------------------------------------------------


def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["H"]
        nbytes = n * (2 + 2 + (4 if case["residual"] else 0)) + 2 * case["H"]
        if case["quant"] != "none":
            nbytes += n + 4 * case["T"] * (1 if case["quant"] == "row" else -(-case["H"] // 128))
        return {"bytes": nbytes, "flops": 5 * n}
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        B, P = case["B"], case["P"]
        need = sum(-(-(c + n) // P) - -(-c // P) for c, n in zip(ctx, new))
        olds = sum(1 for c in ctx if c % P)  # requests whose first new token goes into a page they have
        return {"bytes": 4 * (2 * B + 2 * need + olds + 2 * sum(new) + 2 * B + 1 + 2), "flops": 0}
    if case["op"] == "rotary":
        heads = case["Hq"] + 2 * case["Hkv"]
        n = case["N"]
        return {"bytes": 2 * 2 * n * heads * case["D"] + 8 * n + 4 * case["rot"],
                "flops": 3 * n * (case["Hq"] + case["Hkv"]) * case["rot"]}
    ctx, new = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    kv = sum(c + n for c, n in zip(ctx, new))
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    pages = sum(-(-(c + n) // case["P"]) for c, n in zip(ctx, new))
    return {"bytes": 2 * 2 * kv * Hkv * D + 2 * 2 * sum(new) * Hq * D + 4 * pages + 8 * case["B"],
            "flops": 4 * pairs * Hq * D}


# ---- the definition in 64 bits -----------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "plan":
        return None
    if case["op"] == "norm":
        t = s["x"].to(f64) + (s["residual"].to(f64) if case["residual"] else 0.0)
        norm = torch.linalg.vector_norm(t, dim=1) / math.sqrt(case["H"])
        y = t / torch.sqrt(norm ** 2 + 1e-6)[:, None] * s["weight"].to(f64)
        out8 = scales = None
        if s["out8"] is not None:
            group = s["group"] or case["H"]
            parts = list(torch.split(y, group, dim=1))
            tops = [p.abs().max(dim=1).values / 448.0 for p in parts]
            scales = torch.stack(tops, dim=1)
            out8 = torch.cat([p / top.clamp(min=1e-300)[:, None] for p, top in zip(parts, tops)], dim=1)
        return {"out": y, "residual_out": t if case["residual"] else None, "out8": out8, "scales": scales}
    if case["op"] == "rotary":
        turns = torch.polar(torch.full((), s["mscale"], dtype=f64, device="cuda"),
                            s["positions"].to(f64)[:, None] * s["inv_freq"][None, :])[:, None, :]
        rot = case["rot"]

        def turn(x):
            x = x.to(f64).clone()
            pairs = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
            z = torch.complex(pairs[0].contiguous(), pairs[1].contiguous()) * turns
            pairs[0].copy_(z.real)
            pairs[1].copy_(z.imag)
            return x

        caches = []
        for src in (turn(s["k"]), s["v"].to(f64)):
            flat = torch.zeros(s["k_cache"].shape, dtype=f64, device="cuda").view(-1, case["Hkv"], case["D"])
            flat[s["slots"].long()] = src
            caches.append(flat.view(s["k_cache"].shape))
        return {"q_out": turn(s["q"]), "k_cache": caches[0], "v_cache": caches[1]}
    out = torch.empty(s["q"].shape, dtype=f64, device="cuda")
    ctx, new = _lengths(case)
    G, at = case["Hq"] // case["Hkv"], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        pages = s["block_table"][b, :-(-(c + n) // case["P"])].long()
        k = s["k_cache"][pages].reshape(-1, case["Hkv"], case["D"])[:c + n]
        v = s["v_cache"][pages].reshape(-1, case["Hkv"], case["D"])[:c + n]
        seen = torch.ones(n, c + n, dtype=torch.bool, device="cuda").tril(c)
        for h in range(case["Hkv"]):
            kh, vh = k[:, h].to(f64), v[:, h].to(f64)
            qh = s["q"][at:at + n, h * G:(h + 1) * G].to(f64)
            w = torch.einsum("ngd,ld->ngl", qh, kh) * s["scale"]
            w = torch.softmax(w.masked_fill(~seen[:, None], -math.inf), dim=2)
            out[at:at + n, h * G:(h + 1) * G] = torch.einsum("ngl,ld->ngd", w, vh)
        at += n
    return {"out": out}
