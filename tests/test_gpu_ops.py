"""The operators beside the expert layer on the GPU, against plain 64-bit forms
(ops_reference.py, where every tolerance is derived)."""
import math
import random

import pytest
import torch

import ops_reference as ref
import routed_expert_layer_gb300 as rel

pytestmark = pytest.mark.gpu
BF16, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def inside(got, want, bound):
    """got within bound of want; NaN where want is NaN, the same infinities."""
    got = got.to(torch.float64)
    odd = ~torch.isfinite(want)
    same = torch.where(odd, (got == want) | (got.isnan() & want.isnan()), (got - want).abs() <= bound)
    if not bool(same.all()):
        off = torch.where(odd, torch.full_like(want, math.inf), (got - want).abs() - bound)
        at = int(torch.where(same, torch.full_like(off, -math.inf), off.nan_to_num(math.inf)).argmax())
        raise AssertionError(f"{int((~same).sum())} of {same.numel()} outside the bound, worst at {at}: "
                             f"{got.flatten()[at].item()} for {want.flatten()[at].item()}")


# ---- norm --------------------------------------------------------------------------------------


def check_norm(x, w, eps, residual, group, out, residual_out, out8, scales):
    t, y, s = ref.norm(x, w, eps, residual, group)
    if residual_out is not None:
        inside(residual_out, t, ref.stored(t, x.dtype, 2.0 ** -24 * t.abs()))
    # the mean is a sum of at most 32768 fp32 terms in a tree of chains of at most 64: 2^-17 of itself,
    # so 2^-18 of its root; the products and the root add a few roundings more
    slack = 2.0 ** -17 * y.abs()
    if out is not None:
        inside(out, y, ref.stored(y, x.dtype, slack))
    if group is not None:
        inside(scales, s, 2.0 ** -16 * s)
        width = group or y.shape[1]
        big = s.repeat_interleave(width, dim=1)[:, :y.shape[1]]
        # e4m3 has 4 significant bits (half a unit: 2^-4) and steps of 2^-9 below 2^-6
        got = out8.view(torch.float8_e4m3fn).to(torch.float64) * big
        inside(got, y, 2.0 ** -4 * y.abs() * (1 + 2.0 ** -14) + 2.0 ** -10 * big + 2.0 ** -16 * y.abs())


@pytest.mark.parametrize("T,H,dtype,with_res,group,w32", [
    (1, 7168, BF16, True, None, False), (53, 7168, BF16, True, 0, False), (3, 7168, F16, False, 128, True),
    (300, 256, BF16, True, 128, False), (517, 64, F16, True, 0, False), (70, 8, BF16, False, None, True),
    (5, 14336, BF16, True, 128, True), (2, 32768, F16, True, 0, False), (9, 9000, BF16, True, 128, False),
    (7, 1, BF16, True, 0, False), (33, 129, F16, True, 128, False), (4, 4099, BF16, True, 0, True),
    (2, 32767, BF16, False, 128, False), (1000, 136, BF16, True, 128, False), (2, 16392, F16, True, 128, False),
])
def test_norm_sizes(T, H, dtype, with_res, group, w32):
    g = gen(T * 100003 + H)
    x = randn(g, T, H, dtype=dtype)
    r = randn(g, T, H, dtype=dtype, scale=2.0) if with_res else None
    w = randn(g, H, dtype=F32 if w32 else dtype)
    out, ro = torch.empty_like(x), torch.empty_like(x) if with_res else None
    o8 = sc = None
    if group is not None:
        o8 = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
        sc = torch.empty(T, -(-H // (group or H)), device="cuda")
    rel.add_rmsnorm(x, w, 1e-5, out=out, residual=r, residual_out=ro, out8=o8, scales=sc, group=group or 0)
    check_norm(x, w, 1e-5, r, group, out, ro, o8, sc)


@pytest.mark.parametrize("T,H,group", [(700, 258, 128), (401, 770, 0), (19, 1501, 128), (40, 2050, 128), (330, 3001, 0),
                                       (310, 4098, 128), (309, 7170, 0), (33, 13001, 128), (160, 20002, 128),
                                       (155, 20001, 0)])
def test_norm_widths_not_of_eight(T, H, group):
    """Pairs and single elements, every count of threads per row, more rows than blocks at work at once."""
    test_norm_sizes(T, H, BF16, True, group, False)


@pytest.mark.parametrize("H,off,pad", [(256, 0, 8), (256, 1, 3), (264, 8, 8), (250, 2, 6)])
def test_norm_strides_and_in_place(H, off, pad):
    """Row views into wider buffers (aligned and not), residual updated in place, out over x;
    what lies between the rows stays as it was."""
    g = gen(H + off)
    buf = randn(g, 37, H + off + pad)
    x, res = buf[:, off:off + H], randn(g, 37, H + off + pad)
    r = res[:, off:off + H]
    x0, r0, b0, s0 = x.clone(), r.clone(), buf.clone(), res.clone()
    w = randn(g, H)
    wide8 = torch.full((37, H + 5), 77, dtype=torch.uint8, device="cuda")
    sc = torch.empty(37, -(-H // 128), device="cuda")
    rel.add_rmsnorm(x, w, 1e-6, out=x, residual=r, residual_out=r, out8=wide8[:, :H], scales=sc, group=128)
    check_norm(x0, w, 1e-6, r0, 128, x, r, wide8[:, :H].contiguous(), sc)
    b0[:, off:off + H], s0[:, off:off + H] = x, r
    assert torch.equal(b0, buf) and torch.equal(s0, res) and bool((wide8[:, H:] == 77).all())


@pytest.mark.parametrize("H", [512, 300])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_odd_values(H, group):
    """Zero rows, tiny and huge values, an infinity and a NaN: each stays in its own row."""
    g = gen(H)
    x = randn(g, 6, H)
    x[1] = 0.0
    x[2] *= 2.0 ** -60
    x[3] *= 2.0 ** 40
    x[4, 17] = math.inf
    x[5, 5] = math.nan
    w = randn(g, H)
    out = torch.empty_like(x)
    o8 = torch.empty(6, H, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(6, -(-H // (group or H)), device="cuda")
    rel.add_rmsnorm(x, w, 1e-6, out=out, out8=o8, scales=sc, group=group)
    check_norm(x[:4], w, 1e-6, None, group, out[:4], None, o8[:4], sc[:4])
    assert bool((o8[1].float() == 0).all()) and bool((sc[1] == 0).all())
    # an infinite mean: 1/sqrt is 0, so the infinity's own place is NaN and the others 0
    assert bool(out[4, 17].isnan()) and bool((out[4, :17] == 0).all()) and bool(sc[4, 0].isnan())
    assert bool(out[5].isnan().all()) and bool(o8[5].float().isnan().all()) and bool(sc[5].isnan().all())


def test_norm_empty_and_8bit_alone():
    x = randn(gen(1), 4, 256)
    w = randn(gen(2), 256)
    rel.add_rmsnorm(x[:0], w, 1e-6, out=torch.empty_like(x[:0]))
    o8, sc = torch.empty(4, 256, dtype=torch.uint8, device="cuda"), torch.empty(4, 1, device="cuda")
    rel.add_rmsnorm(x, w, 1e-6, out8=o8, scales=sc)
    check_norm(x, w, 1e-6, None, 0, None, None, o8, sc)
    for kw in (dict(out=x[:3]), dict(out=x.float()), dict(out=x, residual=x[:, :128]), dict(out=x, out8=o8),
               dict(out8=o8, scales=torch.empty(4, 2, device="cuda")), dict(out=x.cpu())):
        with pytest.raises(ValueError):
            rel.add_rmsnorm(x, w, 1e-6, **kw)


# ---- plan --------------------------------------------------------------------------------------


def run_plan(ctx, new, table, free, head, P, N, stride=None):
    B, W = len(ctx), len(table[0])
    buf = torch.full((B, stride or W), -7, dtype=I32, device="cuda")
    buf[:, :W] = ints(table)
    out = dict(block_table=buf[:, :W], q_start=ints([9] * (B + 1)), kv_lens=ints([9] * B), positions=ints([9] * N),
               slots=ints([9] * N), free_head_out=ints([9]))
    err = torch.zeros(1, dtype=I32, device="cuda")
    rel.paged_plan(ints(ctx), ints(new), out["block_table"], ints(free), ints([head]), P, q_start=out["q_start"],
                   kv_lens=out["kv_lens"], positions=out["positions"], slots=out["slots"],
                   free_head_out=out["free_head_out"], err=err)
    got = {k: v.tolist() for k, v in out.items()}
    if stride:
        assert bool((buf[:, W:] == -7).all())
    return got, int(err.item())


def a_step(seed, B, P, top_ctx, top_new):
    r = random.Random(seed)
    ctx = [r.choice([0, r.randint(0, top_ctx), P * r.randint(0, top_ctx // P)]) for _ in range(B)]
    new = [r.choice([0, 1, r.randint(0, top_new)]) for _ in range(B)]
    W = max(-(-(c + n) // P) for c, n in zip(ctx, new)) + r.randint(0, 3)
    W = max(W, 1)
    ids = list(range(sum(-(-(c + n) // P) for c, n in zip(ctx, new)) + 20))
    r.shuffle(ids)
    table = []
    for c in ctx:
        have = -(-c // P)
        table.append([ids.pop() for _ in range(have)] + [-1] * (W - have))
    return ctx, new, table, ids, r


@pytest.mark.parametrize("seed,B,P,top_ctx,top_new", [
    (1, 1, 64, 0, 1), (2, 1, 16, 100, 700), (3, 53, 64, 4000, 1), (4, 255, 16, 300, 9), (5, 256, 32, 300, 40),
    (6, 257, 1, 40, 5), (7, 1021, 16, 900, 30), (8, 4096, 128, 600, 3), (9, 3, 1024, 5000, 5000)])
def test_plan_steps(seed, B, P, top_ctx, top_new):
    ctx, new, table, ids, r = a_step(seed, B, P, top_ctx, top_new)
    head, N = r.randint(0, 3), sum(new) + r.choice([0, 1, 300])
    got, err = run_plan(ctx, new, table, ids, head, P, max(N, 1), stride=len(table[0]) + r.choice([0, 3]))
    assert err == 0 and got == ref.plan(ctx, new, table, ids, head, P, max(N, 1))


@pytest.mark.parametrize("kind", ["pages", "width", "capacity", "negative new", "negative ctx", "head"])
def test_plan_refuses_whole_steps(kind):
    """A step that does not fit changes nothing and says so."""
    ctx, new, table, ids, _ = a_step(11, 40, 16, 300, 40)
    head, N = 2, sum(new)
    if kind == "pages":
        need = ref.plan(ctx, new, table, ids, head, 16, N)["free_head_out"][0]
        ids = ids[:need - 1]
    elif kind == "width":
        b = max(range(40), key=lambda i: ctx[i] + new[i])
        new[b] += 16 * (len(table[0]) + 1) - ctx[b] - new[b]
        N = sum(new)
    elif kind == "capacity":
        N -= 1
    elif kind == "negative new":
        new[7] = -1
    elif kind == "negative ctx":
        ctx[7] = -5
    else:
        head = -1
    got, err = run_plan(ctx, new, table, ids, head, 16, N)
    assert err == rel.MOE_OPS_ERR_PLAN
    assert got == dict(block_table=table, q_start=[0] * 41, kv_lens=[0] * 40, positions=[0] * N, slots=[-1] * N,
                       free_head_out=[head])


def test_plan_reports_a_negative_page():
    got, err = run_plan([3], [2], [[-1]], [0], 0, 16, 2)
    assert err == rel.MOE_OPS_ERR_INDEX and got["slots"] == [-1, -1] and got["positions"] == [3, 4]


# ---- rotary ------------------------------------------------------------------------------------


def check_rotary(N, Hq, Hkv, D, rot, inter, dtype, P=16, mscale=1.0, pos_top=5000, in_place=False, pad=0, heads_first=False,
                 skip=()):
    g = gen(N * 7 + D + rot)
    buf = randn(g, N, (Hq + 2 * Hkv) * D + pad, dtype=dtype)
    q = buf[:, :Hq * D].view(N, Hq, D)
    k = buf[:, Hq * D:(Hq + Hkv) * D].view(N, Hkv, D)
    v = buf[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(N, Hkv, D)
    pos = torch.randint(0, pos_top, (N,), generator=g, device="cuda").to(I32)
    pages = -(-N // P) + 2
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:N].to(I32)
    for n in skip:
        slots[n] = -1
    shape = (pages, Hkv, P, D) if heads_first else (pages, P, Hkv, D)
    kc, vc = (torch.full(shape, 5.0, dtype=dtype, device="cuda") for _ in range(2))
    if heads_first:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    f = rel.rope_frequencies(rot, 10000.0)
    err = torch.zeros(1, dtype=I32, device="cuda")
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    out = None if in_place else torch.empty(N, Hq, D, dtype=dtype, device="cuda")
    rel.rotary_append(q, k, v, pos, slots, f, kc, vc, q_out=out, interleaved=inter, mscale=mscale, err=err)
    assert int(err.item()) == 0
    want, mag = ref.rotate(q0, pos, f, mscale, inter)
    inside(q if in_place else out, want, ref.stored(want, dtype, ref.FP32 * mag))
    assert in_place or torch.equal(q, q0)
    assert torch.equal(k, k0) and torch.equal(v, v0)
    want, mag = ref.rotate(k0, pos, f, mscale, inter)
    kf, vf = torch.full((pages * P, Hkv, D), 5.0, dtype=torch.float64, device="cuda"), None
    bound, vf = torch.zeros_like(kf), torch.full_like(kf, 5.0)
    live = slots >= 0
    at = slots[live].long()
    kf[at], bound[at], vf[at] = want[live], ref.stored(want, dtype, ref.FP32 * mag)[live], v0[live].double()
    inside(kc.reshape(-1, Hkv, D), kf, bound)
    inside(vc.reshape(-1, Hkv, D), vf, torch.zeros_like(vf))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("N,Hq,Hkv,D,rot,dtype", [
    (1, 96, 8, 128, 128, BF16), (53, 12, 2, 128, 64, F16), (300, 4, 4, 64, 64, BF16), (77, 6, 1, 64, 16, BF16),
    (9, 5, 5, 64, 40, F16), (20, 3, 1, 128, 104, BF16), (11, 2, 1, 6, 2, F16), (5, 2, 2, 34, 34, BF16),
    (3, 1, 1, 1024, 1024, BF16), (2000, 8, 1, 128, 128, F16)])
def test_rotary_sizes(N, Hq, Hkv, D, rot, dtype, inter):
    check_rotary(N, Hq, Hkv, D, rot, inter, dtype)


@pytest.mark.parametrize("kw", [dict(in_place=True), dict(pad=3), dict(pad=8, heads_first=True), dict(mscale=1.35),
                                dict(skip=(0, 5, 39)), dict(P=256), dict(P=1), dict(pos_top=2 ** 30)])
def test_rotary_forms(kw):
    check_rotary(40, 6, 2, 64, 32, False, BF16, **kw)
    check_rotary(40, 6, 2, 64, 64, True, F16, **kw)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("N,Hq,Hkv,D,rot,pad", [(61, 12, 2, 64, 64, 4), (700, 6, 2, 128, 104, 0), (350, 24, 4, 68, 36, 0),
                                                (600, 7, 1, 128, 128, 1), (45, 28, 4, 20, 10, 0)])
def test_rotary_narrow_pieces(N, Hq, Hkv, D, rot, pad, inter):
    """Rows, heads or rotated parts that are multiples of 4 elements, or of one, and not of 8."""
    check_rotary(N, Hq, Hkv, D, rot, inter, BF16, pad=pad)


def test_rotary_slots_out_of_range():
    """A slot outside the cache is reported and skipped; its token's q is still rotated."""
    g = gen(3)
    q, k, v = (randn(g, 4, h, 64) for h in (2, 1, 1))
    kc, vc = (torch.zeros(2, 16, 1, 64, dtype=BF16, device="cuda") for _ in range(2))
    f, pos = rel.rope_frequencies(64), ints([0, 1, 2, 3])
    for bad in (32, -2, 2 ** 31 - 1):
        err = torch.zeros(1, dtype=I32, device="cuda")
        out = torch.empty_like(q)
        rel.rotary_append(q, k, v, pos, ints([3, bad, 4, -1]), f, kc, vc, q_out=out, err=err)
        want, mag = ref.rotate(q, pos, f, 1.0, False)
        inside(out, want, ref.stored(want, BF16, ref.FP32 * mag))
        assert int(err.item()) == rel.MOE_OPS_ERR_INDEX
        used = vc.view(32, 64).float().abs().sum(dim=1) > 0
        assert used.nonzero().flatten().tolist() == [3, 4]
    with pytest.raises(ValueError):
        rel.rotary_append(q, k, v, pos, ints([3, 4, 5]), f, kc, vc)
    with pytest.raises(ValueError):
        rel.rotary_append(q, k, v, pos, pos, f.float(), kc, vc)
    with pytest.raises(ValueError):
        rel.rotary_append(q, k, v.half(), pos, pos, f, kc, vc)


# ---- attention ---------------------------------------------------------------------------------


@pytest.fixture(scope="module")
def handle():
    h = rel.PagedAttention(device=0)
    yield h
    h.close()


def a_cache(seed, ctx, new, Hq, Hkv, D, P, dtype, heads_first=False, poison=True, extra=0, q_scale=1.5):
    """Inputs of one call. With poison, every cache row that belongs to no request's tokens
    holds NaN, and the unused part of the table holds page ids that do not exist."""
    g = gen(seed)
    B = len(ctx)
    kv = [c + n for c, n in zip(ctx, new)]
    W = max(1, max(-(-max(t, 0) // P) for t in kv)) + extra
    pages = sum(-(-max(t, 0) // P) for t in kv) + 3
    ids = torch.randperm(pages, generator=g, device="cuda").tolist()
    table = torch.full((B, W), pages + 12345, dtype=I32)
    live = torch.zeros(pages, P, dtype=torch.bool)
    for b, t in enumerate(kv):
        for i in range(-(-max(t, 0) // P)):
            table[b, i] = ids.pop()
            live[table[b, i], :min(P, t - i * P)] = True
    shape = (pages, Hkv, P, D) if heads_first else (pages, P, Hkv, D)
    k, v = randn(g, *shape, dtype=dtype), randn(g, *shape, dtype=dtype)
    if heads_first:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    if poison:
        k[~live.cuda()] = math.nan
        v[~live.cuda()] = math.nan
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    q = randn(g, starts[-1], Hq, D, dtype=dtype, scale=q_scale)
    return dict(q=q, k=k, v=v, table=table.cuda(), q_start=ints(starts), kv_lens=ints(kv))


def run_attention(h, c, max_new=0, lse=True, out=None):
    q = c["q"]
    out = torch.full_like(q, 3.0) if out is None else out
    ls = torch.full(q.shape[:2], 3.0, device="cuda") if lse else None
    h.forward(q, c["k"], c["v"], c["table"], c["q_start"], c["kv_lens"], out, scale=q.shape[2] ** -0.5, lse=ls,
              max_new=max_new)
    return out, ls


def check_attention(h, c, max_new=0, every=1):
    out, ls = run_attention(h, c, max_new)
    assert h.get_error() == 0
    want, wl, slack, ls_slack = ref.attention(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_lens"],
                                              c["q"].shape[2] ** -0.5, every)
    inside(out, want, ref.stored(want, out.dtype, slack))
    inside(ls, wl, ls_slack)
    return out, ls


EDGE = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 300]


@pytest.mark.parametrize("D,G,dtype,P", [(64, 1, BF16, 16), (64, 5, F16, 32), (64, 8, BF16, 64), (128, 1, F16, 64),
                                         (128, 4, BF16, 16), (128, 12, BF16, 64), (128, 7, F16, 128),
                                         (64, 128, BF16, 256), (128, 17, BF16, 1024), (128, 96, F16, 32)])
def test_attention_one_token(handle, D, G, dtype, P):
    """One new token of requests whose lengths sit on and beside every tile edge."""
    c = a_cache(D + G, [t - 1 for t in EDGE], [1] * len(EDGE), 2 * G, 2, D, P, dtype, extra=2)
    check_attention(handle, c, max_new=1)
    check_attention(handle, c)


@pytest.mark.parametrize("D,G,dtype,P", [(64, 1, BF16, 16), (64, 6, F16, 32), (128, 1, BF16, 128), (128, 3, F16, 16),
                                         (128, 8, BF16, 64), (128, 12, BF16, 64), (64, 128, F16, 64),
                                         (128, 9, BF16, 256)])
def test_attention_chunks(handle, D, G, dtype, P):
    """Chunks of odd lengths over contexts of odd lengths, a request without new tokens and one
    without context among them; the variant hint given and not."""
    ctx = [0, 0, 5, 64, 100, 130, 257, 33]
    new = [1, 33, 0, 17, 130, 7, 65, 64]
    c = a_cache(3 * D + G, ctx, new, 2 * G, 2, D, P, dtype, heads_first=G % 2 == 0)
    check_attention(handle, c)
    check_attention(handle, c, max_new=max(new))


@pytest.mark.parametrize("new", [2, 5, 8, 16])
def test_attention_few_tokens(handle, new):
    c = a_cache(new, [0, 40, 513, 1000], [new] * 4, 16, 2, 128, 16, BF16)
    check_attention(handle, c, max_new=new)


@pytest.mark.parametrize("D,Hq,Hkv,ctx,new,every", [
    (128, 24, 2, [20000], [1], 1), (128, 16, 2, [9000, 3], [1, 1], 1), (64, 8, 1, [30000, 100, 7000], [3, 1, 2], 1),
    (128, 8, 2, [3000], [1500], 97), (128, 24, 2, [6000, 0, 100], [400, 700, 1], 53), (64, 4, 4, [0], [2500], 101)])
def test_attention_long(handle, D, Hq, Hkv, ctx, new, every):
    """Long contexts and chunks, where a row's keys are shared out and joined."""
    c = a_cache(len(ctx) + D, ctx, new, Hq, Hkv, D, 64, BF16)
    check_attention(handle, c, every=every)
    check_attention(handle, c, max_new=max(new), every=every)


@pytest.mark.parametrize("D,Hq,Hkv,ctx,new,P", [
    (64, 1, 1, [1700], [1], 16), (64, 48, 4, [11385], [4], 128), (128, 6, 1, [12315], [1], 64),
    (128, 100, 1, [17000], [1], 32), (128, 12, 2, [9000, 400], [10, 2], 64), (64, 2, 1, [40000], [2], 64),
    (128, 2, 1, [5000], [118], 64), (64, 32, 1, [2500, 16000], [3, 9], 64)])
def test_attention_many_pieces(handle, D, Hq, Hkv, ctx, new, P):
    """Few items on many CTAs: runs of pieces joined first, then the runs, with few and with many rows."""
    c = a_cache(len(ctx) + D + P, ctx, new, Hq, Hkv, D, P, BF16)
    check_attention(handle, c, every=3 if max(new) > 20 else 1)
    check_attention(handle, c, max_new=max(new), every=3 if max(new) > 20 else 1)


def test_attention_rows_without_keys(handle):
    """kv_lens below the number of new tokens leaves the first rows nothing to see: zeros and
    a log-sum of -inf; with no key at all every row is empty."""
    c = a_cache(5, [-3, 0, -40, 60], [8, 3, 40, 5], 8, 2, 64, 16, BF16)
    for hint in (0, 40):
        out, ls = check_attention(handle, c, hint)
        assert bool((out[:3] == 0).all()) and bool((ls[:3] == -math.inf).all()) and bool((out[3] != 0).any())
        assert bool((out[11:51] == 0).all())


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("hint", [0, 4])
def test_attention_unseen_values(handle, bad, hint):
    """A token of the chunk whose key or value is not finite reaches the rows that see it and
    no row before it, though they share its tile."""
    ctx, new = [10, 100], [4 if hint else 70, 4 if hint else 30]
    c = a_cache(6, ctx, new, 8, 2, 64, 16, F16)
    clean, clean_ls = run_attention(handle, c, hint)
    spoiled = 2 if hint else 40  # the new token of request 0 that is spoiled
    page, row = int(c["table"][0, (10 + spoiled) // 16]), (10 + spoiled) % 16
    for name in ("k", "v"):
        d = dict(c, **{name: c[name].clone()})
        d[name][page, row, 0, 7] = bad
        out, ls = run_attention(handle, d, hint)
        assert handle.get_error() == 0
        assert torch.equal(out[:spoiled], clean[:spoiled]) and torch.equal(ls[:spoiled], clean_ls[:spoiled])
        assert torch.equal(out[new[0]:], clean[new[0]:])                      # the other request
        assert torch.equal(out[:new[0], 4:], clean[:new[0], 4:])              # the other key head
        seeing = out[spoiled:new[0], :4]
        if name == "v":
            assert torch.equal(seeing[..., :7], clean[spoiled:new[0], :4, :7])
            want = torch.full_like(seeing[..., 7], bad)
            assert torch.equal(seeing[..., 7].nan_to_num(9.0), want.nan_to_num(9.0))
        elif math.isnan(bad):
            assert bool(seeing.isnan().all())


def test_attention_extreme_scores(handle):
    """Scores of a thousand and more: the softmax is one key's weight; and all scores equal."""
    c = a_cache(8, [200, 700], [40, 1], 8, 2, 128, 16, BF16, q_scale=200.0)
    check_attention(handle, c)
    c["q"].zero_()
    check_attention(handle, c)


def test_attention_strides(handle):
    """q inside a fused projection, out rows padded, a table that is part of a wider one, and
    caches that are halves of one allocation."""
    ctx, new = [30, 70], [20, 1]
    c = a_cache(9, ctx, new, 12, 2, 64, 16, BF16)
    want, ls0 = run_attention(handle, c)
    N = sum(new)
    fused = torch.full((N, 12 * 64 + 256), 4.0, dtype=BF16, device="cuda")
    fused[:, 128:896] = c["q"].reshape(N, 768)
    wide = torch.full((N, 12, 72), 4.0, dtype=BF16, device="cuda")
    both = torch.stack((c["k"], c["v"]), dim=2)  # [pages][P][2][Hkv][D]
    table = torch.zeros(2, c["table"].shape[1] + 5, dtype=I32, device="cuda")
    table[:, :-5] = c["table"]
    d = dict(c, q=fused[:, 128:896].view(N, 12, 64), k=both[:, :, 0], v=both[:, :, 1], table=table[:, :-5])
    out, ls = run_attention(handle, d, out=wide[..., :64])
    assert torch.equal(out, want) and torch.equal(ls, ls0) and bool((wide[..., 64:] == 4.0).all())


def test_attention_bad_pages_and_ranges(handle):
    """Pages that do not exist count as zeros and are reported; a request whose rows lie
    outside q is skipped and reported; rows of no request are not written."""
    c = a_cache(10, [50, 20], [2, 3], 4, 2, 64, 16, BF16)
    pages = c["k"].shape[0]
    for page in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        d = dict(c, table=c["table"].clone())
        d["table"][0, 1] = page
        out, _ = run_attention(handle, d)
        assert handle.get_error() == rel.MOE_OPS_ERR_INDEX
        e = dict(c, k=torch.cat((c["k"], torch.zeros_like(c["k"][:1]))), v=torch.cat((c["v"], torch.zeros_like(c["v"][:1]))))
        e["table"] = c["table"].clone()
        e["table"][0, 1] = pages
        check = run_attention(handle, e)[0]
        assert handle.get_error() == 0 and torch.equal(out, check)
    d = dict(c, kv_lens=ints([52, 900]))  # past the table: the missing pages are zeros
    run_attention(handle, d)
    assert handle.get_error() == rel.MOE_OPS_ERR_INDEX
    d = dict(c, q_start=ints([0, 2, 9]))
    out, _ = run_attention(handle, d)
    assert handle.get_error() == rel.MOE_OPS_ERR_INDEX
    assert bool((out[2:] == 3.0).all()) and torch.equal(out[:2], run_attention(handle, c)[0][:2])
    d = dict(c, q_start=ints([1, 3, 4]), kv_lens=ints([52, 21]))
    out, ls = run_attention(handle, d)
    assert bool((out[0] == 3.0).all()) and bool((out[4] == 3.0).all()) and bool((ls[0] == 3.0).all())


def test_attention_same_twice_streams_and_graphs(handle):
    """The same call gives the same bits, also on another stream, behind other calls on the
    same handle, and from a CUDA graph."""
    c = a_cache(12, [3000, 10, 700], [1, 200, 3], 24, 2, 128, 64, BF16)
    other = a_cache(13, [9000], [1], 24, 2, 128, 64, BF16)
    want = run_attention(handle, c)[0].clone()
    for _ in range(3):
        run_attention(handle, other)
        assert torch.equal(run_attention(handle, c)[0], want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    handle.forward(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_lens"], out, scale=128 ** -0.5, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph, stream=s):
        handle.forward(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_lens"], out, scale=128 ** -0.5)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_attention_refusals(handle):
    c = a_cache(14, [10], [2], 4, 2, 64, 16, BF16)
    q, k, v, t, s, n = (c[x] for x in ("q", "k", "v", "table", "q_start", "kv_lens"))
    out = torch.empty_like(q)
    for status, args, kw in [
            (rel.MOE_ERR_INVALID_ARG, (q, k, v, t, s, n, q), dict(scale=1.0)),          # out is q
            (rel.MOE_ERR_INVALID_ARG, (q, k, v, t, s, n, out), dict(scale=0.0)),
            (rel.MOE_ERR_INVALID_ARG, (q, k, v, t, s, n, out), dict(scale=math.nan)),
            (rel.MOE_ERR_INVALID_ARG, (q, k, v, t, s, n, out), dict(scale=1.0, max_new=-1)),
            (rel.MOE_ERR_UNSUPPORTED, (q, k[:, :8], v[:, :8], t, s, n, out), dict(scale=1.0)),
            (rel.MOE_ERR_INVALID_ARG, (q[:, :3], k, v, t, s, n, out[:, :3]), dict(scale=1.0))]:
        with pytest.raises(rel.MoeError) as e:
            handle.forward(*args, **kw)
        assert e.value.status == status
    bad = [(q.float(), k, v, t, s, n, out), (q, k.half(), v, t, s, n, out), (q, k, v, t.long(), s, n, out),
           (q, k, v, t, s[:1], n, out), (q, k, v, t, s, n, out[:1]), (q, k, v[:1], t, s, n, out),
           (q, k, v, t.cpu(), s, n, out), (q.cpu(), k, v, t, s, n, out)]
    for args in bad:
        with pytest.raises(ValueError):
            handle.forward(*args, scale=1.0)
    wide = torch.zeros(2, 4, 66, dtype=BF16, device="cuda")
    with pytest.raises(rel.MoeError):  # rows that are not 16-byte aligned
        handle.forward(wide[..., 2:], k, v, t, s, n, out, scale=1.0)
    handle.forward(q[:0], k, v, t, ints([0, 0]), n, out[:0], scale=1.0)
