"""The operators beside the expert layer where their types, sizes and memory end: values at the
ends of a type's range, empty and many requests, tensors that share memory, other streams and
graphs. Against plain 64-bit forms (ops_reference.py)."""
import math
import random

import pytest
import torch

import ops_reference as ref
import routed_expert_layer_gb300 as rel
from test_gpu_ops import BF16, F16, F32, I32, a_cache, check_attention, check_norm, gen, inside, ints, randn, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = rel.PagedAttention(device=0)
    yield h
    h.close()


# ---- norm --------------------------------------------------------------------------------------

WIDTHS = [512, 2048, 300, 301, 1502, 4001]  # every kernel, piece width and several counts of rows per block


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("exponent", [-120, -127, -130, -134, -140, -148])
def test_norm_8bit_of_tiny_values(H, group, exponent):
    """Rows and blocks whose largest value lies where its scale's reciprocal leaves fp32, zeros among
    them: values keep their proportions and zeros stay zeros."""
    g = gen(H - exponent)
    x = randn(g, 6, H)
    x[:, ::7] = 0.0
    x[3] *= 2.0 ** -130  # subnormal in bf16
    x[5] = 0.0
    w = randn(g, H, dtype=F32)
    w[:128 if group else H] *= 2.0 ** exponent
    out = torch.empty_like(x)
    o8 = torch.empty(6, H, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(6, -(-H // (group or H)), device="cuda")
    rel.add_rmsnorm(x, w, 1e-6, out=out, out8=o8, scales=sc, group=group)
    _, y, s = ref.norm(x, w, 1e-6, None, group)
    # fp32's subnormals are steps of 2^-149: half a step from the last product of y and from the scale's own
    # rounding. 448 times the scale's is what the largest values may lose, or all of a block whose scale is 0.
    step = 2.0 ** -150
    inside(out, y, ref.stored(y, BF16, 2.0 ** -17 * y.abs() + step))
    inside(sc, s, 2.0 ** -16 * s + 2 * step)
    big = sc.double().repeat_interleave(group or H, dim=1)[:, :H]
    got = o8.double()
    assert bool((got[y == 0] == 0).all())
    inside(got * big, y, 2.0 ** -4 * y.abs() * (1 + 2.0 ** -14) + 2.0 ** -10 * big + 2.0 ** -16 * y.abs() + 450 * step)


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.int8, torch.bool])
def test_norm_8bit_types(dtype):
    """Bits of e4m3 go to tensors of that type or of bytes only."""
    x, w = randn(gen(1), 3, 256), randn(gen(2), 256)
    o8, sc = torch.empty(3, 256, dtype=dtype, device="cuda"), torch.empty(3, 1, device="cuda")
    with pytest.raises(ValueError, match="float8_e4m3fn or uint8"):
        rel.add_rmsnorm(x, w, 1e-6, out8=o8, scales=sc)


def test_norm_scales_need_8bit_output():
    x, w = randn(gen(1), 3, 256), randn(gen(2), 256)
    with pytest.raises(ValueError, match="scales"):
        rel.add_rmsnorm(x, w, 1e-6, out=torch.empty_like(x), scales=torch.empty(3, 1, device="cuda"))


# ---- plan --------------------------------------------------------------------------------------


def test_plan_tensors_of_one_allocation():
    """Tensors one behind the other in one allocation, the table's rows with other words between them;
    lengths or the free list's head updated in place are refused."""
    ctx, new, P, W, stride = [5, 0, 33], [4, 3, 20], 16, 5, 7
    N, ids = sum(new), [9, 8, 4, 6, 7]
    sizes = dict(ctx=3, new=3, table=3 * stride, free=5, head=1, q_start=4, kv=3, pos=N, slots=N, head_out=1, err=1)
    buf = torch.zeros(sum(sizes.values()), dtype=I32, device="cuda")
    t = dict(zip(sizes, buf.split(list(sizes.values()))))
    t["table"] = t["table"].view(3, stride)
    for name, v in (("ctx", ctx), ("new", new), ("free", ids), ("head", [1])):
        t[name].copy_(ints(v))
    table = [[3, -1, -1, -1, -1], [-1] * 5, [1, 2, 0, -1, -1]]
    t["table"].fill_(-7)
    t["table"][:, :W].copy_(ints(table))
    before = buf.clone()

    def call(**kw):
        a = dict(q_start=t["q_start"], kv_lens=t["kv"], positions=t["pos"], slots=t["slots"], free_head_out=t["head_out"], err=t["err"])
        a.update(kw)
        rel.paged_plan(t["ctx"], t["new"], t["table"][:, :W], t["free"], t["head"], P, **a)

    for kw in (dict(kv_lens=t["ctx"]), dict(kv_lens=t["new"]), dict(free_head_out=t["head"]), dict(positions=t["slots"]),
               dict(q_start=buf[1:5]), dict(err=t["head"])):
        with pytest.raises(rel.MoeError) as e:
            call(**kw)
        assert e.value.status == rel.MOE_ERR_INVALID_ARG and torch.equal(buf, before)
    call()
    want = ref.plan(ctx, new, table, ids, 1, P, N)
    for name, key in (("q_start", "q_start"), ("kv", "kv_lens"), ("pos", "positions"), ("slots", "slots"), ("head_out", "free_head_out")):
        assert t[name].tolist() == want[key], key
    assert t["table"][:, :W].tolist() == want["block_table"] and bool((t["table"][:, W:] == -7).all())
    assert t["ctx"].tolist() == ctx and t["new"].tolist() == new and t["free"].tolist() == ids and t["err"].tolist() == [0]


def test_plan_without_free_pages():
    """A step inside the pages its requests have needs no free page; one that needs a page is refused whole."""
    empty, err = torch.empty(0, dtype=I32, device="cuda"), ints([0])
    for new, fits in (([1, 2], True), ([1, 20], False)):
        table = ints([[3, -1], [5, 1]])
        q_start, kv, pos, slots, head = (ints([9] * n) for n in (3, 2, sum(new), sum(new), 1))
        err.zero_()
        rel.paged_plan(ints([2, 17]), ints(new), table, empty, ints([0]), 16, q_start=q_start, kv_lens=kv, positions=pos,
                       slots=slots, free_head_out=head, err=err)
        assert table.tolist() == [[3, -1], [5, 1]] and head.tolist() == [0]
        if fits:
            assert err.tolist() == [0] and q_start.tolist() == [0, 1, 3] and kv.tolist() == [3, 19]
            assert pos.tolist() == [2, 17, 18] and slots.tolist() == [50, 17, 18]
        else:
            assert err.tolist() == [rel.MOE_OPS_ERR_PLAN] and kv.tolist() == [0, 0] and set(slots.tolist()) == {-1}


# ---- attention ---------------------------------------------------------------------------------


@pytest.mark.parametrize("D,Hq,Hkv,ctx,new", [(64, 4, 2, [4000, 40], [1, 1]), (128, 8, 1, [40000], [1]),
                                              (64, 4, 4, [3000, 200], [150, 9]), (128, 24, 2, [6000], [40]),
                                              (64, 4, 2, [2000] * 160, [1] * 160)])
@pytest.mark.parametrize("nats", [16.0, 18.0, 20.0])
def test_attention_f16_small_weights(handle, D, Hq, Hkv, ctx, new, nats):
    """One key's score lies 16 to 20 above thousands of others' and its value is zero: what is left is
    the others' sum, though none of their weights is an f16 number of its own beside 1."""
    c = a_cache(len(ctx) + D, ctx, new, Hq, Hkv, D, 64, F16)
    c["q"].zero_()
    c["q"][..., 0] = 8.0
    c["k"] = torch.where(c["k"].isnan(), c["k"], torch.zeros_like(c["k"]))
    c["v"] = (100.0 + 10.0 * c["v"].float()).to(F16)
    for b in range(len(ctx)):
        first = int(c["table"][b, 0])
        c["k"][first, 0, :, 0] = nats * D ** 0.5 / 8.0
        c["v"][first, 0] = 0.0
    every = 1 if max(new) == 1 else 37
    want, wl, slack, ls_slack = ref.attention(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_lens"], D ** -0.5,
                                              every)
    # a weight is held to half of 2^-24 (f16's smallest) where the largest is at least 2^7: 2^-32 of the
    # largest, for every key; values are below 160
    seen = c["kv_lens"].double().max()
    for hint in (0, max(new)):
        out, ls = run_attention(handle, c, hint)
        assert handle.get_error() == 0
        inside(out, want, ref.stored(want, F16, slack + 160.0 * seen * 2.0 ** -32))
        inside(ls, wl, ls_slack)


def test_handle_is_ready_on_every_stream():
    """A new handle's workspace has been cleared when the call returns, whatever the default stream was
    busy with: streams that do not wait for that one may use the handle at once."""
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # some 0.1 s of the default stream
    h = rel.PagedAttention(device=0)
    assert torch.cuda.default_stream().query()
    h.close()


def test_attention_without_requests(handle):
    """A call without requests, with rows of q or without, writes nothing."""
    c = a_cache(14, [10], [2], 4, 2, 64, 16, BF16)
    none = torch.empty(0, dtype=I32, device="cuda")
    for rows in (0, 2):
        out = torch.full_like(c["q"][:rows], 3.0)
        handle.forward(c["q"][:rows], c["k"], c["v"], c["table"][:0], ints([0]), none, out, scale=1.0)
        assert bool((out == 3.0).all()) and handle.get_error() == 0


@pytest.mark.parametrize("by", ["columns", "heads", "rows"])
def test_attention_out_beside_q(handle, by):
    """q and out in one allocation without a shared element: halves of a row, of a head's row, every
    other row."""
    c = a_cache(15, [30, 70], [20, 3], 6, 2, 64, 16, BF16)
    want, _ = run_attention(handle, c)
    N = c["q"].shape[0]
    if by == "columns":
        buf = torch.zeros(N, 12, 64, dtype=BF16, device="cuda")
        q, out = buf[:, 6:], buf[:, :6]
    elif by == "heads":
        buf = torch.zeros(N, 6, 128, dtype=BF16, device="cuda")
        q, out = buf[..., :64], buf[..., 64:]
    else:
        buf = torch.zeros(2 * N, 6, 64, dtype=BF16, device="cuda")
        q, out = buf[1::2], buf[::2]
    q.copy_(c["q"])
    run_attention(handle, dict(c, q=q), out=out)
    assert torch.equal(out, want) and torch.equal(q, c["q"])
    with pytest.raises(rel.MoeError):
        run_attention(handle, dict(c, q=q), out=q)
    if by == "columns":
        with pytest.raises(rel.MoeError):  # the last head of one is the first of the other
            run_attention(handle, dict(c, q=buf[:, 5:11]), out=buf[:, :6])


@pytest.mark.parametrize("B", [128, 129, 257, 600])
@pytest.mark.parametrize("top", [1, 40])
def test_attention_many_requests(handle, B, top):
    """More requests than a CTA keeps cost sums for, idle ones at both ends of the batch, at the ends of
    the runs that share a sum, and whole runs of them."""
    r = random.Random(B + top)
    seg = -(-B // 128)
    ctx, new = [], []
    for b in range(B):
        idle = b < 5 or b >= B - 4 or b % (3 * seg) >= 2 * seg or b % seg == seg - 1 and r.random() < 0.5
        ctx.append(r.choice([0, 1, 63, 64, r.randint(0, 200), r.randint(0, 900) if b % 50 == 9 else 5]))
        new.append(0 if idle else r.choice([1, 1, 1, r.randint(1, top)]))
    c = a_cache(B + top, ctx, new, 4, 2, 64, 16, BF16)
    check_attention(handle, c)
    check_attention(handle, c, max_new=top)
    check_attention(handle, c, max_new=1)


# ---- streams and graphs ------------------------------------------------------------------------


def test_two_handles_on_two_streams(handle):
    """Two handles at work at once, each on a stream of its own, give what each gives alone."""
    other = rel.PagedAttention(device=0)
    calls = [a_cache(21, [5000, 10, 700], [1, 200, 3], 24, 2, 128, 64, BF16), a_cache(22, [9000, 40], [1, 2], 24, 2, 128, 64, BF16)]
    want = [run_attention(handle, c)[0].clone() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for h, c, out, s in zip((handle, other), calls, outs, streams):
            h.forward(c["q"], c["k"], c["v"], c["table"], c["q_start"], c["kv_lens"], out, scale=128 ** -0.5, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert handle.get_error() == 0 and other.get_error() == 0
    other.close()


def test_step_on_another_stream_and_in_a_graph():
    """Plan, rotary with its append and the norm, one behind the other on a side stream and from a
    CUDA graph of all three, give what they give call by call."""
    g = gen(31)
    B, P, Hq, Hkv, D = 70, 16, 6, 2, 64
    r = random.Random(31)
    ctx, new = [r.randint(0, 90) for _ in range(B)], [r.choice([0, 1, 9]) for _ in range(B)]
    N, W = sum(new), 8
    ids = list(range(B * W))
    r.shuffle(ids)
    table0 = ints([[ids.pop() for _ in range(-(-t // P))] + [-1] * (W - -(-t // P)) for t in ctx])
    lens, fresh, free = ints(ctx), ints(new), ints(ids)
    q, k, v = (randn(g, N, h, D) for h in (Hq, Hkv, Hkv))
    x, res, w = randn(g, N, 2048), randn(g, N, 2048), randn(g, 2048)
    f = rel.rope_frequencies(D)

    def buffers():
        return dict(table=table0.clone(), q_start=ints([0] * (B + 1)), kv=ints([0] * B), pos=ints([0] * N), slots=ints([0] * N),
                    head=ints([0]), q=torch.empty_like(q), kc=torch.zeros(B * W, P, Hkv, D, dtype=BF16, device="cuda"),
                    vc=torch.zeros(B * W, P, Hkv, D, dtype=BF16, device="cuda"), h=torch.empty_like(x), n=torch.empty_like(x),
                    n8=torch.empty(N, 2048, dtype=torch.uint8, device="cuda"), sc=torch.empty(N, 16, device="cuda"))

    head = ints([3])

    def step(b, stream=None):
        rel.paged_plan(lens, fresh, b["table"], free, head, P, q_start=b["q_start"], kv_lens=b["kv"], positions=b["pos"],
                       slots=b["slots"], free_head_out=b["head"], stream=stream)
        rel.rotary_append(q, k, v, b["pos"], b["slots"], f, b["kc"], b["vc"], q_out=b["q"], stream=stream)
        rel.add_rmsnorm(x, w, 1e-6, out=b["n"], residual=res, residual_out=b["h"], out8=b["n8"], scales=b["sc"], group=128,
                        stream=stream)

    want, side, captured = buffers(), buffers(), buffers()
    rel.paged_plan(lens, fresh, want["table"], free, head, P, q_start=want["q_start"], kv_lens=want["kv"],
                   positions=want["pos"], slots=want["slots"], free_head_out=want["head"])
    torch.cuda.synchronize()
    plan = ref.plan(ctx, new, table0.tolist(), ids, 3, P, N)
    assert want["slots"].tolist() == plan["slots"] and want["table"].tolist() == plan["block_table"]
    want["table"].copy_(table0)
    step(want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(side, s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(captured)
    for _ in range(2):
        captured["table"].copy_(table0)
        captured["kc"].zero_()
        graph.replay()
        torch.cuda.synchronize()
    for name in want:
        assert torch.equal(want[name], side[name]) and torch.equal(want[name], captured[name]), name
