"""8-bit projections on the GPU: quantisation and the product with block scales, against plain 64-bit forms
(draft_reference.py, where every tolerance is derived)."""
import math
import random

import pytest
import torch

import draft_reference as dref
import ops_reference as ref
import routed_expert_layer_gb300 as rel
from test_gpu_ops import inside

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3 = torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def run_quantize(x, group, rows):
    T, H = x.shape
    out8 = torch.full((T, H), 99, dtype=torch.uint8, device="cuda").view(E4M3)
    scales = torch.full((-(-T // rows), -(-H // (group or H))), -1.0, device="cuda")
    rel.quantize8(x, out8, scales, group=group, rows=rows)
    return out8, scales


def check_quantize(x, group, rows, out8, scales):
    y, s = dref.quantize(x, group, rows)
    inside(scales, s, 2.0 ** -24 * s + 2.0 ** -150)
    # e4m3 has 4 significant bits (half a unit: 2^-4) and steps of 2^-9 below 2^-6; the quotient of fp32 values has
    # two roundings of 2^-24 before
    inside(out8.view(E4M3).float(), y, y.abs() * (2.0 ** -4 + 2.0 ** -20) + 2.0 ** -10)
    # to the bit: the quotient in fp32, rounded to nearest even
    T, H = x.shape
    big = scales.repeat_interleave(rows, dim=0)[:T].repeat_interleave(group or H, dim=1)[:, :H]
    want = torch.where(big > 0, x.float() / big, torch.zeros_like(big)).to(E4M3)
    assert torch.equal(out8.view(E4M3).float(), want.float())


@pytest.mark.parametrize("T,H,group,rows,dtype", [
    (1, 128, 128, 1, BF16), (1, 1, 128, 1, F16), (53, 7168, 128, 1, BF16), (3, 12288, 0, 1, F16), (300, 520, 128, 1, BF16),
    (7, 129, 128, 1, BF16), (5, 4099, 0, 1, BF16), (65, 72, 0, 1, F16), (2, 32768, 0, 1, BF16), (1000, 136, 128, 1, F16),
    (1, 1, 128, 128, BF16), (128, 128, 128, 128, F16), (300, 700, 128, 128, BF16), (129, 257, 128, 128, F16), (1811, 7152, 128, 128, BF16),
    (40, 100000, 0, 1, BF16), (4096, 8, 0, 1, BF16), (517, 7168, 128, 1, F16), (2000, 1024, 0, 1, BF16), (16, 16384, 128, 128, BF16),
])
def test_quantize(T, H, group, rows, dtype):
    x = (torch.randn(T, H, generator=gen(T + H), device="cuda") * 3).to(dtype)
    check_quantize(x, group, rows, *run_quantize(x, group, rows))


@pytest.mark.parametrize("group,rows", [(128, 1), (0, 1), (128, 128)])
@pytest.mark.parametrize("H", [512, 301])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_quantize_odd_values(group, rows, H, dtype):
    """Zeros, the type's smallest and largest values and values between two e4m3 numbers in blocks of their own; an
    infinity and a NaN stay in theirs."""
    T = 6 * rows
    x = torch.randn(T, H, generator=gen(H), device="cuda").to(dtype)
    part = lambda i: x[i * rows:(i + 1) * rows]
    tiny, top = torch.finfo(dtype).smallest_normal, torch.finfo(dtype).max
    part(1).zero_()
    part(2).copy_((part(2).float() * tiny).to(dtype))       # subnormal, or near
    part(3).copy_(torch.where(part(3) > 0, top, -top))
    grid = torch.arange(H, device="cuda") % 449
    part(4).copy_(grid.to(dtype).expand(rows, H))            # halves between e4m3 numbers among them
    part(4)[:, 0::128] = 448.0
    out8, scales = run_quantize(x, group, rows)
    check_quantize(x, group, rows, out8, scales)
    assert bool((scales[1] == 0).all()) and bool((out8.float()[rows:2 * rows] == 0).all())
    part(0)[0, 17] = math.inf
    part(5)[0, 200] = math.nan
    again, s2 = run_quantize(x, group, rows)
    assert torch.equal(again[rows:5 * rows].float(), out8[rows:5 * rows].float()) and torch.equal(s2[1:5], scales[1:5])
    assert math.isinf(float(s2[0, 0])) and bool(again.float()[0, 17].isnan())
    width = 128 if group else H
    first = again.float()[0, :width]
    assert bool((torch.cat([first[:17], first[18:]]) == 0).all())
    b = 200 // width
    assert bool(s2[5, b].isnan()) and bool(again.float()[5 * rows:6 * rows, b * width:(b + 1) * width].isnan().all())
    if group:
        assert torch.equal(again[:rows, 128:].float(), out8[:rows, 128:].float())


@pytest.mark.parametrize("off,pad,H", [(0, 8, 256), (8, 8, 264), (1, 2, 250), (2, 6, 130), (3, 13, 1)])
@pytest.mark.parametrize("group,rows", [(128, 1), (0, 1), (128, 128)])
def test_quantize_strides(off, pad, H, group, rows):
    """Rows inside wider buffers, aligned and not; what lies between them stays."""
    T = 140
    buf = torch.randn(T, H + off + pad, generator=gen(H), device="cuda").to(BF16)
    x = buf[:, off:off + H]
    wide = torch.full((T, H + off + pad), 77, dtype=torch.uint8, device="cuda")
    scales = torch.empty(-(-T // rows), -(-H // (group or H)), device="cuda")
    rel.quantize8(x, wide[:, off:off + H], scales, group=group, rows=rows)
    check_quantize(x, group, rows, wide[:, off:off + H].contiguous(), scales)
    assert bool((wide[:, :off] == 77).all()) and bool((wide[:, off + H:] == 77).all())


def test_quantize_refusals():
    x = torch.zeros(4, 256, dtype=BF16, device="cuda")
    o, s = torch.empty(4, 256, dtype=E4M3, device="cuda"), torch.empty(4, 2, device="cuda")
    rel.quantize8(x, o, s)
    rel.quantize8(x[:0], o[:0], s[:0])
    for kw in (dict(group=64), dict(group=0), dict(rows=128), dict(rows=2)):
        with pytest.raises((ValueError, rel.MoeError)):
            rel.quantize8(x, o, s, **kw)
    with pytest.raises(rel.MoeError):  # a scale per row of 128 rows
        rel.quantize8(x, o, torch.empty(1, 1, device="cuda"), group=0, rows=128)
    for args in ((x.float(), o, s), (x, o[:3], s), (x, o.view(torch.int8), s), (x, o, s.double()), (x, o, s[:, :1]), (x[0], o, s),
                 (x, o.view(torch.float8_e5m2), s), (x, o.t(), s)):
        with pytest.raises(ValueError):
            rel.quantize8(*args)
    with pytest.raises(rel.MoeError):  # out8 in x's bytes
        rel.quantize8(x, x.view(torch.uint8)[:, :256], s)


@pytest.fixture(scope="module")
def mm():
    h = rel.Matmul8(device=0)
    yield h
    h.close()


class Product:
    def __init__(self, T, N, K, dtype=BF16, row_scale=False, seed=0, pad=0, odd_scales=False):
        g = gen(seed + T + N + K)
        bytes8 = lambda r: torch.randn(r, K + pad, generator=g, device="cuda").mul(120).clamp(-448, 448).to(E4M3)[:, :K]
        self.a8, self.w8 = bytes8(T), bytes8(N)
        blocks = -(-K // 128)
        scale = lambda r, b: torch.exp(torch.randn(r, b, generator=g, device="cuda")) * 0.01
        self.a_scales, self.w_scales = scale(T, 1 if row_scale else blocks), scale(-(-N // 128), blocks)
        self.out = torch.full((T, N), 7.0, dtype=dtype, device="cuda")

    def forward(self, mm, **kw):
        mm.forward(self.a8, self.a_scales, self.w8, self.w_scales, self.out, **kw)
        return self.out

    def check(self, mm):
        out = self.forward(mm)
        want, slack = dref.matmul8(self.a8, self.a_scales, self.w8, self.w_scales)
        inside(out, want, ref.stored(want, out.dtype, slack))
        assert mm.get_error() == 0


SHAPES = [(1, 1, 16), (1, 128, 128), (1, 7168, 12288), (2, 100, 4096), (5, 129, 272), (8, 14336, 7168), (16, 257, 2048),
          (17, 3584, 7168), (33, 1024, 144), (53, 14336, 7168), (64, 640, 12288), (65, 64, 8192), (100, 511, 1040), (127, 256, 256),
          (128, 255, 7168), (129, 1811, 7152), (255, 100, 384), (256, 2048, 7168), (257, 300, 640), (300, 14336, 512), (517, 1811, 7152),
          (1000, 1000, 1008), (1024, 7168, 256), (2049, 129, 2064), (4096, 513, 128), (300, 8, 16)]


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_matmul8(mm, T, N, K):
    Product(T, N, K, BF16 if T % 2 else F16, row_scale=N % 3 == 0).check(mm)


@pytest.mark.parametrize("seed", range(12))
def test_matmul8_random_sizes(mm, seed):
    r = random.Random(seed)
    log = lambda lo, hi: int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))
    Product(log(1, 3000), log(1, 5000), 16 * log(1, 400), r.choice([BF16, F16]), r.random() < 0.3, seed, pad=r.choice([0, 16, 112])).check(mm)


@pytest.mark.parametrize("T,N,K", [(3, 200, 400), (130, 300, 1008), (600, 260, 256)])
def test_matmul8_strides(mm, T, N, K):
    """Rows of every tensor inside wider buffers, out at odd addresses; what lies between the rows of out stays."""
    for off in (0, 1, 8):
        p = Product(T, N, K, pad=48, seed=off)
        blocks = -(-K // 128)
        p.a_scales = torch.nn.functional.pad(p.a_scales, (0, 3))[:, :blocks]
        p.w_scales = torch.nn.functional.pad(p.w_scales, (0, 5))[:, :blocks]
        wide = torch.full((T, N + off + 7), 7.0, dtype=BF16, device="cuda")
        p.out = wide[:, off:off + N]
        p.check(mm)
        assert bool((wide[:, :off] == 7).all()) and bool((wide[:, off + N:] == 7).all())


def test_matmul8_bytes_views_and_nothing(mm):
    """Tensors of bytes, a column of a wider tensor as the scales per row, and calls without rows or columns."""
    p = Product(33, 300, 528, row_scale=True)
    want = p.forward(mm).clone()
    wide = torch.full((33, 5), 9.0, device="cuda")
    wide[:, 3:4] = p.a_scales
    p.a8, p.w8, p.a_scales = p.a8.view(torch.uint8), p.w8.view(torch.uint8), wide[:, 3:4]
    p.out = torch.zeros_like(p.out)
    assert torch.equal(p.forward(mm), want)
    p.w8, p.w_scales, p.out = p.w8[:0], p.w_scales[:0], p.out[:, :0]
    p.forward(mm)
    assert mm.get_error() == 0


def test_matmul8_beside_attention(mm):
    """A product and an attention call on two streams at once, both of which fill tensor memory."""
    attn = rel.PagedAttention(device=0)
    p = Product(200, 4000, 4096)
    g = gen(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
    k, v, q = rand(40, 64, 2, 128), rand(40, 64, 2, 128), rand(300, 16, 128)
    table = torch.arange(40, dtype=torch.int32, device="cuda")[None]
    start = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    kv = torch.tensor([2500], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    call = lambda s=None: attn.forward(q, k, v, table, start, kv, out, scale=0.1, stream=s)
    call()
    want = p.forward(mm).clone(), out.clone()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        p.out.zero_(), out.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            p.forward(mm, stream=a)
            call(b)
        torch.cuda.synchronize()
        assert torch.equal(p.out, want[0]) and torch.equal(out, want[1])
    assert mm.get_error() == 0 and attn.get_error() == 0
    attn.close()


@pytest.mark.parametrize("T", [4, 200, 700])
def test_matmul8_odd_values(mm, T):
    """NaN and infinite scales and NaN values reach their row or column and no other; zeros and huge scales."""
    p = Product(T, 300, 640)
    clean = p.forward(mm).clone()
    p.a8.view(torch.uint8)[1, 130] = 0x7F              # e4m3's NaN
    p.a_scales[2, 3] = math.nan
    p.a_scales[3, 0] = math.inf
    out = p.forward(mm).clone()
    assert bool(out[1:3].isnan().all()) and not bool(out[3].isfinite().any())
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[1:4] = False
    assert torch.equal(out[keep], clean[keep])
    p.w8.view(torch.uint8)[77, 5] = 0xFF
    p.w_scales[2, 4] = math.nan                         # columns 256..299
    out = p.forward(mm)
    cols = torch.ones(300, dtype=torch.bool, device="cuda")
    cols[77] = False
    cols[256:] = False
    assert bool(out[:, ~cols].isnan().all()) and torch.equal(out[keep][:, cols], clean[keep][:, cols])
    p = Product(T, 300, 640)
    p.a_scales[0] = 0.0
    p.a_scales[1] = 2.0 ** -100
    p.a_scales[3] = 2.0 ** 100
    p.check(mm)


def test_matmul8_is_the_same_every_time(mm):
    """The same call gives the same bits: sums do not depend on timing."""
    for T, N, K in ((1, 7168, 12288), (53, 2048, 7168), (200, 1000, 4096), (1500, 2000, 2048)):
        p = Product(T, N, K)
        first = p.forward(mm).clone()
        for _ in range(5):
            p.out.fill_(0)
            assert torch.equal(p.forward(mm), first)


def test_matmul8_streams_graphs_and_handles(mm):
    """A side stream, a captured call replayed on other inputs, and two handles on two streams at once."""
    p, q = Product(40, 2000, 4096, seed=1), Product(300, 1500, 2048, seed=2)
    want = [t.forward(mm).clone() for t in (p, q)]
    torch.cuda.synchronize()
    other = rel.Matmul8(device=0)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        p.out.zero_(), q.out.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            p.forward(mm, stream=a)
            q.forward(other, stream=b)
        torch.cuda.synchronize()
        assert torch.equal(p.out, want[0]) and torch.equal(q.out, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.forward(mm)
        q.forward(mm)
    p.out.zero_(), q.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.out, want[0]) and torch.equal(q.out, want[1])
    p.a_scales.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.out, want[0] * 2)
    assert mm.get_error() == 0 and other.get_error() == 0
    other.close()
    with pytest.raises(ValueError):
        p.forward(other)


def test_matmul8_after_the_norm_and_quantize(mm):
    """The scales that the norm and quantize8 write, as they are: a projection of the norm's 8-bit output is the product of
    its 16-bit output within the 8-bit roundings."""
    g = gen(5)
    T, H, N = 37, 7168, 640
    x = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    w = (torch.randn(N, H, generator=g, device="cuda") * H ** -0.5).to(BF16)
    gamma = torch.ones(H, dtype=BF16, device="cuda")
    w8, ws = run_quantize(w, 128, 128)
    for group in (0, 128):
        o8, s = torch.empty(T, H, dtype=E4M3, device="cuda"), torch.empty(T, -(-H // (group or H)), device="cuda")
        rel.add_rmsnorm(x, gamma, 1e-6, out8=o8, scales=s, group=group)
        out = torch.empty(T, N, dtype=BF16, device="cuda")
        mm.forward(o8, s, w8, ws, out)
        want, slack = dref.matmul8(o8, s, w8, ws)
        inside(out, want, ref.stored(want, BF16, slack))
        # a value is off by 2^-4 of itself at most, or by 2^-10 scales; the sum's error is at most the sum of the terms'
        y = ref.norm(x, gamma, 1e-6)[1]
        full, size = y @ w.double().t(), y.abs() @ w.double().abs().t()
        assert bool(((out.double() - full).abs() <= 0.14 * size).all())


def test_matmul8_refusals(mm):
    p = Product(4, 200, 256)
    for field, bad in (("a8", p.a8[:, :128]), ("a8", p.a8.float()), ("a8", p.a8.view(torch.int8)), ("w8", p.w8.cpu()),
                       ("a_scales", p.a_scales[:3]), ("a_scales", p.a_scales.double()), ("w_scales", p.w_scales[:1]), ("out", p.out[:, :100]),
                       ("out", p.out.float()), ("out", p.out[0])):
        q = Product(4, 200, 256)
        setattr(q, field, bad)
        with pytest.raises(ValueError):
            q.forward(mm)
    q = Product(4, 200, 264)
    with pytest.raises(rel.MoeError):  # K not a multiple of 16
        q.forward(mm)
    q = Product(4, 200, 256, pad=8)
    with pytest.raises(rel.MoeError):  # row strides
        q.forward(mm)
    q = Product(4, 200, 256)
    q.a8 = torch.zeros(4 * 256 + 8, dtype=torch.uint8, device="cuda")[8:].view(4, 256)
    with pytest.raises(rel.MoeError):  # address
        q.forward(mm)
    q = Product(4, 256, 256)
    q.out = q.w8.view(torch.uint8)[:8].view(BF16).view(4, 256)
    with pytest.raises(rel.MoeError):  # out in the weights
        q.forward(mm)
    q = Product(4, 200, 256)
    q.a8, q.a_scales, q.out = q.a8[:0], q.a_scales[:0], q.out[:0]
    q.forward(mm)
    assert mm.get_error() == 0 and mm.device_bytes() > 0
