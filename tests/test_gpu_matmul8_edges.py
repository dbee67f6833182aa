"""8-bit projections on the GPU at the edges of the values' and the calls' range, and products of every way of sharing them out
(test_gpu_matmul8.py has the others)."""
import pytest
import torch

import draft_reference as dref
import ops_reference as ref
import routed_expert_layer_gb300 as rel
from test_gpu_matmul8 import BF16, E4M3, F16, Product, gen, inside, run_quantize

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    h = rel.Matmul8(device=0)
    yield h
    h.close()


@pytest.mark.parametrize("group,rows", [(128, 1), (0, 1), (128, 128)])
@pytest.mark.parametrize("H", [512, 301])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_quantize_negative_zeros(group, rows, H, dtype):
    """The bytes of e4m3(x / s), zeros of both signs and values that round to them among x. A block of zeros has zeros
    (0x00), whatever their sign."""
    T = 4 * rows
    x = torch.randn(T, H, generator=gen(H), device="cuda")
    x[:, 3::7] = -0.0
    x[:, 5::7] = 0.0
    x[:, 6::7] *= 2.0 ** -14
    x[rows:2 * rows] = -0.0
    x = x.to(dtype)
    out8, scales = run_quantize(x, group, rows)
    big = scales.repeat_interleave(rows, dim=0)[:T].repeat_interleave(group or H, dim=1)[:, :H]
    want = torch.where(big > 0, x.float() / big, torch.zeros_like(big)).to(E4M3).view(torch.uint8)
    assert bool((want == 0x80).any()) and bool((want == 0).any()) and bool((want[rows:2 * rows] == 0).all())
    assert torch.equal(out8.view(torch.uint8), want)


# One CTA a tile, with one row of tiles and with two, and a pair of CTAs (on 152 SMs).
@pytest.mark.parametrize("T,N,K", [(6, 400, 640), (200, 300, 1168), (1291, 1677, 1040)])
@pytest.mark.parametrize("row_scale", [False, True])
def test_matmul8_scales_out_of_range(mm, T, N, K, row_scale):
    """Scales whose product lies below fp32's normal range or above its largest value."""
    p = Product(T, N, K, row_scale=row_scale)
    clean = p.forward(mm).clone()
    small = lambda r: (torch.randint(0, 8, (r, K), generator=gen(r), device="cuda") +
                       128 * torch.randint(0, 2, (r, K), generator=gen(r + 1), device="cuda")).to(torch.uint8)  # up to 7 * 2^-9
    a8, w8 = p.a8.view(torch.uint8), p.w8.view(torch.uint8)
    a8[:2] &= 0x7F                                  # positive: sums of some 2^20
    w8[128:256] &= 0x7F
    p.a_scales[0] = 1.1 * 2.0 ** -72
    p.a_scales[1] = -1.1 * 2.0 ** -77
    p.w_scales[1] = 1.27 * 2.0 ** -74               # products of 2^-146 (3 bits left) and 2^-151 (none)
    a8[2:5] = small(3)
    w8[:128] = small(128)
    p.a_scales[2:4] = 1.5 * 2.0 ** 66
    p.w_scales[0] = 1.25 * 2.0 ** 66                # 2^133: sums of some 2^-10
    a8[3] = 0                                       # infinity times 0
    p.a_scales[4] = 0.0
    p.w_scales[2, 1] = 0.0
    out = p.forward(mm)
    want, slack = dref.matmul8(p.a8, p.a_scales, p.w8, p.w_scales)
    # Below 2^-126 the product of two scales is off by half of 2^-149 at most, and a block's sum is 128 * 448^2 < 2^25 at most.
    # (Where one is infinite there is no bound to hold: looked at apart.)
    blocks = -(-K // 128)
    apart = torch.zeros_like(want, dtype=torch.bool)
    apart[2:4, :128] = True
    inside(out.masked_fill(apart, 0.0), want.masked_fill(apart, 0.0), ref.stored(want, BF16, slack + blocks * 2.0 ** -125))
    assert bool((want[0, 128:256] > 2.0 ** -125).all()) and bool((out[0, 128:256] != 0).all())
    assert not bool(out[2:4, :128].isfinite().any()) and bool(out[3, :128].isnan().all())
    assert bool((out[3, 128:] == 0).all()) and bool((out[4] == 0).all())
    assert torch.equal(out[5:, 384:], clean[5:, 384:])  # rows and columns whose scales and values are as they were
    assert mm.get_error() == 0


def test_matmul8_of_seconds(mm):
    """A product that takes more than two seconds, the time after which a wait inside the kernel gives up: its waits are
    for a unit of the work each, so no error is raised. Small whole numbers: every sum is exact."""
    T = N = 458 * 256
    K = 1832 * 128
    need = T * K + N * K + 2 * T * N
    if torch.cuda.mem_get_info()[0] < 1.1 * need:
        pytest.skip("needs 82 GB of device memory")
    base = lambda seed: torch.randint(-2, 3, (16, 128), generator=gen(seed), device="cuda").float()
    a, w = base(1), base(2)

    def spread(t, rows):
        out = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
        out.view(rows // 16, 16, K // 128, 128).copy_(t.to(E4M3).view(torch.uint8).view(1, 16, 1, 128))
        return out

    a8, w8 = spread(a, T), spread(w, N)
    out = torch.zeros(T, N, dtype=BF16, device="cuda")
    ones = torch.ones(T, 1, device="cuda")
    w_ones = torch.ones(N // 128, K // 128, device="cuda")
    mm.forward(a8, ones, w8, w_ones, out)  # (about 2.8 s)
    assert mm.get_error() == 0
    want = ((a.double() @ w.double().t()) * (K // 128)).to(BF16)
    for rows in out.split(16 * 512):
        assert bool((rows.view(-1, 16, N // 16, 16) == want.view(1, 16, 1, 16)).all())
    del a8, w8, out, rows
    torch.cuda.empty_cache()


# On 152 SMs: tiles of pairs of CTAs, and tiles of one; tiles whole, all cut into as many pieces, or cut by stretches whose borders lie
# inside tiles; and whole rounds of tiles before tiles cut either way.
SHARED_OUT = [
    ("pair, whole", 1500, 2000, 2048), ("pair, whole, odd rows", 1348, 1733, 272), ("pair, two rounds", 1037, 6505, 144),
    ("pair, pieces", 1606, 398, 5728), ("pair, five pieces, odd rows", 1537, 415, 6256), ("pair, one row of tiles", 131, 3359, 6688),
    ("pair, borders inside", 1297, 1762, 3376), ("pair, borders inside, odd rows", 1291, 1677, 3536),
    ("pair, half a tile of tokens, borders inside", 141, 9889, 3232), ("pair, a round and pieces", 2150, 2205, 3104),
    ("pair, a round and borders inside", 2821, 2477, 3744), ("pair, rounds and borders inside", 4096, 14336, 6800),
    ("one, borders inside", 1, 9753, 8416), ("one, a round and borders inside", 1, 29185, 8224), ("one, many tokens, borders inside", 258, 2074, 9760),
    ("one, a round and borders inside, many tokens", 276, 9793, 5520), ("one, a round and pieces", 520, 3865, 3504),
]


@pytest.mark.parametrize("what,T,N,K", SHARED_OUT, ids=[s[0] for s in SHARED_OUT])
@pytest.mark.parametrize("dtype,row_scale", [(BF16, False), (BF16, True), (F16, False)])
def test_matmul8_shared_out(mm, what, T, N, K, dtype, row_scale):
    p = Product(T, N, K, dtype, row_scale=row_scale)
    first = p.forward(mm).clone()
    want, slack = dref.matmul8(p.a8, p.a_scales, p.w8, p.w_scales)
    # values of 65520, the middle of f16's largest and what would follow it, and more are rounded to infinity
    beyond = (want.abs() - slack >= 65520.0) & (dtype == F16)
    inside(first, torch.where(beyond, want.sign() * torch.inf, want), ref.stored(want, dtype, slack))
    assert mm.get_error() == 0
    p.out.zero_()
    assert torch.equal(p.forward(mm), first)


@pytest.mark.parametrize("T,N,K", [(1348, 1733, 272), (1291, 1677, 3536), (2821, 2477, 3744)])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_matmul8_pair_strides(mm, T, N, K, off):
    """Rows of every tensor inside wider buffers, out at odd addresses, by pairs of CTAs; what lies between out's rows stays."""
    p = Product(T, N, K, pad=48, seed=off)
    blocks = -(-K // 128)
    p.a_scales = torch.nn.functional.pad(p.a_scales, (0, 3))[:, :blocks]
    p.w_scales = torch.nn.functional.pad(p.w_scales, (0, 5))[:, :blocks]
    wide = torch.full((T, N + off + 7), 7.0, dtype=BF16, device="cuda")
    p.out = wide[:, off:off + N]
    p.check(mm)
    assert bool((wide[:, :off] == 7).all()) and bool((wide[:, off + N:] == 7).all())


def test_matmul8_pairs_in_graphs_and_beside_each_other(mm):
    """Two products by pairs of CTAs with pieces, on one handle in a graph replayed on other inputs, and on two handles and
    streams at once."""
    p, q = Product(1606, 398, 5728, seed=1), Product(1291, 1677, 3536, seed=2)
    want = [t.forward(mm).clone() for t in (p, q)]
    torch.cuda.synchronize()
    other = rel.Matmul8(device=0)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
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
    p.a_scales.mul_(2.0)
    q.a_scales.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.out, want[0] * 2) and torch.equal(q.out, want[1] * 0.5)
    assert mm.get_error() == 0 and other.get_error() == 0
    other.close()


def test_matmul8_pair_odd_values(mm):
    """NaN and infinite scales and NaN values, by pairs of CTAs with borders inside tiles: their rows and columns, no others."""
    p = Product(1291, 1677, 3536)
    clean = p.forward(mm).clone()
    p.a8.view(torch.uint8)[700, 130] = 0x7F             # e4m3's NaN
    p.a_scales[1, 3] = float("nan")
    p.a_scales[1290, 27] = float("inf")
    p.w8.view(torch.uint8)[1601, 5] = 0xFF
    p.w_scales[2, 4] = float("nan")                     # columns 256..383
    out = p.forward(mm)
    rows, cols = torch.ones(1291, dtype=torch.bool, device="cuda"), torch.ones(1677, dtype=torch.bool, device="cuda")
    rows[[700, 1, 1290]] = False
    cols[256:384] = False
    cols[1601] = False
    assert torch.equal(out[rows][:, cols], clean[rows][:, cols])
    assert bool(out[[1, 700]].isnan().all()) and not bool(out[1290].isfinite().any()) and bool(out[:, ~cols].isnan().all())
    assert mm.get_error() == 0
