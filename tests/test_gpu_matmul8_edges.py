"""8-bit projections on the GPU at the edges of the values' and the calls' range (test_gpu_matmul8.py has the others)."""
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
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    mm.forward(a8, ones, w8, w_ones, out)
    end.record()
    assert mm.get_error() == 0
    assert start.elapsed_time(end) > 2000.0  # (about 2,800 ms)
    want = ((a.double() @ w.double().t()) * (K // 128)).to(BF16)
    for rows in out.split(16 * 512):
        assert bool((rows.view(-1, 16, N // 16, 16) == want.view(1, 16, 1, 16)).all())
    del a8, w8, out, rows
    torch.cuda.empty_cache()
