"""8-bit projections on the GPU at the edges of the values' and the calls' range (test_gpu_matmul8.py has the others)."""
import pytest
import torch

from test_gpu_matmul8 import BF16, E4M3, F16, gen, run_quantize

pytestmark = pytest.mark.gpu


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
