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
