"""The product of e4m3 activations and weights on the host: what the library refuses before any GPU work. Without a handle a call
whose arguments are right is refused too (MOE_ERR_INVALID_ARG), after its sizes have been looked at."""
import pytest

import routed_expert_layer_gb300 as rel
from test_ops_host import A, B_, BAD, C, D_, E_, UNSUP, pack


@pytest.fixture(scope="module")
def L():
    rel.build()
    return rel.lib()


def forward(L, **kw):
    base = dict(a8=A, a_scales=B_, w8=C, w_scales=D_, out=E_, T=4, N=128, K=128, a_blocks=1, a8_stride=128, w8_stride=128,
                a_scales_stride=1, w_scales_stride=1, out_stride=128)
    return L.moe_matmul8_forward(None, None, pack("moe_matmul8_args", **{**base, **kw}))


BIG = 1 << 20


@pytest.mark.parametrize("T,N,K,status", [
    (BIG << 10, 128, 16, BAD), ((BIG << 10) + 1, 128, 16, UNSUP), (128, BIG << 10, 16, BAD), (128, (BIG << 10) + 1, 16, UNSUP),
    (128, 128, BIG, BAD), (128, 128, BIG + 16, UNSUP), (BIG, 1 << 16, 1 << 16, BAD), (BIG, BIG, BIG, BAD),
    (1 << 22, 1 << 22, 16, BAD), ((1 << 22) + 1, 1 << 22, 16, UNSUP), (1 << 22, (1 << 22) + 1, BIG, UNSUP), (1 << 30, 1 << 30, 128, UNSUP),
])
def test_matmul8_sizes(L, T, N, K, status):
    """The limits that the header names, and no other: products of sizes have none but the number of tiles."""
    blocks = -(-K // 128)
    far = 1 << 61  # each tensor in a range of its own
    got = forward(L, T=T, N=N, K=K, a_blocks=blocks, a8=far, w8=2 * far, a_scales=3 * far, w_scales=3 * far + (1 << 58),
                  out=3 * far + (1 << 59), a8_stride=K, w8_stride=K, a_scales_stride=blocks, w_scales_stride=blocks, out_stride=N)
    assert got == status
