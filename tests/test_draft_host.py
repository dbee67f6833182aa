"""Operators for drafted tokens and 8-bit projections, on the host: refusals before any GPU work, binding checks, and
the tests' own references on numbers worked by hand."""
import os
import struct

import pytest
import torch

import draft_reference as dref
import routed_expert_layer_gb300 as rel
from test_ops_host import A, B_, BAD, C, D_, E_, F_, UNSUP, fields, pack

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK = rel.MOE_OK


@pytest.fixture(scope="module")
def L():
    rel.build()
    return rel.lib()


def test_structs_pack_as_expected(tmp_path):
    import subprocess
    names = ["moe_tree_plan_args", "moe_tree_accept_args", "moe_quantize8_args", "moe_matmul8_args"]
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "moe_ops_gb300.h"\nint main(void) {\n' + "".join(
        f'  printf("%zu\\n", sizeof({n}));\n' for n in names) + "  return 0;\n}\n")
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe],
                   check=True)
    for name, size in zip(names, map(int, subprocess.check_output([exe]).split())):
        assert -(-struct.calcsize("@" + fields(name)[1]) // 8) * 8 == size, name


def tree_plan_args(**kw):
    return pack("moe_tree_plan_args", **{**dict(parents=A, q_start=B_, ctx_lens=C, positions=D_, mask=E_, N=10, B=3, words=2), **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(parents=0), BAD), (dict(q_start=0), BAD), (dict(ctx_lens=0), BAD), (dict(positions=0), BAD), (dict(mask=0), BAD),
    (dict(parents=A + 2), BAD), (dict(err=F_ + 1), BAD), (dict(N=-1), BAD), (dict(B=-1), BAD), (dict(words=0), BAD), (dict(words=9), UNSUP),
    (dict(positions=A), BAD), (dict(positions=A + 36), BAD), (dict(mask=D_ + 36), BAD), (dict(mask=B_ - 4), BAD), (dict(err=C + 8), BAD),
    (dict(N=0, parents=0, mask=0), OK), (dict(B=0, q_start=0), OK),
])
def test_tree_plan_refusals(L, kw, status):
    assert L.moe_tree_plan(None, tree_plan_args(**kw)) == status
    assert L.moe_tree_plan(None, None) == BAD


def accept_args(**kw):
    base = dict(parents=A, tokens=A + 64, targets=A + 128, q_start=A + 192, ctx_lens=A + 256, block_table=A + 512, k_cache=B_, v_cache=C,
                path=D_, accepted=D_ + 512, ctx_out=D_ + 1024, next_tokens=D_ + 2048, table_stride=8, kc_layer=4096, kc_page=1024,
                kc_row=64, kc_head=64, vc_layer=4096, vc_page=1024, vc_row=64, vc_head=64, N=10, B=3, W=8, depth=4, layers=2, Hkv=1,
                D=64, page_size=16, num_pages=4)
    return pack("moe_tree_accept_args", **{**base, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(parents=0), BAD), (dict(targets=A + 129), BAD), (dict(q_start=0), BAD), (dict(block_table=0), BAD), (dict(path=0), BAD),
    (dict(next_tokens=0), BAD), (dict(k_cache=0), BAD), (dict(v_cache=C + 1), BAD), (dict(certain=F_ + 2), BAD), (dict(N=-1), BAD),
    (dict(depth=0), BAD), (dict(layers=0), BAD), (dict(Hkv=0), BAD), (dict(D=0), BAD), (dict(page_size=24), BAD), (dict(num_pages=0), BAD),
    (dict(table_stride=7), BAD), (dict(kc_page=-8), BAD), (dict(W=0), BAD), (dict(depth=257), UNSUP), (dict(B=65536), UNSUP),
    (dict(W=1 << 27, table_stride=1 << 27), UNSUP), (dict(ctx_out=A + 256), BAD), (dict(accepted=D_ + 1024), BAD), (dict(path=A + 128), BAD),
    (dict(next_tokens=A + 512 + 4 * (2 * 8 + 7)), BAD), (dict(certain=D_ + 512), BAD), (dict(err=D_ + 44), BAD), (dict(B=0, q_start=0), OK),
])
def test_tree_accept_refusals(L, kw, status):
    assert L.moe_tree_accept(None, accept_args(**kw)) == status
    assert L.moe_tree_accept(None, None) == BAD


def quantize_args(**kw):
    return pack("moe_quantize8_args", **{**dict(x=A, out8=B_, scales=C, x_stride=256, out8_stride=256, T=4, H=256, group=128, rows=1), **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), BAD), (dict(out8=0), BAD), (dict(scales=0), BAD), (dict(x=A + 1), BAD), (dict(scales=C + 2), BAD), (dict(T=-1), BAD),
    (dict(H=0), BAD), (dict(dtype=2), BAD), (dict(group=64), BAD), (dict(rows=2), BAD), (dict(group=0, rows=128), BAD),
    (dict(x_stride=255), BAD), (dict(out8_stride=255), BAD), (dict(out8=A + 100), BAD), (dict(scales=A + 2044), BAD), (dict(out8=C - 1000), BAD),
    (dict(T=0, x=0), OK), (dict(H=(1 << 30) + 1, x_stride=1 << 31, out8_stride=1 << 31), UNSUP),
])
def test_quantize_refusals(L, kw, status):
    assert L.moe_quantize8(None, quantize_args(**kw)) == status
    assert L.moe_quantize8(None, None) == BAD


def test_matmul8_handle_refusals(L):
    assert L.moe_matmul8_create(0, None) == BAD
    assert L.moe_matmul8_forward(None, None, None) == BAD
    assert L.moe_matmul8_get_error(None, None) == BAD
    assert L.moe_matmul8_destroy(None) == OK
    assert L.moe_matmul8_device_bytes(None) == 0
    assert L.moe_attn_forward_tree(None, None, None, None, 1) == BAD


def test_bindings_refuse_host_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    m = torch.zeros(4, 1, dtype=torch.int32)
    c = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rel.tree_plan(i, i, i[:3], positions=i, mask=m)
    with pytest.raises(ValueError, match="CUDA"):
        rel.tree_accept(i, i, i, i, i[:3], m, c, c, path=m[:3], accepted=i, ctx_out=i, next_tokens=i)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rel.quantize8(x, torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 1))
    with pytest.raises(TypeError, match="tensor"):
        rel.quantize8([1.0], x, x)


def test_references_by_hand():
    """A tree of 6 nodes: 0 has children 1, 2, 3; 1 has 4; 4 has 5."""
    parents = [-1, 0, 0, 0, 1, 4]
    bits, depth = dref.ancestors(parents)
    assert bits == [1, 3, 5, 9, 19, 51] and depth == [0, 1, 1, 1, 2, 3]
    assert dref.words_of(0x1_80000001, 2) == [-0x7FFFFFFF, 1]
    tokens = [7, 3, 5, 3, 8, 9]
    assert dref.accept(parents, tokens, [3, 8, 0, 0, 2, 4], 1, 5) == ([1, 4], 3, 2)   # of 1 and 3 the lower
    assert dref.accept(parents, tokens, [3, 8, 0, 0, 9, 4], 1, 5) == ([1, 4, 5], 4, 4)
    assert dref.accept(parents, tokens, [3, 8, 0, 0, 9, 4], 1, 2) == ([1, 4], 3, 9)
    assert dref.accept(parents, tokens, [6, 8, 0, 0, 9, 4], 1, 5) == ([], 1, 6)
    assert dref.accept(parents, tokens, [6, 8, 0, 0, 9, 4], 2, 5) == ([4, 5], 4, 4)
    assert dref.accept([], [], [], 1, 5) == ([], 0, -1)
    seen = dref.by_bits([bits], 1)
    assert seen(0, 4, 6, 2, 8).tolist() == [True, True, True, True, False, False, True, False]
    assert seen(0, 1, 33, 2, 35).tolist() == [True] * 4 + [False] * 31
    y, s = dref.quantize(torch.tensor([[1.0, -896.0, 0.0]]), 0, 1)
    assert s.tolist() == [[2.0]] and y.tolist() == [[0.5, -448.0, 0.0]]
    a8 = torch.tensor([[1.0, 2.0] + [0.0] * 126 + [4.0] + [0.0] * 15]).to(torch.float8_e4m3fn)
    w8 = torch.tensor([[3.0, 0.5] + [0.0] * 126 + [0.25] + [0.0] * 15]).to(torch.float8_e4m3fn)
    out, _ = dref.matmul8(a8, torch.tensor([[2.0, 10.0]]), w8, torch.tensor([[0.5, 3.0]]))
    assert out.tolist() == [[2.0 * 0.5 * 4.0 + 10.0 * 3.0 * 1.0]]
