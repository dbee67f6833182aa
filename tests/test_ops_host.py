"""The operators beside the expert layer, on the host: struct layouts, refusals before any
GPU work, binding checks, and the frequency helper."""
import ctypes
import math
import os
import re
import struct
import subprocess

import pytest
import torch

import routed_expert_layer_gb300 as rel

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNSUP = rel.MOE_ERR_INVALID_ARG, rel.MOE_ERR_UNSUPPORTED
A, B_, C, D_, E_, F_ = 0x10000, 0x2000000, 0x4000000, 0x6000000, 0x8000000, 0xA000000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    rel.build()
    return rel.lib()


def fields(struct_name):
    """Field names of a struct of the header, in order, with their struct format letters."""
    text = open(os.path.join(ROOT, "include", "moe_ops_gb300.h")).read()
    body = re.search(r"typedef struct \{([^}]*)\} " + struct_name + ";", text).group(1)
    names, fmt = [], ""
    for line in body.split(";"):
        line = line.strip()
        if not line:
            continue
        pointer = "*" in line
        kind = line.replace("const", "").split()[0]
        for n in re.sub(r"^(const\s+)?\w+\s*\**", "", line).split(","):
            names.append(n.strip().lstrip("*"))
            fmt += "P" if pointer else {"int64_t": "q", "int32_t": "i", "float": "f"}[kind]
    return names, fmt


def pack(struct_name, **kw):
    names, fmt = fields(struct_name)
    assert set(kw) <= set(names)
    return struct.pack("@" + fmt, *[kw.get(n, 0) for n in names])


STRUCTS = ["moe_rmsnorm_args", "moe_paged_plan_args", "moe_rotary_args", "moe_attn_args"]


def test_header_is_plain_c_and_packs_as_expected(tmp_path):
    """The header compiles as C99 without warnings, and the structs these tests pack by hand
    have C's sizes."""
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "moe_ops_gb300.h"\nint main(void) {\n' + "".join(
        f'  printf("%zu\\n", sizeof({n}));\n' for n in STRUCTS) + "  return 0;\n}\n")
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", exe], check=True)
    sizes = [int(v) for v in subprocess.check_output([exe]).split()]
    for name, size in zip(STRUCTS, sizes):
        assert -(-struct.calcsize("@" + fields(name)[1]) // 8) * 8 == size, name


def norm_args(**kw):
    base = dict(x=A, weight=B_, out=C, x_stride=256, out_stride=256, T=2, H=256, eps=1e-6)
    base.update(kw)
    return pack("moe_rmsnorm_args", **base)


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), BAD), (dict(weight=0), BAD), (dict(out=0), BAD), (dict(T=-1), BAD), (dict(H=0), BAD),
    (dict(dtype=2), BAD), (dict(group=64), BAD), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD),
    (dict(x=A + 1), BAD), (dict(x_stride=255), BAD), (dict(out_stride=100), BAD),
    (dict(out8=D_, out8_stride=256), BAD),                          # 8-bit output without scales
    (dict(scales=D_), BAD),                                         # scales without 8-bit output
    (dict(residual_out=D_, residual_out_stride=256), BAD),          # nothing was added
    (dict(residual=D_, residual_stride=8), BAD),
    (dict(H=32769, x_stride=40000, out_stride=40000), UNSUP),
    (dict(T=0, x=0, out=0), rel.MOE_OK),
])
def test_norm_refusals(L, kw, status):
    assert L.moe_add_rmsnorm(None, norm_args(**kw)) == status
    assert L.moe_add_rmsnorm(None, None) == BAD


def plan_args(**kw):
    base = dict(ctx_lens=A, new_lens=A, block_table=B_, free_pages=C, free_head=D_, q_start=E_, kv_lens=E_,
                positions=F_, slots=F_, free_head_out=D_ + 64, table_stride=8, B=4, W=8, F=10, N=4, page_size=16)
    base.update(kw)
    return pack("moe_paged_plan_args", **base)


@pytest.mark.parametrize("kw,status", [
    (dict(ctx_lens=0), BAD), (dict(block_table=0), BAD), (dict(free_head_out=D_), BAD), (dict(q_start=0), BAD),
    (dict(positions=0), BAD), (dict(slots=F_ + 2), BAD), (dict(B=0), BAD), (dict(W=0), BAD), (dict(N=-1), BAD),
    (dict(F=-1), BAD), (dict(table_stride=7), BAD), (dict(page_size=24), BAD), (dict(page_size=0), BAD),
    (dict(B=4097), UNSUP), (dict(W=1 << 27, table_stride=1 << 27), UNSUP),
])
def test_plan_refusals(L, kw, status):
    assert L.moe_paged_plan(None, plan_args(**kw)) == status
    assert L.moe_paged_plan(None, None) == BAD


def plan_memory():
    """Addresses, sizes in words and lengths of a plan call whose tensors lie one behind the other."""
    B, W, F, N = 4, 8, 10, 6
    words = dict(ctx_lens=B, new_lens=B, block_table=(B - 1) * 9 + W, free_pages=F, free_head=1, q_start=B + 1, kv_lens=B,
                 positions=N, slots=N, free_head_out=1, err=1)
    at, base = {}, 1 << 20
    for name, n in words.items():
        at[name] = base
        base += 4 * n
    return at, words, dict(table_stride=9, B=B, W=W, F=F, N=N, page_size=16)


OUTPUTS = ["block_table", "q_start", "kv_lens", "positions", "slots", "free_head_out", "err"]


@pytest.mark.parametrize("out", OUTPUTS)
def test_plan_refuses_outputs_that_are_inputs_or_each_other(L, out):
    """No output may share a word with an input (other blocks still read it) or with another output:
    refused at the tensor's first word and at its last."""
    at, words, sizes = plan_memory()
    for other in words:
        if other == out:
            continue
        for place in (at[other], at[other] + 4 * (words[other] - 1), at[other] - 4 * (words[out] - 1)):
            moved = dict(at, **{out: place})
            assert L.moe_paged_plan(None, pack("moe_paged_plan_args", **moved, **sizes)) == BAD, (out, other)


def rotary_args(**kw):
    base = dict(q=A, k=B_, v=C, q_out=A, k_cache=D_, v_cache=E_, positions=F_, slots=F_, inv_freq=F_, q_tok=512,
                q_head=128, k_tok=128, k_head=128, v_tok=128, v_head=128, qo_tok=512, qo_head=128, kc_page=2048,
                kc_row=128, kc_head=128, vc_page=2048, vc_row=128, vc_head=128, N=3, Hq=4, Hkv=1, D=128, rot=128,
                page_size=16, num_pages=4, mscale=1.0)
    base.update(kw)
    return pack("moe_rotary_args", **base)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), BAD), (dict(k_cache=0), BAD), (dict(inv_freq=F_ + 4), BAD), (dict(positions=0), BAD),
    (dict(rot=130), BAD), (dict(rot=63), BAD), (dict(rot=0), BAD), (dict(D=127, rot=64), BAD), (dict(Hkv=0), BAD),
    (dict(N=-1), BAD), (dict(page_size=17), BAD), (dict(num_pages=0), BAD), (dict(q_tok=-8), BAD), (dict(dtype=5), BAD),
    (dict(D=1026, rot=2), UNSUP), (dict(num_pages=1 << 27), UNSUP), (dict(N=0, q=0), rel.MOE_OK),
])
def test_rotary_refusals(L, kw, status):
    assert L.moe_rotary_append(None, rotary_args(**kw)) == status
    assert L.moe_rotary_append(None, None) == BAD


def test_attention_handle_refusals(L):
    assert L.moe_attn_create(0, None) == BAD
    assert L.moe_attn_forward(None, None, None) == BAD
    assert L.moe_attn_get_error(None, None) == BAD
    assert L.moe_attn_destroy(None) == rel.MOE_OK
    assert L.moe_attn_device_bytes(None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rel.add_rmsnorm(x, x[0], 1e-6, out=x)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        rel.paged_plan(i, i, torch.zeros(4, 2, dtype=torch.int32), i, i[:1], 16, q_start=i, kv_lens=i, positions=i,
                       slots=i, free_head_out=i[:1])
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rel.rotary_append(q, q, q, i, i, torch.zeros(32, dtype=torch.float64), c, c)


def test_binding_refuses_other_objects():
    from routed_expert_layer_gb300 import ops
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="tensor"):
        rel.add_rmsnorm([1.0], t[0], 1e-6, out=t)
    with pytest.raises(TypeError):
        ops._norm(t)


def test_rope_frequencies():
    f = rel.rope_frequencies(64, base=500.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,)
    for i in range(32):
        assert math.isclose(float(f[i]), 500.0 ** (-2 * i / 64), rel_tol=1e-14)
    assert torch.allclose(rel.rope_frequencies(64, base=500.0, linear=4.0, device="cpu"), f / 4, rtol=1e-15, atol=0)
    g = rel.rope_frequencies(64, base=500.0, blend=(8.0, 2048.0, 1.0, 32.0), device="cpu")
    turns = 2048.0 * f / (2 * math.pi)
    for i in range(32):
        keep = min(1.0, max(0.0, (float(turns[i]) - 1.0) / 31.0))
        assert math.isclose(float(g[i]), float(f[i]) * (keep + (1 - keep) / 8.0), rel_tol=1e-14)
    for bad in (0, 3, -2):
        with pytest.raises(ValueError):
            rel.rope_frequencies(bad, device="cpu")


@pytest.mark.parametrize("kw", [dict(base=0.0), dict(base=-2.0), dict(linear=0.0), dict(linear=math.nan),
                                dict(blend=(8.0, 2048.0, 32.0, 1.0)), dict(blend=(8.0, 2048.0, 1.0, 1.0)),
                                dict(blend=(0.0, 2048.0, 1.0, 32.0)), dict(blend=(8.0, -1.0, 1.0, 32.0))])
def test_rope_frequencies_refusals(kw):
    """Turns given fast before slow would keep the slow pairs and slow the fast ones."""
    with pytest.raises(ValueError):
        rel.rope_frequencies(64, device="cpu", **kw)


def test_package_knows_its_operators():
    with pytest.raises(AttributeError):
        rel.no_such_operator
    for name in rel._OPS:
        assert callable(getattr(rel, name))


def test_plan_reference_by_hand():
    """The tests' own plan reference on numbers worked by hand: P = 4, request 0 has 5 cached
    tokens (pages 7, 9) and brings 4 (one new page), request 1 starts empty with 3."""
    from ops_reference import plan
    got = plan([5, 0], [4, 3], [[7, 9, -1], [-1, -1, -1]], [20, 21, 22], 1, 4, 8)
    assert got["block_table"] == [[7, 9, 21], [22, -1, -1]]
    assert got["positions"] == [5, 6, 7, 8, 0, 1, 2, 0]
    assert got["slots"] == [37, 38, 39, 84, 88, 89, 90, -1]
    assert got["q_start"] == [0, 4, 7] and got["kv_lens"] == [9, 3] and got["free_head_out"] == [3]
    assert plan([5, 0], [4, 3], [[7, 9, -1], [-1, -1, -1]], [20, 21], 1, 4, 8) is None
