"""The operators and the expert layer together (examples/decoder_layer.py): a layer fed whole
prompts, chunks or single tokens over one paged cache gives the same residual stream, the
plain 64-bit layer's, and the experts' outputs of its own norm."""
import math
import os
import sys

import pytest
import torch

import ops_reference as ref
import routed_expert_layer_gb300 as rel
import synth

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

LENGTHS = [150, 40, 1]
STEPS = {"whole": [LENGTHS], "chunks": [[64, 40, 0], [80, 0, 1], [6, 0, 0]],
         "tokens": [[120, 30, 0]] + [[1, 1, 0]] * 10 + [[20, 0, 1]]}


def plain(layer, x, residual):
    """The residual stream after attention of one request's tokens, in 64 bits from the same
    bf16 inputs and weights, without intermediate roundings."""
    f = torch.float64
    h, n, _ = ref.norm(x, layer.norm1, 1e-6, residual)
    qkv = n @ layer.w_qkv.to(f)
    a, b = layer.Hq * layer.D, (layer.Hq + layer.Hkv) * layer.D
    q, k, v = (t.view(len(x), -1, layer.D) for t in (qkv[:, :a], qkv[:, a:b], qkv[:, b:]))
    pos = torch.arange(len(x), device="cuda")
    q, k = (ref.rotate(t, pos, layer.inv_freq, 1.0, False)[0] for t in (q, k))
    G = layer.Hq // layer.Hkv
    s = torch.einsum("nhd,lhd->hnl", q, k.repeat_interleave(G, dim=1)) / math.sqrt(layer.D)
    s = s.masked_fill(~torch.ones(len(x), len(x), dtype=torch.bool, device="cuda").tril(), -math.inf)
    o = torch.einsum("hnl,lhd->nhd", torch.softmax(s, dim=2), v.repeat_interleave(G, dim=1))
    return h + o.reshape(len(x), a) @ layer.w_o.to(f)


def test_decoder_layer_in_steps():
    from decoder_layer import DecoderLayer, run
    H, I, E, k = 512, 256, 64, 8
    moe = rel.MoeLayer(H, I, E, k, max_tokens=512)
    moe.load(synth.layer(H, I, E, seed_weights=1, seed_router=2))
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x, residual = ([torch.randn(n, H, generator=g, device="cuda").bfloat16() for n in LENGTHS] for _ in range(2))
    for name, steps in STEPS.items():
        layer = DecoderLayer(moe, q_heads=8, kv_heads=2, head_dim=64, requests=3, max_len=200, page_size=16)
        out, h, m = run(layer, x, residual, LENGTHS, steps)
        torch.cuda.synchronize()
        assert int(layer.err.item()) == 0 and layer.attention.get_error() == 0 and moe.get_error() == 0
        assert layer.ctx.tolist() == LENGTHS
        used = layer.table[layer.table >= 0].tolist()
        assert len(used) == len(set(used)) == sum(-(-n // 16) for n in LENGTHS) == int(layer.heads[0].item())
        for r in range(3):
            want = plain(layer, x[r], residual[r])
            # Seven roundings to bf16 (n, qkv, rotary, weights, o, o W_o, h), each 2^-9 of its value on average at
            # most and spread over sums of hundreds of terms; the residual stream is about 2: 2^-6 of the
            # larger of the value and 2 holds each alone at its worst, and their sum for independent signs.
            off = (h[r].double() - want).abs() / want.abs().clamp(min=2.0)
            assert float(off.max()) <= 2.0 ** -6, (name, r, float(off.max()))
            t, y, _ = ref.norm(h[r], layer.norm2, 1e-6)  # h was rounded after the norm used it
            assert float(((m[r].double() - y).abs() / y.abs().clamp(min=1.0)).max()) <= 2.0 ** -6, (name, r)
            again = torch.empty_like(out[r])
            moe.forward(m[r].contiguous(), again)
            torch.cuda.synchronize()
            # other batch sizes take other kernels and sum orders; tokens near a routing tie may differ wholly
            rms = float(again.float().pow(2).mean().sqrt())
            far = ((out[r].float() - again.float()).abs().amax(dim=1) > 4e-2 * rms + 2.0 ** -7 * again.float().abs().amax(dim=1))
            assert float(far.float().mean()) <= 0.02, (name, r)
        layer.close()
    moe.close()


def test_example_runs(capsys):
    import decoder_layer
    decoder_layer.main()
    assert "max difference" in capsys.readouterr().out


def test_refused_step_leaves_the_layer_as_it_was():
    """A step past the cache is reported, and the steps after it go on from the lengths and pages before it."""
    from decoder_layer import DecoderLayer
    H, I, E, k = 512, 256, 64, 8
    moe = rel.MoeLayer(H, I, E, k, max_tokens=512)
    moe.load(synth.layer(H, I, E, seed_weights=1, seed_router=2))
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x, residual = ([torch.randn(n, H, generator=g, device="cuda").bfloat16() for n in (25, 15)] for _ in range(2))

    def step(layer, a, b):
        rows = [slice(*a), slice(*b)]
        return layer.step(torch.cat([t[r] for t, r in zip(x, rows)]), torch.cat([t[r] for t, r in zip(residual, rows)]),
                          [a[1] - a[0], b[1] - b[0]])

    results = []
    for refused in (False, True):
        layer = DecoderLayer(moe, q_heads=8, kv_heads=2, head_dim=64, requests=2, max_len=32, page_size=16)
        step(layer, (0, 20), (0, 10))
        if refused:
            kept = layer.table.clone()
            step(layer, (0, 13), (10, 11))  # 33 tokens of 32
            assert int(layer.err.item()) == rel.MOE_OPS_ERR_PLAN
            layer.err.zero_()
            assert layer.ctx.tolist() == [20, 10] and int(layer.heads[0].item()) == 3 and torch.equal(layer.table, kept)
        results.append(step(layer, (20, 25), (10, 15)))
        torch.cuda.synchronize()
        assert layer.ctx.tolist() == [25, 15] and int(layer.err.item()) == 0
        assert layer.attention.get_error() == 0 and moe.get_error() == 0
        layer.close()
    assert all(torch.equal(a, b) for a, b in zip(*results))
    moe.close()


def test_example_agrees_with_itself():
    """The example's residual streams, fed whole and in steps, differ by no more than each may from the
    64-bit layer's: 2^-6 of the larger of the value and 2 (test_decoder_layer_in_steps), so twice that."""
    import decoder_layer
    for whole, steps in decoder_layer.main():
        a, b = whole.double(), steps.double()
        assert whole.shape == steps.shape and bool(a.isfinite().all())
        assert float(((a - b).abs() / a.abs().clamp(min=2.0)).max()) <= 2.0 ** -5 * (1 + 2.0 ** -5)
