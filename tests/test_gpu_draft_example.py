"""What examples/draft_step.py shows, beyond that it runs: with drafts it takes fewer steps, and every token that it decodes is one
that the model gives after those before it."""
import os
import sys

import pytest
import torch

import routed_expert_layer_gb300 as rel
import synth

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_decodes_what_the_model_gives():
    """The sequences of both runs are fed once more, whole, and every token that a run decoded is looked up among the scores behind the one
    before it. The same kernels ran over other batches, so the layer's output y may be off: by 2^-5 of it (2 at least) for
    the residual, as test_gpu_draft_step.py derives, and as much for the experts' output beside it. A score is a
    sum of y times an embedding, so two of them may change places where they are less apart than the sums of those errors' sizes."""
    import draft_step
    plain, drafted, plain_steps, steps = draft_step.main()
    assert steps < plain_steps == 24
    H = 512
    moe = rel.MoeLayer(H, 256, 64, 8, max_tokens=1024)
    moe.load(synth.layer(H, 256, 64, seed_weights=1, seed_router=2))
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    embed = torch.randn(300, H, generator=g, device="cuda").bfloat16()
    lengths = [50, 7, 1]  # of the prompts
    for sequences in (plain, drafted):
        layer = draft_step.DraftLayer(moe, q_heads=8, kv_heads=2, head_dim=64, requests=3, max_len=160)
        tokens = torch.tensor([t for s in sequences for t in s], device="cuda")
        x = embed[tokens]
        out, h, _ = layer.step(x, torch.zeros_like(x), [list(range(-1, len(s) - 1)) for s in sequences])
        y = (out + h).double()
        e = embed.double()
        scores = y @ e.t()
        off = (2.0 ** -4 * y.abs().clamp(min=2.0)) @ e.abs().t()
        at, close = 0, []
        for s, n in zip(sequences, lengths):
            assert s[:n] == plain[lengths.index(n)][:n] and len(s) == n + 24
            for i in range(n, len(s)):
                row, most = scores[at + i - 1], off[at + i - 1]
                top = int(row.argmax())
                assert float(row[top] - row[s[i]]) <= float(most[top] + most[s[i]]), (n, i)
                close.append(int((row[top] - row <= most[top] + most).sum()))
            at += len(s)
        assert sum(close) / len(close) < 30  # of 300: the bound tells a right token from a wrong one
        assert int(layer.err.item()) == 0 and layer.attention.get_error() == 0 and layer.matmul.get_error() == 0
        layer.close()
    moe.close()
