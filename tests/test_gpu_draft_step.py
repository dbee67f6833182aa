"""The operators for drafted tokens and 8-bit projections together with the others and the expert layer
(examples/draft_step.py): a tree of drafts, the path accepted and the steps behind it give what the same tokens fed one by
one give."""
import os
import sys

import pytest
import torch

import routed_expert_layer_gb300 as rel
import synth

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

H = 512


@pytest.fixture(scope="module")
def moe():
    layer = rel.MoeLayer(H, 256, 64, 8, max_tokens=512)
    layer.load(synth.layer(H, 256, 64, seed_weights=1, seed_router=2))
    yield layer
    layer.close()


def chain(n):
    return list(range(-1, n - 1))


def close_enough(got, want):
    """Both ran the same kernels over other batches: fp32 sums in another order, so a value beside the middle of two bf16
    numbers (2^-8 of itself apart) may go to the other one, and then one of e4m3's (2^-3 apart at most) in about one of 2^4
    cases. A projection of 512 terms of about 0.8 * 0.04 each is then off by sqrt(512 / 16) * 2^-3 * 0.03 = 0.02, and
    three projections and the residual's own rounding (2^-8 of 2) stay below 2^-4 for values of about 2."""
    off = (got.double() - want.double()).abs() / want.double().abs().clamp(min=2.0)
    assert float(off.max()) <= 2.0 ** -5, float(off.max())


def test_tree_step_equals_single_tokens(moe):
    """Request 0: 37 known tokens, then a tree of 12 whose nodes 2, 5, 9 are the right ones; request 1: 5 known tokens,
    a tree of which nothing is right; request 2: a chunk of 40 (longer than the mask) while the others decode; then one
    more token each."""
    from draft_step import DraftLayer
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    rand = lambda n: torch.randn(n, H, generator=g, device="cuda").bfloat16()
    prompt, true0, last = [rand(37), rand(5)], rand(4), rand(3)
    tree = [-1, 0, 0, 0, 1, 2, 2, 3, 5, 5, 9, 7]
    make = lambda: DraftLayer(moe, q_heads=8, kv_heads=2, head_dim=64, requests=3, max_len=96)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    zero = torch.zeros_like

    def feed(layer, rows, parents, tokens=None, targets=None, certain=None):
        x = torch.cat(rows)
        n = x.shape[0]
        parts = layer.step(x, zero(x), parents)
        certain = i32([len(p) for p in parents]) if certain is None else i32(certain)
        got = layer.accept(i32(tokens or [0] * n), i32(targets or [1] * n), certain, depth=6)
        return parts, got

    # with a tree
    a = make()
    none = rand(0)
    feed(a, [*prompt], [chain(37), chain(5), []])
    other = rand(12)
    rows0 = other.clone()
    for node, row in zip((0, 2, 5, 9), true0):
        rows0[node] = row
    chunk = rand(40)
    tokens = [100 + j for j in range(12)] + [50, 51, 52] + [7] * 40
    targets = [1] * len(tokens)
    targets[0], targets[2], targets[5], targets[9] = 102, 105, 109, 55  # node 10 is not 55
    rows1 = rand(3)
    (_, h, _), (path, following) = feed(a, [rows0, rows1, chunk], [tree, [-1, 0, 0], chain(40)], tokens, targets, [1, 1, 40])
    assert path.tolist() == [[2, 5, 9, -1, -1, -1], [-1] * 6, [-1] * 6]
    assert following.tolist() == [55, 1, 1] and a.ctx.tolist() == [41, 6, 40]
    used = a.table[a.table >= 0].tolist()
    assert len(used) == len(set(used)) == 3 + 1 + 3 and int(a.heads[0].item()) == 7
    rest = a.free[7:].tolist()
    assert sorted(rest + used) == list(range(a.k_cache.shape[0]))  # no page is lost or twice there
    (_, end, _), _ = feed(a, [last], [[-1]] * 3)
    torch.cuda.synchronize()
    # one by one
    b = make()
    feed(b, [*prompt], [chain(37), chain(5), []])
    singles = []
    for i in range(4):
        rows = [true0[i:i + 1], rows1[:1] if i == 0 else none, chunk if i == 0 else none]
        (_, hb, _), _ = feed(b, rows, [[-1], [-1] if i == 0 else [], chain(40) if i == 0 else []])
        singles.append(hb[0])
        if i == 0:
            first_b = hb
    assert b.ctx.tolist() == [41, 6, 40]
    (_, end_b, _), _ = feed(b, [last], [[-1]] * 3)
    torch.cuda.synchronize()
    close_enough(h[[0, 2, 5, 9]], torch.stack(singles))
    close_enough(h[12], first_b[1])
    close_enough(h[15:], first_b[2:])
    close_enough(end, end_b)
    for layer in (a, b):
        assert int(layer.err.item()) == 0 and layer.attention.get_error() == 0 and layer.matmul.get_error() == 0
        layer.close()
    assert moe.get_error() == 0


def test_example_runs(capsys):
    import draft_step
    plain, drafted, plain_steps, steps = draft_step.main()
    assert "steps token by token" in capsys.readouterr().out
    assert [len(s) for s in plain] == [len(s) for s in drafted] == [74, 31, 25]
    assert steps <= plain_steps == 24
