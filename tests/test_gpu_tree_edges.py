"""Attention by masks at the edges of its calls (test_gpu_tree.py has the others)."""
import pytest
import torch

import routed_expert_layer_gb300 as rel
from test_gpu_tree import F32, I32, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = rel.PagedAttention(device=0)
    yield h
    h.close()


def test_tree_attention_mask_in_outputs(handle):
    """A mask that shares memory with out or lse would change under the call: refused, as the plan and the acceptance refuse the like. One
    that lies between the heads of out's rows shares nothing."""
    c = Case([40, 9], [20, 7], 8, 2, 64, 16, 1, seed=2)
    want, mask, N = c.check(handle), c.mask.clone(), 27
    out, lse = torch.empty_like(c.q), torch.empty(N, 8, dtype=F32, device="cuda")
    wide = torch.zeros(N, 8, 192, dtype=c.q.dtype, device="cuda")  # heads of 128 bytes, 256 between them
    ints = lambda t: t.view(-1).view(I32)

    def at(t, word):
        piece = ints(t)[word:word + N].view(N, 1)
        piece.copy_(mask)
        return piece

    call = lambda m, o, l=None: handle.forward(c.q, c.k, c.v, c.table, c.q_start, c.kv, o, scale=c.scale, lse=l, tree=m)
    last = ints(out).numel() - N
    head = 96  # words of a head of `wide` and what follows it
    for m, o, l in ((at(out, 0), out, None), (at(out, last), out, None), (at(out, 500), out, lse), (at(lse, 0), out, lse),
                    (at(lse, 8 * N - N), out, lse), (at(wide, 10 * head + 31), wide[:, :, :64], None),
                    (at(wide, 11 * head - N + 1), wide[:, :, :64], None), (at(wide, 215 * head), wide[:, :, :64], None)):
        with pytest.raises(rel.MoeError):
            call(m, o, l)
    for word in (10 * head + 32, 11 * head - N, 215 * head + 32):
        wide.zero_()
        m = at(wide, word)
        call(m, wide[:, :, :64])
        assert torch.equal(wide[:, :, :64], want) and torch.equal(m, mask)
    both = torch.empty(2 * N, dtype=I32, device="cuda")
    call(at(both, N), out)
    assert torch.equal(out, want) and handle.get_error() == 0


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,words", [
    ([700, 3], [33, 90], 24, 2, 128, 1), ([64, 1000, 0], [130, 65, 100], 8, 1, 64, 2), ([40, 500], [40, 60], 2, 2, 64, 1),
    ([300, 9], [300, 20], 12, 1, 128, 8),
])
def test_tree_attention_chunks_longer_than_the_mask(handle, ctx, new, Hq, Hkv, D, words):
    """Requests of more new tokens than the mask has bits see what is before them, beside trees or alone; max_new picks the same
    variant as the number of all tokens here, so it changes no bit."""
    c = Case(ctx, new, Hq, Hkv, D, 16, words, masks="tree", seed=sum(new))
    assert max(new) > 32 * words
    a = c.check(handle)
    assert torch.equal(a, c.check(handle, max_new=max(new)))
    if min(new) > 32 * words:  # no request with a tree: what the call without masks computes
        assert torch.equal(a, c.check(handle, mask=False))
