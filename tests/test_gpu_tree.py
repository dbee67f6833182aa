"""Trees of drafted tokens on the GPU: plan, attention by masks, acceptance, against plain forms
(draft_reference.py, where every tolerance is derived)."""
import math
import random

import pytest
import torch

import draft_reference as dref
import ops_reference as ref
import routed_expert_layer_gb300 as rel
from test_gpu_ops import inside

pytestmark = pytest.mark.gpu
BF16, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


def ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def flat(lists):
    return [v for row in lists for v in row]


def starts_of(lists):
    at = [0]
    for row in lists:
        at.append(at[-1] + len(row))
    return at


# ---- plan --------------------------------------------------------------------------------------


def run_plan(parents, ctx, words, extra=0, err=True):
    N = sum(map(len, parents)) + extra
    pos = torch.full((N,), -7, dtype=I32, device="cuda")
    mask = torch.full((N, words), 0x5A5A5A5A, dtype=I32, device="cuda")
    e = torch.zeros(1, dtype=I32, device="cuda")
    rel.tree_plan(ints(flat(parents) + [0] * extra), ints(starts_of(parents)), ints(ctx), positions=pos, mask=mask,
                  err=e if err else None)
    return pos.tolist(), mask.tolist(), int(e.item())


def want_plan(parents, ctx, words, extra=0):
    pos, mask = [], []
    for p, c in zip(parents, ctx):
        if len(p) > 32 * words:
            pos += [c + t for t in range(len(p))]
            mask += [[0x5A5A5A5A] * words] * len(p)
            continue
        bits, depth = dref.ancestors(p)
        pos += [c + d for d in depth]
        mask += [dref.words_of(m, words) for m in bits]
    return pos + [-7] * extra, mask + [[0x5A5A5A5A] * words] * extra


@pytest.mark.parametrize("words", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("B", [1, 5, 70])
def test_tree_plan(words, B):
    """Sizes from none to the mask's full width, chains, stars and trees, and chunks longer than the mask."""
    r = random.Random(words * 1000 + B)
    parents = []
    for b in range(B):
        n = r.choice([0, 1, 2, 31, 32, 33, 32 * words, 32 * words - 1, r.randint(1, 32 * words)])
        n = min(n, 32 * words)
        kind = r.randrange(5)
        if kind == 0:
            parents.append(list(range(-1, n - 1)))
        elif kind == 1:
            parents.append([-1] + [0] * (n - 1) if n else [])
        elif kind == 2:
            parents.append(list(range(-1, 32 * words + r.randint(0, 90))))  # a chunk
        elif kind == 3:
            parents.append([-1 if j == 0 else r.randrange(-1, j) for j in range(n)])  # a forest in any order
        else:
            parents.append(dref.random_tree(r, n) if n else [])
    ctx = [r.choice([0, 1, 5000, 1 << 29]) for _ in range(B)]
    pos, mask, err = run_plan(parents, ctx, words, extra=3)
    assert err == 0
    want = want_plan(parents, ctx, words, extra=3)
    assert pos == want[0]
    assert mask == want[1]


@pytest.mark.parametrize("words", [1, 3, 8])
def test_tree_plan_long_chunks(words):
    """Prompts of thousands of tokens beside trees; one that is no chain in its last token."""
    r = random.Random(words)
    parents = [dref.random_tree(r, 20), list(range(-1, 4999)), dref.random_tree(r, 31), [], list(range(-1, 700)), [-1]]
    ctx = [3, 70000, 0, 5, 12, 1]
    pos, mask, err = run_plan(parents, ctx, words, extra=2)
    assert err == 0 and (pos, mask) == want_plan(parents, ctx, words, extra=2)
    parents[1][-1] = 7
    pos, mask, err = run_plan(parents, ctx, words)
    assert err == rel.MOE_OPS_ERR_PLAN and (pos, mask) == want_plan(parents, ctx, words)


def test_tree_plan_bad_input():
    """A parent that is not before its node counts as -1, a long request that is no chain as a chain, a negative
    context as 0; a request outside the rows is skipped. Each raises its bit, and the others are as ever."""
    good = [-1, 0, 0, 1]
    pos, mask, err = run_plan([good, [-1, 1, 0, 9], good], [5, 5, 5], 1)
    want = want_plan([good, [-1, -1, 0, -1], good], [5, 5, 5], 1)
    assert (pos, mask) == want and err == rel.MOE_OPS_ERR_PLAN
    pos, mask, err = run_plan([[-5, 0], good], [0, -3], 1)
    assert (pos, mask) == want_plan([[-1, 0], good], [0, 0], 1) and err == rel.MOE_OPS_ERR_PLAN
    chunk = list(range(-1, 39))
    assert run_plan([chunk, good], [7, 7], 1)[2] == 0
    pos, mask, err = run_plan([chunk[:20] + [3] + chunk[21:], good], [7, 7], 1)
    assert (pos, mask) == want_plan([chunk, good], [7, 7], 1) and err == rel.MOE_OPS_ERR_PLAN
    assert run_plan([[-1, 7]], [1], 1, err=False)[0] == [1, 1]  # no error word
    for starts in ([0, 4, 9], [-1, 4, 8], [0, 4, 2], [0, 4, 1 << 30]):
        pos = torch.full((8,), -7, dtype=I32, device="cuda")
        m = torch.full((8, 1), -7, dtype=I32, device="cuda")
        e = torch.zeros(1, dtype=I32, device="cuda")
        rel.tree_plan(ints(good + good), ints(starts), ints([3, 3]), positions=pos, mask=m, err=e)
        assert int(e.item()) == rel.MOE_OPS_ERR_INDEX
        bad_first = starts[0] < 0
        p, k = want_plan([good], [3], 1)
        got = pos.tolist()
        assert got[:4] == ([-7] * 4 if bad_first else p)
        assert got[4:] == (p if bad_first else [-7] * 4)


def test_tree_plan_refusals():
    p, s, c = ints([-1, 0]), ints([0, 2]), ints([4])
    pos, m = ints([0, 0]), torch.zeros(2, 1, dtype=I32, device="cuda")
    with pytest.raises(rel.MoeError):
        rel.tree_plan(p, s, c, positions=p, mask=m)
    with pytest.raises(rel.MoeError):
        rel.tree_plan(p, s, c, positions=pos, mask=torch.zeros(2, 9, dtype=I32, device="cuda"))
    for kw in (dict(positions=pos[:1], mask=m), dict(positions=pos, mask=m[:1]), dict(positions=pos, mask=m.long()),
               dict(positions=pos, mask=torch.zeros(2, 2, dtype=I32, device="cuda")[:, :1]), dict(positions=pos, mask=m[:, 0])):
        with pytest.raises(ValueError):
            rel.tree_plan(p, s, c, **kw)
    with pytest.raises(ValueError):
        rel.tree_plan(p, s[:1], c, positions=pos, mask=m)
    rel.tree_plan(p[:0], ints([0, 0]), c, positions=pos[:0], mask=m[:0])  # nothing to write


# ---- attention ---------------------------------------------------------------------------------


class Case:
    """Requests of (context, new) tokens over a paged cache with random masks (or trees' masks)."""

    def __init__(self, ctx, new, Hq, Hkv, D, P, words, dtype=BF16, masks="tree", seed=0, head_layout=False, scale_q=1.5):
        r = random.Random(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.ctx, self.new, self.words = ctx, new, words
        kv = [c + n for c, n in zip(ctx, new)]
        B, N = len(ctx), sum(new)
        W = max(1, -(-max(kv) // P)) + 1
        pages = sum(-(-max(t, 0) // P) for t in kv) + 3
        order = torch.randperm(pages, generator=g, device="cuda").tolist()
        table = [[-1] * W for _ in range(B)]
        for b, t in enumerate(kv):
            for i in range(-(-max(t, 0) // P)):
                table[b][i] = order.pop()
        self.table, self.kv = ints(table), ints(kv)
        shape = (pages, Hkv, P, D) if head_layout else (pages, P, Hkv, D)
        self.k, self.v = randn(*shape).to(dtype), randn(*shape).to(dtype)
        if head_layout:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.q = (randn(N, Hq, D) * scale_q).to(dtype)
        self.q_start = ints(starts_of([[0] * n for n in new]))
        self.masks = []
        for n in new:
            if masks == "tree":
                self.masks.append(dref.ancestors(dref.random_tree(r, n))[0] if n else [])
            elif masks == "any":  # any bits, empty rows and bits behind the last new token among them
                self.masks.append([r.choice([0, r.getrandbits(32 * words), 1 << r.randrange(32 * words)]) for _ in range(n)])
            else:
                self.masks.append([(2 << t) - 1 for t in range(n)])
        rows = flat([[dref.words_of(m, words) for m in q] for q in self.masks])
        self.mask = ints(rows) if rows else torch.zeros(0, words, dtype=I32, device="cuda")
        self.scale = D ** -0.5

    def forward(self, handle, mask=True, max_new=0, out=None, lse=None, stream=None):
        out = torch.full_like(self.q, 7.0) if out is None else out
        handle.forward(self.q, self.k, self.v, self.table, self.q_start, self.kv, out, scale=self.scale, lse=lse,
                       max_new=max_new, tree=self.mask if mask else None, stream=stream)
        return out

    def check(self, handle, **kw):
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        out = self.forward(handle, lse=lse, **kw)
        want, wl, slack, ls = dref.attention(self.q, self.k, self.v, self.table, self.q_start, self.kv,
                                             dref.by_bits(self.masks, self.words), self.scale)
        inside(out, want, ref.stored(want, self.q.dtype, slack))
        inside(lse, wl, ls)
        assert handle.get_error() == 0
        return out


@pytest.fixture(scope="module")
def handle():
    h = rel.PagedAttention(device=0)
    yield h
    h.close()


@pytest.mark.parametrize("masks", ["tree", "any"])
@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,P,words,dtype,head_layout", [
    ([0], [1], 1, 1, 64, 16, 1, BF16, False),
    ([7], [5], 8, 2, 128, 16, 1, F16, False),
    ([100, 0, 33], [4, 4, 4], 12, 1, 128, 64, 1, BF16, True),
    ([63, 64, 65, 0], [32, 31, 1, 0], 8, 4, 64, 32, 1, F16, True),
    ([200, 129], [64, 33], 24, 2, 128, 16, 2, BF16, False),
    ([1000, 3], [60, 256], 5, 1, 64, 64, 8, BF16, False),
    ([5, 300], [130, 100], 128, 1, 128, 128, 5, F16, False),
    ([31, 95], [40, 7], 4, 4, 128, 1024, 2, BF16, True),
    ([2500], [17], 20, 4, 128, 32, 3, BF16, False),
])
def test_tree_attention(handle, masks, ctx, new, Hq, Hkv, D, P, words, dtype, head_layout):
    c = Case(ctx, new, Hq, Hkv, D, P, words, dtype, masks, seed=sum(ctx) + D, head_layout=head_layout)
    a = c.check(handle)
    b = c.check(handle, max_new=max(new))
    if max(new) > 32 * words:
        assert torch.equal(a, b)


def test_tree_attention_mixed_with_chunks(handle):
    """Trees, decoding requests, a prompt longer than the mask and an idle request in one call."""
    c = Case([50, 700, 0, 129, 9], [33, 1, 90, 0, 64], 12, 2, 128, 16, 2, masks="tree", seed=5)
    c.check(handle)
    c = Case([50, 700, 0, 9], [33, 1, 300, 64], 8, 2, 64, 32, 2, F16, masks="any", seed=6)
    c.check(handle)


@pytest.mark.parametrize("D,Hq,Hkv,new", [(128, 12, 1, [10, 3, 1]), (64, 8, 8, [40, 16, 64]), (128, 4, 1, [1, 1, 1])])
def test_tree_attention_in_a_row_is_plain_attention(handle, D, Hq, Hkv, new):
    """Masks of all tokens before a row: what the call without masks computes."""
    c = Case([300, 77, 4000], new, Hq, Hkv, D, 64, 2, masks="row", seed=D)
    c.check(handle, max_new=max(new))
    c.check(handle, max_new=max(new), mask=False)


def test_tree_attention_short_context_and_negative(handle):
    """kv_lens below the number of new tokens: the first new tokens have no key (bit j is cache row ctx + j)."""
    c = Case([-3, -40, -1], [8, 40, 1], 8, 2, 64, 16, 2, masks="any", seed=3)
    out = c.check(handle)
    assert bool((out[8:] == 0).all())


def test_tree_attention_empty_rows(handle):
    """Rows that see nothing get zeros and -inf beside rows that see something."""
    c = Case([0, 0], [32, 5], 8, 2, 128, 16, 1, masks="any", seed=4)
    for t in range(0, 32, 2):
        c.masks[0][t] = 0
    c.masks[1] = [0] * 5
    c.mask = ints(flat([[dref.words_of(m, 1) for m in q] for q in c.masks]))
    out = c.check(handle)
    assert bool((out[0:32:2] == 0).all()) and bool((out[32:] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv", [(24, 2), (2, 2)])
def test_tree_attention_hidden_values(handle, dtype, Hq, Hkv):
    """NaN and infinities in keys and values that a row does not see leave it as it was; rows that see them are not
    finite where the formula is not."""
    c = Case([40, 130], [20, 50], Hq, Hkv, 64, 16, 2, dtype, masks="tree", seed=8)
    clean = c.check(handle)
    for b, t in ((0, 7), (1, 33)):
        at = c.ctx[b] + t
        page, row = int(c.table[b, at // 16]), at % 16
        c.k[page, row] = math.nan
        c.v[page, row, :, ::3] = math.inf
        c.v[page, row, :, 1::3] = math.nan
    out = c.forward(handle)
    n0 = [0, 20]
    for b, t in ((0, 7), (1, 33)):
        for row in range(c.new[b]):
            if c.masks[b][row] >> t & 1:
                assert bool(out[n0[b] + row].isnan().any())
            else:
                assert torch.equal(out[n0[b] + row], clean[n0[b] + row]), (b, row)
    # values alone: the infinity arrives at the rows that see it, with its sign
    c = Case([40, 130], [20, 50], Hq, Hkv, 64, 16, 2, dtype, masks="tree", seed=8)
    page, row = int(c.table[1, (130 + 33) // 16]), (130 + 33) % 16
    c.v[page, row, :, 5] = -math.inf
    out = c.forward(handle)
    for t in range(50):
        if c.masks[1][t] >> 33 & 1:
            assert bool((out[20 + t, :, 5] == -math.inf).all())
            keep = [d for d in range(64) if d != 5]
            assert torch.equal(out[20 + t][:, keep], clean[20 + t][:, keep])
        else:
            assert torch.equal(out[20 + t], clean[20 + t])


def test_tree_attention_split_items(handle):
    """Few requests with long contexts: items cut into pieces and joined, the masked tiles in the last ones."""
    Case([9000], [3], 12, 1, 128, 64, 1, masks="tree", seed=11).check(handle)
    Case([5000, 12], [24, 24], 16, 2, 64, 16, 1, F16, masks="tree", seed=12).check(handle)
    Case([8000], [64], 8, 1, 128, 128, 2, masks="tree", seed=13).check(handle)


def test_tree_attention_does_not_write_beyond_its_requests(handle):
    c = Case([20, 30], [6, 9], 4, 1, 64, 16, 1, seed=1)
    wide = torch.full((20, 4, 64), 3.0, dtype=BF16, device="cuda")
    q = torch.cat([c.q, c.q[:5]])
    mask = torch.cat([c.mask, c.mask[:5]])
    handle.forward(q, c.k, c.v, c.table, c.q_start, c.kv, wide, scale=c.scale, tree=mask)
    assert bool((wide[15:] == 3.0).all())
    assert torch.equal(wide[:15], c.forward(handle))


def test_tree_attention_strides_and_nothing(handle):
    """q and out inside wider rows, a table of wider rows; calls without tokens or requests write nothing."""
    c = Case([40, 130, 3], [20, 50, 7], 8, 2, 64, 16, 2, masks="tree", seed=30)
    want = c.check(handle)
    wide = torch.full((77, 8, 192), 2.0, dtype=BF16, device="cuda")
    wide[:, :, :64] = c.q
    c.q = wide[:, :, :64]
    table = torch.nn.functional.pad(c.table, (1, 3), value=-1)
    c.table = table[:, 1:1 + c.table.shape[1]]
    out = wide[:, :, 128:]
    c.forward(handle, out=out)
    assert torch.equal(out, want) and bool((wide[:, :, 64:128] == 2).all())
    handle.forward(c.q[:0], c.k, c.v, c.table, torch.zeros(4, dtype=I32, device="cuda"), c.kv, out[:0], scale=1.0, tree=c.mask[:0])
    handle.forward(c.q, c.k, c.v, c.table[:0], c.q_start[:1], c.kv[:0], out, scale=1.0, tree=c.mask)
    assert torch.equal(out, want) and handle.get_error() == 0


def test_tree_attention_refusals(handle):
    c = Case([20], [6], 4, 1, 64, 16, 1, seed=1)
    for bad in (c.mask[:5], c.mask.long(), c.mask.flatten(), c.mask.cpu(), torch.zeros(6, 2, dtype=I32, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            handle.forward(c.q, c.k, c.v, c.table, c.q_start, c.kv, torch.empty_like(c.q), scale=1.0, tree=bad)
    for words in (0, 9):
        with pytest.raises(rel.MoeError):
            handle.forward(c.q, c.k, c.v, c.table, c.q_start, c.kv, torch.empty_like(c.q), scale=1.0,
                           tree=torch.zeros(6, words, dtype=I32, device="cuda"))
    assert handle.get_error() == 0


# ---- acceptance --------------------------------------------------------------------------------


class Drafts:
    def __init__(self, sizes, ctx, layers, Hkv, D, P, seed=0, dtype=BF16, certain=None, follow=0.8, vocabulary=50):
        r = random.Random(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.parents = [dref.random_tree(r, n) if n else [] for n in sizes]
        self.certain = certain
        if certain:
            for p, c in zip(self.parents, certain):
                p[:c] = list(range(-1, c - 1))
                for j in range(c, len(p)):
                    p[j] = max(p[j], c - 1)
        # few different tokens: siblings often share one, and the lowest has to win
        self.tokens = [[r.randrange(vocabulary) for _ in p] for p in self.parents]
        self.targets = []
        for p, t in zip(self.parents, self.tokens):
            kids = [[j for j in range(len(p)) if p[j] == i] for i in range(len(p))]
            self.targets.append([t[r.choice(k)] if k and r.random() < follow else r.randrange(vocabulary, 2 * vocabulary) for k in kids])
        self.ctx, self.P = ctx, P
        W = max(c + n for c, n in zip(ctx, sizes)) // P + 2
        pages = sum(-(-(c + n) // P) for c, n in zip(ctx, sizes)) + 2
        order = torch.randperm(pages, generator=g, device="cuda").tolist()
        self.table = [[order.pop() if i < -(-(c + n) // P) else -1 for i in range(W)] for c, n in zip(ctx, sizes)]
        self.k, self.v = (torch.randn(layers, pages, P, Hkv, D, generator=g, device="cuda").to(dtype) for _ in range(2))

    def run(self, depth, err=None, k=None, v=None, stream=None):
        B = len(self.parents)
        self.path = torch.full((B, depth), -9, dtype=I32, device="cuda")
        self.accepted, self.ctx_out, self.next = (torch.full((B,), -9, dtype=I32, device="cuda") for _ in range(3))
        rel.tree_accept(ints(flat(self.parents)), ints(flat(self.tokens)), ints(flat(self.targets)),
                        ints(starts_of(self.parents)), ints(self.ctx), ints(self.table), self.k if k is None else k,
                        self.v if v is None else v, path=self.path, accepted=self.accepted, ctx_out=self.ctx_out,
                        next_tokens=self.next, certain=None if self.certain is None else ints(self.certain), err=err,
                        stream=stream)

    def check(self, depth, k=None, v=None):
        wk, wv = self.k.clone(), self.v.clone()
        err = torch.zeros(1, dtype=I32, device="cuda")
        self.run(depth, err, k, v)
        moved = 0
        for b, p in enumerate(self.parents):
            c = self.certain[b] if self.certain else 1
            path, accepted, nxt = dref.accept(p, self.tokens[b], self.targets[b], c, depth)
            assert self.path[b].tolist() == path + [-1] * (depth - len(path))
            assert [int(t[b]) for t in (self.accepted, self.ctx_out, self.next)] == [accepted, self.ctx[b] + accepted, nxt]
            for cache in (wk, wv):
                dref.move(cache, self.table[b], self.ctx[b], c, path, self.P)
            moved += sum(j != c + i for i, j in enumerate(path))
        assert torch.equal(self.k.view(torch.int16), wk.view(torch.int16))
        assert torch.equal(self.v.view(torch.int16), wv.view(torch.int16))
        assert int(err.item()) == 0
        return moved


@pytest.mark.parametrize("sizes,layers,Hkv,D,P,depth,dtype", [
    ([1], 1, 1, 64, 16, 1, BF16), ([25], 1, 8, 128, 64, 6, BF16), ([60] * 7 + [0, 1, 2], 3, 2, 128, 16, 8, F16),
    ([300, 40, 33], 2, 4, 64, 32, 12, BF16), ([64] * 60, 5, 1, 128, 16, 5, BF16), ([17, 90], 2, 3, 33, 16, 20, F16),
    ([12] * 3, 40, 8, 128, 4, 7, BF16), ([256], 1, 1, 1, 1, 256, F16), ([513, 1200], 1, 2, 64, 64, 30, BF16),
])
def test_tree_accept(sizes, layers, Hkv, D, P, depth, dtype):
    moved = 0
    for seed in range(4):
        ctx = [random.Random(seed + b).randrange(70) for b in range(len(sizes))]
        moved += Drafts(sizes, ctx, layers, Hkv, D, P, seed, dtype, follow=0.95 if seed else 0.0, vocabulary=4).check(depth)
    assert moved > 0 or max(sizes) < 3


def test_tree_accept_chain_of_many():
    """A path longer than a warp, and rows that move by one place each: sources are others' destinations."""
    d = Drafts([200], [33], 2, 2, 64, 16, seed=1)
    d.parents = [[-1, 0] + [0 if j == 2 else j - 1 for j in range(2, 200)]]  # node 1 is a leaf, 2.. a chain below the root
    d.tokens = [list(range(200))]
    d.targets = [[2] + [999] + list(range(3, 200)) + [777]]
    assert d.check(198) == 198
    assert int(d.next[0]) == 777


def test_tree_accept_certain():
    """Prompt tokens that stay in any case: all of a chunk, some before a tree, one."""
    for seed in range(3):
        d = Drafts([40, 40, 7, 9], [5, 100, 0, 31], 2, 2, 64, 16, seed=seed, certain=[40, 10, 1, 9], vocabulary=3)
        d.check(6)


def test_tree_accept_layouts():
    """A cache of one layer without the layers' dimension, heads before rows, strides between layers, elements that
    start off a 16-byte boundary, keys and values in one allocation."""
    for seed, form in enumerate(["one", "heads", "offset", "paired"]):
        d = Drafts([30, 50], [9, 22], 1 if form == "one" else 3, 4, 64, 16, seed=seed, vocabulary=3, follow=0.95)
        k, v = d.k, d.v
        if form == "one":
            d.check(8, k=k[0], v=v[0])
            continue
        if form == "heads":
            d.k, d.v = (t.transpose(2, 3).contiguous().transpose(2, 3) for t in (k, v))
        elif form == "offset":
            d.k, d.v = (torch.nn.functional.pad(t, (3, 2))[..., 3:67] for t in (k, v))
        else:
            both = torch.stack([k, v], dim=2)
            d.k, d.v = both[:, :, 0], both[:, :, 1]
        wk, wv = d.k.contiguous(), d.v.contiguous()
        d.run(8)
        for b, p in enumerate(d.parents):
            path = dref.accept(p, d.tokens[b], d.targets[b], 1, 8)[0]
            for cache in (wk, wv):
                dref.move(cache, d.table[b], d.ctx[b], 1, path, 16)
        assert torch.equal(d.k, wk) and torch.equal(d.v, wv), form


def test_tree_accept_bad_input():
    """certain outside [1, new] is clamped; rows without a page stay; a request outside the rows counts as empty."""
    d = Drafts([20, 20], [3, 40], 1, 1, 64, 16, seed=3, certain=[1, 1])
    d.certain = [0, 21]
    err = torch.zeros(1, dtype=I32, device="cuda")
    d.run(5, err)
    path, accepted, nxt = dref.accept(d.parents[0], d.tokens[0], d.targets[0], 1, 5)
    assert int(err.item()) == rel.MOE_OPS_ERR_PLAN
    assert d.accepted.tolist() == [accepted, 20] and int(d.next[1]) == d.targets[1][19]
    for spoil in (-1, 1 << 20):
        d = Drafts([200], [33], 1, 1, 64, 16, seed=1)
        d.parents = [[-1, 0] + [0 if j == 2 else j - 1 for j in range(2, 200)]]
        d.tokens, d.targets = [list(range(200))], [[2] + [999] + list(range(3, 200)) + [777]]
        d.table[0][5] = spoil
        k0, wk = d.k.clone(), d.k.clone()
        err.zero_()
        d.run(198, err)
        assert int(err.item()) == rel.MOE_OPS_ERR_INDEX and d.path[0].tolist() == list(range(2, 200))
        for i, j in enumerate(range(2, 200)):
            s, t = 33 + j, 33 + 1 + i
            if 5 not in (s // 16, t // 16):
                wk[:, d.table[0][t // 16], t % 16] = k0[:, d.table[0][s // 16], s % 16]
        assert torch.equal(wk, d.k)
    d = Drafts([20, 20], [3, 40], 1, 1, 64, 16, seed=3)
    k0 = d.k.clone()
    err.zero_()
    B = 2
    outs = [torch.full((B, 4), -9, dtype=I32, device="cuda")] + [torch.full((B,), -9, dtype=I32, device="cuda") for _ in range(3)]
    rel.tree_accept(ints(flat(d.parents)), ints(flat(d.tokens)), ints(flat(d.targets)), ints([-4, 41, 30]), ints(d.ctx),
                    ints(d.table), d.k, d.v, path=outs[0], accepted=outs[1], ctx_out=outs[2], next_tokens=outs[3], err=err)
    assert int(err.item()) == rel.MOE_OPS_ERR_INDEX and outs[1].tolist() == [0, 0] and outs[2].tolist() == d.ctx
    assert outs[3].tolist() == [-1, -1] and outs[0].tolist() == [[-1] * 4] * 2 and torch.equal(k0, d.k)


def test_tree_accept_refusals():
    d = Drafts([20], [3], 1, 1, 64, 16, seed=3)
    one = lambda: torch.zeros(1, dtype=I32, device="cuda")
    args = [ints(flat(d.parents)), ints(flat(d.tokens)), ints(flat(d.targets)), ints([0, 20]), ints(d.ctx), ints(d.table), d.k, d.v]
    outs = dict(path=torch.zeros(1, 4, dtype=I32, device="cuda"), accepted=one(), ctx_out=one(), next_tokens=one())
    rel.tree_accept(*args, **outs)
    for kw in (dict(ctx_out=args[4]), dict(accepted=outs["ctx_out"]), dict(next_tokens=args[1][:1]),
               dict(path=torch.zeros(1, 257, dtype=I32, device="cuda")), dict(path=torch.zeros(1, 0, dtype=I32, device="cuda"))):
        with pytest.raises(rel.MoeError):
            rel.tree_accept(*args, **{**outs, **kw})
    for kw in (dict(path=outs["path"][0]), dict(accepted=torch.zeros(2, dtype=I32, device="cuda")),
               dict(certain=torch.zeros(2, dtype=I32, device="cuda")), dict(ctx_out=one().long())):
        with pytest.raises(ValueError):
            rel.tree_accept(*args, **{**outs, **kw})
    for i, bad in ((1, args[1][:5]), (3, args[3][:1]), (6, d.k[0, 0]), (6, d.k.float()), (7, d.v[:, :2]), (5, args[5][0])):
        with pytest.raises(ValueError):
            rel.tree_accept(*(bad if j == i else t for j, t in enumerate(args)), **outs)


def test_tree_steps_in_graphs_and_on_streams(handle):
    """Plan, attention and acceptance on a side stream and captured, replayed on other inputs: as called plainly."""
    c = Case([300, 20], [24, 9], 8, 2, 64, 16, 1, seed=21)
    parents = [dref.random_tree(random.Random(1), n) for n in c.new]
    pp, ctx = ints(flat(parents)), ints(c.ctx)
    pos, mask = torch.zeros(33, dtype=I32, device="cuda"), torch.zeros(33, 1, dtype=I32, device="cuda")
    out = torch.zeros_like(c.q)
    tokens, targets = ints(list(range(33))), ints([0] * 33)
    path, acc, ctx2, nxt = (torch.zeros(*s, dtype=I32, device="cuda") for s in ((2, 4), (2,), (2,), (2,)))

    def step(s):
        rel.tree_plan(pp, c.q_start, ctx, positions=pos, mask=mask, stream=s)
        handle.forward(c.q, c.k, c.v, c.table, c.q_start, c.kv, out, scale=c.scale, tree=mask, stream=s)
        rel.tree_accept(pp, tokens, targets, c.q_start, ctx, c.table, c.k, c.v, path=path, accepted=acc, ctx_out=ctx2,
                        next_tokens=nxt, stream=s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.synchronize()
    want = [t.clone() for t in (pos, mask, out, acc, nxt)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    for t in (pos, mask, out, acc, nxt):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for t, w in zip((pos, mask, out, acc, nxt), want):
        assert torch.equal(t, w)
    other = [dref.random_tree(random.Random(2), n, width=1.2) for n in c.new]
    pp.copy_(ints(flat(other)))
    graph.replay()
    torch.cuda.synchronize()
    again = out.clone()
    step(None)
    torch.cuda.synchronize()
    assert torch.equal(again, out) and not torch.equal(again, want[2])
    assert mask.tolist() == flat([[dref.words_of(m, 1) for m in dref.ancestors(p)[0]] for p in other])
    assert handle.get_error() == 0
