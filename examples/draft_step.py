"""One decoder layer with 8-bit projections that checks drafted tokens: every step brings a tree of drafts per request, the
model's own tokens choose a path through it, and the cache keeps the path.

    plan, mask = pages and slots; positions and ancestor masks    paged_plan, tree_plan
    h, n8      = residual norm, e4m3 with scales per 128          add_rmsnorm
    q, k, v    = n8 W_qkv                                         Matmul8
    q, cache   = rotary, k and v appended                         rotary_append
    o          = attention by the masks over the pages            PagedAttention
    h, m       = residual norm of (o in e4m3) W_o                 quantize8, Matmul8, add_rmsnorm
    out        = routed experts of m                              MoeLayer
    ctx        = the path accepted, its rows moved in the cache   tree_accept

    python examples/draft_step.py      # greedy decoding of a small model token by token, then with drafts
"""
from __future__ import annotations

import os
import random
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import torch  # noqa: E402

import routed_expert_layer_gb300 as rel  # noqa: E402

E4M3 = torch.float8_e4m3fn


def quantized(x, rows: int = 1):
    """x [T][H] in e4m3 and its scales: blocks of 128 of a row, or (rows = 128, weights) of 128 x 128."""
    T, H = x.shape
    x8 = torch.empty(T, H, dtype=E4M3, device=x.device)
    scales = torch.empty(-(-T // rows), -(-H // 128), device=x.device)
    rel.quantize8(x, x8, scales, group=128, rows=rows)
    return x8, scales


class DraftLayer:
    """A layer with its paged cache for up to `requests` requests of `max_len` tokens, drafts included."""

    def __init__(self, moe, q_heads: int, kv_heads: int, head_dim: int, requests: int, max_len: int, page_size: int = 16,
                 mask_words: int = 1, seed: int = 0):
        self.moe, self.H = moe, moe.H
        self.Hq, self.Hkv, self.D, self.P, self.words = q_heads, kv_heads, head_dim, page_size, mask_words
        dev, dt = torch.device("cuda"), torch.bfloat16
        g = torch.Generator(device=dev)
        g.manual_seed(seed)

        def weight(out, inner):
            return quantized((torch.randn(out, inner, generator=g, device=dev) * inner ** -0.5).to(dt), rows=128)

        self.qkv8 = weight((q_heads + 2 * kv_heads) * head_dim, self.H)
        self.o8 = weight(self.H, q_heads * head_dim)
        self.norm1, self.norm2 = (1.0 + (torch.randn(self.H, generator=g, device=dev) * 0.1).to(dt) for _ in range(2))
        self.inv_freq = rel.rope_frequencies(head_dim)
        width = -(-max_len // page_size)
        pages = requests * width
        self.k_cache, self.v_cache = (torch.empty(pages, page_size, kv_heads, head_dim, dtype=dt, device=dev)
                                      for _ in range(2))
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device=dev)
        self.free = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        self.heads = torch.zeros(2, 1, dtype=torch.int32, device=dev)  # position in the free list: now, after the step
        self.ctx = torch.zeros(requests, dtype=torch.int32, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.attention, self.matmul = rel.PagedAttention(device=0), rel.Matmul8(device=0)

    def project(self, x8, scales, weight):
        out = torch.empty(x8.shape[0], weight[0].shape[0], dtype=torch.bfloat16, device=x8.device)
        self.matmul.forward(x8, scales, *weight, out)
        return out

    def step(self, x, residual, parents: list[list[int]]):
        """x, residual [nodes][H] of the requests' new tokens, parents[b] of request b's (a chain of known tokens, or a
        tree behind its root). Returns (expert output, residual, norm2 output); the drafts stay in the cache until
        accept()."""
        new = [len(p) for p in parents]
        N, B = sum(new), len(new)
        i32 = dict(dtype=torch.int32, device=x.device)
        self.parents = torch.tensor([p for q in parents for p in q], **i32)
        self.q_start, kv_lens = torch.empty(B + 1, **i32), torch.empty(B, **i32)
        positions, slots = torch.empty(N, **i32), torch.empty(N, **i32)
        mask = torch.empty(N, self.words, **i32)
        rel.paged_plan(self.ctx, torch.tensor(new, **i32), self.table, self.free, self.heads[0], self.P, q_start=self.q_start,
                       kv_lens=kv_lens, positions=positions, slots=slots, free_head_out=self.heads[1], err=self.err)
        rel.tree_plan(self.parents, self.q_start, self.ctx, positions=positions, mask=mask, err=self.err)

        h, n8 = torch.empty_like(x), torch.empty(N, self.H, dtype=E4M3, device=x.device)
        scales = torch.empty(N, -(-self.H // 128), device=x.device)
        rel.add_rmsnorm(x, self.norm1, 1e-6, residual=residual, residual_out=h, out8=n8, scales=scales, group=128)
        qkv = self.project(n8, scales, self.qkv8)
        a, b = self.Hq * self.D, (self.Hq + self.Hkv) * self.D
        q, k, v = (t.view(N, -1, self.D) for t in (qkv[:, :a], qkv[:, a:b], qkv[:, b:]))
        rel.rotary_append(q, k, v, positions, slots, self.inv_freq, self.k_cache, self.v_cache, err=self.err)  # q in place
        o = torch.zeros(N, self.Hq, self.D, dtype=x.dtype, device=x.device)
        self.attention.forward(q, self.k_cache, self.v_cache, self.table, self.q_start, kv_lens, o, scale=self.D ** -0.5,
                               max_new=max(new), tree=mask)
        m = torch.empty_like(x)
        rel.add_rmsnorm(self.project(*quantized(o.view(N, a)), self.o8), self.norm2, 1e-6, out=m, residual=h, residual_out=h)
        out = torch.empty_like(x)
        self.moe.forward(m, out)
        self.heads = self.heads.flip(0)
        self.kv_lens = kv_lens
        return out, h, m

    def accept(self, tokens, targets, certain, depth: int):
        """tokens, targets int32 [nodes]: the nodes' tokens and the model's after each; certain int32 [B]: how many first
        nodes are known. Returns (path [B][depth], next tokens [B]); the pages that the drafts no longer need are
        free again."""
        B = self.ctx.numel()
        i32 = dict(dtype=torch.int32, device=tokens.device)
        path, accepted = torch.empty(B, depth, **i32), torch.empty(B, **i32)
        ctx, following = torch.empty(B, **i32), torch.empty(B, **i32)
        rel.tree_accept(self.parents, tokens, targets, self.q_start, self.ctx, self.table, self.k_cache, self.v_cache, path=path,
                        accepted=accepted, ctx_out=ctx, next_tokens=following, certain=certain, err=self.err)
        col = torch.arange(self.table.shape[1], device=tokens.device)[None, :]
        kept, had = (-(-t[:, None] // self.P) for t in (ctx, self.kv_lens))
        unused = (col >= kept) & (col < had)
        back = self.table[unused]
        head = int(self.heads[0].item())
        self.free[head - back.numel():head] = back
        self.heads[0] -= back.numel()
        self.table[unused] = -1
        self.ctx = ctx
        return path, following

    def close(self) -> None:
        self.attention.close()
        self.matmul.close()


def decode(layer, embed, prompts, count: int, draft):
    """Greedy decoding of `count` tokens a request. draft(b, tokens so far) gives (tokens, parents) of a tree behind the
    last token, whose parent is -1. Returns the sequences and the number of steps."""
    B = len(prompts)
    sequences = [list(p) for p in prompts]
    fresh = [list(p) for p in prompts]  # known tokens that are not in the cache yet
    steps = 0
    while min(len(s) - len(p) for s, p in zip(sequences, prompts)) < count:
        tokens, parents = [], []
        for b in range(B):
            more, up = draft(b, sequences[b]) if steps else ([], [])
            c = len(fresh[b])
            tokens.append(fresh[b] + more)
            parents.append(list(range(-1, c - 1)) + [c - 1 + (p + 1) for p in up])
        flat = torch.tensor([t for row in tokens for t in row], dtype=torch.int32, device="cuda")
        x = embed[flat.long()]
        out, h, _ = layer.step(x, torch.zeros_like(x), parents)
        targets = ((out + h).float() @ embed.float().t()).argmax(dim=1).to(torch.int32)
        certain = torch.tensor([len(f) for f in fresh], dtype=torch.int32, device="cuda")
        path, following = layer.accept(flat, targets, certain, depth=8)
        steps += 1
        for b, (row, nxt) in enumerate(zip(path.tolist(), following.tolist())):
            fresh[b] = [nxt]
            sequences[b] += [tokens[b][j] for j in row if j >= 0] + [nxt]
    return [s[:len(p) + count] for s, p in zip(sequences, prompts)], steps


def main():
    """Returns the sequences decoded plainly and with drafts, and the steps of both."""
    import synth
    H, I, E, k, vocabulary, count = 512, 256, 64, 8, 300, 24
    moe = rel.MoeLayer(H, I, E, k, max_tokens=1024)
    moe.load(synth.layer(H, I, E, seed_weights=1, seed_router=2))
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    embed = torch.randn(vocabulary, H, generator=g, device="cuda").bfloat16()
    r = random.Random(3)
    prompts = [[r.randrange(vocabulary) for _ in range(n)] for n in (50, 7, 1)]
    make = lambda: DraftLayer(moe, q_heads=8, kv_heads=2, head_dim=64, requests=3, max_len=160)

    def finish(layer):
        torch.cuda.synchronize()
        assert int(layer.err.item()) == 0 and layer.attention.get_error() == 0 and layer.matmul.get_error() == 0
        layer.close()

    layer = make()
    plain, plain_steps = decode(layer, embed, prompts, count, lambda b, s: ([], []))
    finish(layer)

    def draft(b, so_far):
        """Two branches from each level: the plain run's next tokens, one in five wrong, beside random ones."""
        tokens, parents, up = [], [], -1
        for t in plain[b][len(so_far):len(so_far) + 4]:
            tokens += [r.randrange(vocabulary), t if r.random() < 0.8 else r.randrange(vocabulary)]
            parents += [up, up]
            up = len(tokens) - 1
        return tokens, parents

    layer = make()
    drafted, steps = decode(layer, embed, prompts, count, draft)
    finish(layer)
    moe.close()
    same = sum(a == b for x, y in zip(plain, drafted) for a, b in zip(x, y))
    print(f"{len(prompts)} requests of {count} tokens: {plain_steps} steps token by token, {steps} with drafts; {same} of "
          f"{sum(map(len, plain))} tokens the same")
    return plain, drafted, plain_steps, steps


if __name__ == "__main__":
    main()
