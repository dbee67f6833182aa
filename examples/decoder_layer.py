"""One decoder layer served over a paged cache: the operators beside the expert layer and the
expert layer itself, as a serving step uses them.

    h, n   = residual norm                     add_rmsnorm
    q, k, v = n W_qkv                          (library product)
    plan   = pages, slots and positions        paged_plan
    q, cache = rotary, k and v appended        rotary_append
    o      = attention over the pages          PagedAttention
    h, m   = residual norm of o W_o            add_rmsnorm
    out    = routed experts of m               MoeLayer

    python examples/decoder_layer.py           # prompts in chunks, then decoding, on a small layer
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import torch  # noqa: E402

import routed_expert_layer_gb300 as rel  # noqa: E402


class DecoderLayer:
    """A layer with its paged cache for up to `requests` requests of `max_len` tokens."""

    def __init__(self, moe, q_heads: int, kv_heads: int, head_dim: int, requests: int, max_len: int, page_size: int = 64,
                 seed: int = 0):
        self.moe, self.H = moe, moe.H
        self.Hq, self.Hkv, self.D, self.P = q_heads, kv_heads, head_dim, page_size
        dev, dt = torch.device("cuda"), torch.bfloat16
        g = torch.Generator(device=dev)
        g.manual_seed(seed)

        def weight(*shape, scale):
            return (torch.randn(*shape, generator=g, device=dev) * scale).to(dt)

        self.w_qkv = weight(self.H, (q_heads + 2 * kv_heads) * head_dim, scale=self.H ** -0.5)
        self.w_o = weight(q_heads * head_dim, self.H, scale=(q_heads * head_dim) ** -0.5)
        self.norm1, self.norm2 = (1.0 + weight(self.H, scale=0.1) for _ in range(2))
        self.inv_freq = rel.rope_frequencies(head_dim)
        width = -(-max_len // page_size)
        pages = requests * width
        self.k_cache, self.v_cache = (torch.empty(pages, page_size, kv_heads, head_dim, dtype=dt, device=dev)
                                      for _ in range(2))
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device=dev)
        self.free = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        self.heads = torch.zeros(2, 1, dtype=torch.int32, device=dev)  # position in the free list: now, after the step
        self.ctx = torch.zeros(requests, dtype=torch.int32, device=dev)  # cached tokens of each request
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.attention = rel.PagedAttention(device=0)

    def step(self, x, residual, new: list[int]):
        """x, residual [sum(new)][H]: the layer below's output and the residual stream of each
        request's new tokens, request after request. Returns (expert output, residual, norm2 output).
        A step that does not fit the cache raises MOE_OPS_ERR_PLAN in self.err and leaves the layer's
        state as it was; what it returns is of no use."""
        N, B = sum(new), len(new)
        i32 = dict(dtype=torch.int32, device=x.device)
        new_lens = torch.tensor(new, **i32)
        q_start, kv_lens = torch.empty(B + 1, **i32), torch.empty(B, **i32)
        positions, slots = torch.empty(N, **i32), torch.empty(N, **i32)
        rel.paged_plan(self.ctx, new_lens, self.table, self.free, self.heads[0], self.P, q_start=q_start, kv_lens=kv_lens,
                       positions=positions, slots=slots, free_head_out=self.heads[1], err=self.err)

        h, n = torch.empty_like(x), torch.empty_like(x)
        rel.add_rmsnorm(x, self.norm1, 1e-6, out=n, residual=residual, residual_out=h)
        qkv = n @ self.w_qkv
        a, b = self.Hq * self.D, (self.Hq + self.Hkv) * self.D
        q, k, v = (t.view(N, -1, self.D) for t in (qkv[:, :a], qkv[:, a:b], qkv[:, b:]))
        rel.rotary_append(q, k, v, positions, slots, self.inv_freq, self.k_cache, self.v_cache, err=self.err)  # q in place
        # zeros: where the plan refuses the step (self.err says so) there is no request whose rows attention writes
        o = torch.zeros(N, self.Hq, self.D, dtype=x.dtype, device=x.device)
        self.attention.forward(q, self.k_cache, self.v_cache, self.table, q_start, kv_lens, o, scale=self.D ** -0.5,
                               max_new=max(new))
        m = torch.empty_like(x)
        rel.add_rmsnorm(o.view(N, a) @ self.w_o, self.norm2, 1e-6, out=m, residual=h, residual_out=h)
        out = torch.empty_like(x)
        self.moe.forward(m, out)
        self.ctx = self.ctx + q_start.diff()  # what the step brought: nothing if it was refused, where kv_lens is zeros
        self.heads = self.heads.flip(0)
        return out, h, m

    def close(self) -> None:
        self.attention.close()


def run(layer, x, residual, lengths, steps):
    """Feed each request's tokens (x, residual [request][token][H]) in `steps`, a list of new
    token counts per request; returns (out, h, m) put back in [request][token] order."""
    done = [0] * len(lengths)
    back = [[torch.empty(n, layer.H, dtype=x[0].dtype, device="cuda") for n in lengths] for _ in range(3)]
    for new in steps:
        rows = [slice(d, d + n) for d, n in zip(done, new)]
        parts = layer.step(torch.cat([t[r] for t, r in zip(x, rows)]), torch.cat([t[r] for t, r in zip(residual, rows)]),
                           new)
        for kept, got in zip(back, parts):
            for t, r, piece in zip(kept, rows, got.split(new)):
                t[r] = piece
        done = [d + n for d, n in zip(done, new)]
    assert done == list(lengths)
    return back


def main() -> list:
    """Returns each request's residual stream whole and in steps."""
    import synth
    H, I, E, k = 512, 256, 64, 8
    lengths = [333, 70, 1]
    moe = rel.MoeLayer(H, I, E, k, max_tokens=1024)
    moe.load(synth.layer(H, I, E, seed_weights=1, seed_router=2))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, residual = ([torch.randn(n, H, generator=g, device="cuda").bfloat16() for n in lengths] for _ in range(2))
    whole = [lengths]
    chunks = [[200, 64, 1], [100, 5, 0]] + [[1, 0, 0]] * 33 + [[0, 1, 0]]
    results = []
    for steps in (whole, chunks):
        layer = DecoderLayer(moe, q_heads=8, kv_heads=2, head_dim=64, requests=3, max_len=400, page_size=16)
        results.append(run(layer, x, residual, lengths, steps))
        torch.cuda.synchronize()
        assert int(layer.err.item()) == 0 and layer.attention.get_error() == 0 and moe.get_error() == 0
        layer.close()
    pairs = list(zip(results[0][1], results[1][1]))
    off = max(float((a.float() - b.float()).abs().max()) for a, b in pairs)
    print(f"{sum(lengths)} tokens of {len(lengths)} requests: residual stream whole against in {len(chunks)} steps, "
          f"max difference {off:.3g}")
    moe.close()
    return pairs


if __name__ == "__main__":
    main()
