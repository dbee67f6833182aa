"""Plain 64-bit forms of the operators for drafted tokens and 8-bit projections, and the error each result may have
(imported by test modules, not a test). Rounding units: ops_reference.py."""
from __future__ import annotations

import math

import torch

from ops_reference import F64, UNIT


def ancestors(parents):
    """(mask as a Python integer, depth) of each node."""
    bits, depth = [], []
    for t, up in enumerate(parents):
        bits.append(1 << t | (bits[up] if up >= 0 else 0))
        depth.append(depth[up] + 1 if up >= 0 else 0)
    return bits, depth


def words_of(bits, words):
    """A mask as `words` signed 32-bit integers."""
    out = []
    for w in range(words):
        v = bits >> (32 * w) & 0xFFFFFFFF
        out.append(v - (1 << 32) if v >> 31 else v)
    return out


def random_tree(r, n, width=3):
    """Parents in breadth-first order, about `width` children a node; node 0 is the root."""
    parents, up = [-1], 0
    for j in range(1, n):
        while up < j - 1 and r.random() < 1.0 / width:
            up += 1
        parents.append(up)
    return parents


def accept(parents, tokens, targets, certain, depth):
    """(path, accepted, next token) of one request."""
    if not parents:
        return [], 0, -1
    cur, path = certain - 1, []
    while len(path) < depth:
        child = [j for j in range(cur + 1, len(parents)) if parents[j] == cur and tokens[j] == targets[cur]]
        if not child:
            break
        cur = child[0]
        path.append(cur)
    return path, certain + len(path), targets[cur]


def move(cache, table, ctx, certain, path, P):
    """The accepted rows of one request in cache [layers][pages][P][Hkv][D], in place."""
    rows = [cache[:, table[(ctx + j) // P], (ctx + j) % P].clone() for j in path]
    for i, row in enumerate(rows):
        at = ctx + certain + i
        cache[:, table[at // P], at % P] = row


def attention(q, k_cache, v_cache, table, q_start, kv_lens, seen, scale):
    """64-bit attention over the keys that seen(b, t, n_new, ctx, kv) (a bool tensor [kv]) lets row t of request b see.
    Returns out, lse and the bounds of their errors before the output's own rounding, which are derived as
    ops_reference.attention's are: they do not depend on which keys are seen."""
    N, Hq, D = q.shape
    P, Hkv = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    out = torch.zeros(N, Hq, D, dtype=F64, device=q.device)
    lse = torch.full((N, Hq), -math.inf, dtype=F64, device=q.device)
    slack, lse_slack = torch.zeros_like(out), torch.zeros_like(lse)
    unit = UNIT[q.dtype]
    starts, lens = q_start.tolist(), kv_lens.tolist()
    for b, kv in enumerate(lens):
        n0, n1 = starts[b], starts[b + 1]
        if n1 <= n0 or kv <= 0:
            continue
        at = torch.arange(kv, device=q.device)
        pages = table[b].long()[at // P]
        k, v = (c[pages, at % P].to(F64) for c in (k_cache, v_cache))
        for n in range(n0, n1):
            see = seen(b, n - n0, n1 - n0, kv - (n1 - n0), kv).to(q.device)
            if not bool(see.any()):
                continue
            kk = k[see].permute(1, 2, 0).repeat_interleave(G, dim=0)
            vv = v[see].permute(1, 0, 2).repeat_interleave(G, dim=0)
            row = q[n].to(F64)[:, None]
            s = (row @ kk).squeeze(1) * scale
            size = (row.abs() @ kk.abs()).squeeze(1) * scale
            top = s.amax(dim=1, keepdim=True)
            p = torch.exp(s - top)
            total = p.sum(dim=1, keepdim=True)
            out[n] = (p[:, None] @ vv).squeeze(1) / total
            lse[n] = (top + torch.log(total)).squeeze(1)
            d = (2.0 ** -18 * size + 2.0 ** -21 * (s.abs() + top.abs())).amax(dim=1)
            mean_abs = (p[:, None] @ vv.abs()).squeeze(1) / total
            slack[n] = mean_abs * (unit + 2.0 * d[:, None] + 2.0 ** -17)
            lse_slack[n] = d + 2.0 ** -17 + 2.0 ** -22 * lse[n].abs()
    return out, lse, slack, lse_slack


def by_bits(masks, words):
    """seen() for attention(): masks[b][t] as Python integers; requests longer than 32 * words in a row."""
    def seen(b, t, n_new, ctx, kv):
        at = torch.arange(kv) - ctx
        if n_new > 32 * words:
            return at <= t
        bits = torch.tensor([masks[b][t] >> j & 1 for j in range(n_new)] + [0], dtype=torch.bool)
        return (at < 0) | bits[at.clamp(0, n_new)]
    return seen


def quantize(x, group, rows):
    """(x / scale, scale) in 64 bits over blocks of rows x group (group 0: the row)."""
    T, H = x.shape
    g = group or H
    f = torch.nn.functional.pad(x.to(F64), (0, -H % g, 0, -T % rows))
    blocks = f.view(f.shape[0] // rows, rows, f.shape[1] // g, g)
    s = blocks.abs().amax(dim=(1, 3)) / 448.0
    y = blocks / torch.where(s > 0, s, torch.ones_like(s))[:, None, :, None]
    return y.reshape(f.shape)[:T, :H], s


def matmul8(a8, a_scales, w8, w_scales):
    """(product, bound of its error before the output's own rounding) in 64 bits.

    A product of two e4m3 values has 8 significant bits and is exact in fp32. A block's 128 are summed by the tensor
    cores in fp32, 32 at a time: at worst each of 132 additions truncates at 2^-23 of the largest partial sum, which is no
    more than the sum of magnitudes: 2^-15 of it. Products of two scales and the sums over the blocks round once each."""
    (T, K), N = a8.shape, w8.shape[0]
    blocks = -(-K // 128)
    pad = lambda t: torch.nn.functional.pad(t.to(F64), (0, blocks * 128 - K))
    out = torch.zeros(T, N, dtype=F64, device=a8.device)
    size = torch.zeros_like(out)
    a, w = pad(a8.view(torch.float8_e4m3fn).float()), pad(w8.view(torch.float8_e4m3fn).float())
    ws = w_scales.to(F64).repeat_interleave(128, dim=0)[:N]
    for b in range(blocks):
        some = slice(128 * b, 128 * b + 128)
        s = a_scales.to(F64)[:, b if a_scales.shape[1] > 1 else 0, None] * ws[None, :, b]
        out += s * (a[:, some] @ w[:, some].t())
        size += s.abs() * (a[:, some].abs() @ w[:, some].abs().t())
    return out, size * (2.0 ** -15 + (blocks + 8) * 2.0 ** -24)
