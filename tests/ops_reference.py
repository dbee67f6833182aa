"""Plain 64-bit forms of the operators beside the expert layer, and the error each result
may have (imported by test modules, not a test).

Rounding units: a value rounded to bf16 (8 significant bits) is off by at most 2^-8 of itself, to
f16 (11 bits) by 2^-11 (2^-25 at least: half the smallest subnormal); fp32 arithmetic of a few
operations by less than 2^-20 (16 roundings of 2^-24)."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
FP32 = 2.0 ** -20


def stored(ref, dtype, slack):
    """Bound on |stored - ref|: rounding of a value within slack of ref to dtype, plus slack."""
    return UNIT[dtype] * (ref.abs() + slack) + TINY[dtype] + slack


def norm(x, weight, eps, residual=None, group=None):
    """(t, y, scales or None) of the residual norm; group None: no 8-bit output."""
    t = x.to(F64) + (0.0 if residual is None else residual.to(F64))
    y = t / torch.sqrt((t * t).mean(dim=1, keepdim=True) + eps) * weight.to(F64)
    if group is None:
        return t, y, None
    width = group or y.shape[1]
    tops = [b.abs().amax(dim=1) / 448.0 for b in torch.split(y, width, dim=1)]
    return t, y, torch.stack(tops, dim=1)


def plan(ctx, new, table, free, head, P, N):
    """The step's plan with Python integers; table: list of rows. Returns a dict of lists, or
    None where the step does not fit."""
    table = [list(r) for r in table]
    q_start, pos, slots, kv = [0], [], [], []
    at = head
    if any(c < 0 or n < 0 for c, n in zip(ctx, new)) or sum(new) > N or head < 0:
        return None
    for b, (c, n) in enumerate(zip(ctx, new)):
        for col in range(-(-c // P), -(-(c + n) // P)):
            if col >= len(table[b]) or at >= len(free):
                return None
            table[b][col] = free[at]
            at += 1
        if c + n > len(table[b]) * P:
            return None
        for t in range(n):
            p = c + t
            pos.append(p)
            slots.append(table[b][p // P] * P + p % P)
        q_start.append(q_start[-1] + n)
        kv.append(c + n)
    pad = N - len(pos)
    return dict(block_table=table, q_start=q_start, kv_lens=kv, positions=pos + [0] * pad, slots=slots + [-1] * pad,
                free_head_out=[at])


def rotate(x, positions, inv_freq, mscale, interleaved):
    """(rotated x, sum of the magnitudes that entered each element), [N][heads][D] in 64 bits."""
    x = x.to(F64)
    half = inv_freq.numel()
    angle = positions.to(F64)[:, None] * inv_freq.to(F64)[None, :]
    c, s = (torch.cos(angle) * mscale)[:, None], (torch.sin(angle) * mscale)[:, None]
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., first], x[..., second]
    out, mag = x.clone(), torch.zeros_like(x)
    out[..., first], out[..., second] = a * c - b * s, a * s + b * c
    mag[..., first] = mag[..., second] = (a.abs() + b.abs()) * abs(mscale)
    return out, mag


def attention(q, k_cache, v_cache, table, q_start, kv_lens, scale, every=1):
    """64-bit attention of every row (or of each request's first, last and every `every`-th row:
    the others' error is unbounded) over the keys it sees only. Returns out, lse, and for
    each out element the bound of its error before the output's own rounding."""
    N, Hq, D = q.shape
    P, Hkv = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    out = torch.zeros(N, Hq, D, dtype=F64, device=q.device)
    lse = torch.full((N, Hq), -math.inf, dtype=F64, device=q.device)
    slack = torch.zeros_like(out)
    lse_slack = torch.zeros_like(lse)
    unit = UNIT[q.dtype]
    starts, lens = q_start.tolist(), kv_lens.tolist()
    for b, kv in enumerate(lens):
        n0, n1 = starts[b], starts[b + 1]
        if n1 <= n0 or kv <= 0:
            continue
        at = torch.arange(kv, device=q.device)
        pages = table[b].long()[at // P]
        k = k_cache[pages, at % P].to(F64)
        v = v_cache[pages, at % P].to(F64)
        for n in range(n0, n1):
            if (n - n0) % every and n + 1 < n1:
                slack[n] = lse_slack[n] = math.inf
                lse[n] = 0.0
                continue
            seen = kv - (n1 - n0) + (n - n0) + 1
            if seen <= 0:
                continue
            kk = k[:seen].permute(1, 2, 0).repeat_interleave(G, dim=0)  # [Hq, D, seen]
            vv = v[:seen].permute(1, 0, 2).repeat_interleave(G, dim=0)  # [Hq, seen, D]
            row = q[n].to(F64)[:, None]
            s = (row @ kk).squeeze(1) * scale
            size = (row.abs() @ kk.abs()).squeeze(1) * scale
            top = s.amax(dim=1, keepdim=True)
            p = torch.exp(s - top)
            total = p.sum(dim=1, keepdim=True)
            out[n] = (p[:, None] @ vv).squeeze(1) / total
            lse[n] = (top + torch.log(total)).squeeze(1)
            # products of 16-bit values are exact; D of them added in fp32, at worst truncating each of
            # D/16 + 16 additions: 2^-18 of the sum of magnitudes for D <= 128. The logarithm's base
            # change and the exponential add 2^-21 of the score's size. A score off by d changes a
            # weight by d, and the sum of weights by at most as much.
            d = (2.0 ** -18 * size + 2.0 ** -21 * (s.abs() + top.abs())).amax(dim=1)
            mean_abs = (p[:, None] @ vv.abs()).squeeze(1) / total
            slack[n] = mean_abs * (unit + 2.0 * d[:, None] + 2.0 ** -17)  # weights rounded to the type
            lse_slack[n] = d + 2.0 ** -17 + 2.0 ** -22 * lse[n].abs()
    return out, lse, slack, lse_slack
