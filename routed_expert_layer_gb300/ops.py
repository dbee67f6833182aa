"""The operators beside the expert layer (``include/moe_ops_gb300.h``): the residual norm, a
serving step's plan, rotary positions with the cache append, paged attention, drafted trees
(plan, attention by masks, acceptance) and 8-bit projections (quantisation, product). Outputs are
allocated by the caller, and calls run on the current stream unless one is given. A wrong
shape, type or device raises ValueError before anything is enqueued (``csrc/binding.cpp``
checks and calls); what the library refuses raises MoeError.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os

import torch

from . import BINDING_PATH, MOE_ERR_DEVICE_FLAG, MOE_OK, _check, lib


def _load_binding():
    """The compiled binding. Raises if it has not been built (no fallback)."""
    lib()  # the C library first: the binding resolves its entry points in it
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"binding not built: {BINDING_PATH} (run __graft_entry__.build())")
    loader = importlib.machinery.ExtensionFileLoader("_ops_binding", BINDING_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_ops_binding", loader))
    loader.exec_module(module)
    return module


_binding = _load_binding()
_norm, _plan, _rotary, _attention = _binding.norm, _binding.plan, _binding.rotary, _binding.attention
_tree_plan, _tree_accept, _quantize8, _matmul8 = _binding.tree_plan, _binding.tree_accept, _binding.quantize8, _binding.matmul8


def add_rmsnorm(x, weight, eps: float, out=None, residual=None, residual_out=None, out8=None, scales=None,
                group: int = 0, err=None, stream=None) -> None:
    """t = x + residual; residual_out = t; out = y = t / sqrt(mean(t^2) + eps) * weight;
    out8 = e4m3(y / scale) with scales[row] (group 0) or scales[row][block of 128] (group 128).

    x, residual, out, residual_out: bf16 or f16 [T][H] (rows may be strided); weight: [H] of
    that type or float32; out8: float8_e4m3fn or uint8 [T][H]; scales: float32, contiguous,
    [T][blocks]. residual_out may be residual (in place), out may be x."""
    st = _norm(x, weight, eps, out, residual, residual_out, out8, scales, group, err, stream)
    if st:
        _check(st, "moe_add_rmsnorm")


def paged_plan(ctx_lens, new_lens, block_table, free_pages, free_head, page_size: int, *, q_start, kv_lens, positions,
               slots, free_head_out, err=None, stream=None) -> None:
    """Plan one serving step on the device (moe_paged_plan): from ctx_lens and new_lens [B]
    the new pages (entered into block_table [B][W], taken from free_pages [F] at free_head
    [1]), q_start [B+1], kv_lens [B], positions and slots [N], and the new free_head_out [1].
    All int32. N may exceed the new tokens: the rest gets position 0 and slot -1. No output may share
    memory with an input or another output (kv_lens is not ctx_lens, free_head_out not free_head)."""
    st = _plan(ctx_lens, new_lens, block_table, free_pages, free_head, page_size, q_start, kv_lens, positions, slots,
               free_head_out, err, stream)
    if st:
        _check(st, "moe_paged_plan")


def rope_frequencies(rot: int, base: float = 10000.0, linear: float = 1.0, blend: tuple | None = None, device="cuda"):
    """Radians per position of each rotary pair (float64 [rot/2]) for rotary_append:
    base^(-2i/rot), divided by `linear` (positions interpolated), or with
    blend = (factor, trained, slow, fast) scaled by parts for a context `factor` times the
    `trained` length: pairs that turn more than `fast` times over the trained length are kept,
    those that turn fewer than `slow` times are divided by factor, those between are blended
    linearly in the number of turns. (The magnitude factor that goes with blended scaling,
    0.1 ln(factor) + 1, is rotary_append's mscale.)"""
    if rot < 2 or rot % 2:
        raise ValueError("rope_frequencies: rot must be even and positive")
    if not (base > 0.0 and linear > 0.0):
        raise ValueError("rope_frequencies: base and linear must be positive")
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot) / linear
    if blend is not None:
        factor, trained, slow, fast = blend
        if not (factor > 0.0 and trained > 0.0 and slow < fast):
            raise ValueError("rope_frequencies: blend is (factor, trained, slow, fast), positive and slow below fast")
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f.to(device)


def rotary_append(q, k, v, positions, slots, inv_freq, k_cache, v_cache, q_out=None, interleaved: bool = False,
                  mscale: float = 1.0, err=None, stream=None) -> None:
    """Rotate q [N][Hq][D] (into q_out, or in place) and k [N][Hkv][D], and append k and v to
    the paged caches [pages][P][Hkv][D] (any strides, D contiguous) at slots int32 [N]
    (-1: not appended); positions int32 [N]; inv_freq float64 [rot/2], rot <= D."""
    st = _rotary(q, k, v, positions, slots, inv_freq, k_cache, v_cache, q_out, interleaved, mscale, err, stream)
    if st:
        _check(st, "moe_rotary_append")


def tree_plan(parents, q_start, ctx_lens, *, positions, mask, err=None, stream=None) -> None:
    """Positions and masks of drafted trees (moe_tree_plan): from parents int32 [N] (a node's parent as its place in the
    request, -1 behind the cached tokens), q_start [B+1] and ctx_lens [B], positions int32 [N] (context plus depth) and
    mask int32 [N][words], bit j set where the node sees node j: its ancestors and itself. A request with more than
    32 * words new tokens has to be a chain and keeps its mask rows as they are."""
    st = _tree_plan(parents, q_start, ctx_lens, positions, mask, err, stream)
    if st:
        _check(st, "moe_tree_plan")


def tree_accept(parents, tokens, targets, q_start, ctx_lens, block_table, k_cache, v_cache, *, path, accepted, ctx_out,
                next_tokens, certain=None, err=None, stream=None) -> None:
    """The drafted tokens that the model confirms, and their keys and values moved behind the cached ones
    (moe_tree_accept): from each request's root (or its certain[b] first tokens) on, the child whose token is the
    model's target for the node, the lowest if several. parents, tokens, targets int32 [N]; caches [pages][P][Hkv][D] or
    [layers][pages][P][Hkv][D], 16-bit, any strides, D contiguous; path int32 [B][depth] (places of the drafted nodes
    taken, then -1), accepted, ctx_out (ctx_lens + accepted) and next_tokens int32 [B]; certain int32 [B] or None
    (one). No output shares memory with an input."""
    st = _tree_accept(parents, tokens, targets, q_start, ctx_lens, block_table, k_cache, v_cache, path, accepted, ctx_out,
                      next_tokens, certain, err, stream)
    if st:
        _check(st, "moe_tree_accept")


def quantize8(x, out8, scales, group: int = 128, rows: int = 1, stream=None) -> None:
    """out8 = e4m3(x / scale), scale = max|x| / 448 (moe_quantize8) over 128 elements of a row (group 128: scales
    [T][ceil(H/128)]), over a row (group 0: [T][1]) or, rows = 128, over blocks of 128 x 128
    ([ceil(T/128)][ceil(H/128)], as Matmul8 takes weights). x bf16 or f16 [T][H], out8 float8_e4m3fn or uint8 (rows of
    both may be strided), scales float32, contiguous."""
    st = _quantize8(x, out8, scales, group, rows, stream)
    if st:
        _check(st, "moe_quantize8")


class Matmul8:
    """Products of e4m3 activations and weights with block scales on one GPU (wraps a moe_matmul8_ctx: workspace and
    device error word). One host thread and one stream use a handle at a time."""

    def __init__(self, device: int = 0):
        self.device = device
        self.ctx = ctypes.c_void_p()
        _check(lib().moe_matmul8_create(device, ctypes.byref(self.ctx)), "moe_matmul8_create")

    def forward(self, a8, a_scales, w8, w_scales, out, stream=None) -> None:
        """out[t][n] = sum over blocks of 128 of a_scales[t][b] w_scales[n / 128][b] (a8 w8^T of the block)
        (moe_matmul8_forward; the product of the two scales is formed first, in fp32). a8 [T][K], w8 [N][K]:
        float8_e4m3fn or uint8, K a multiple of 16; a_scales float32 [T][ceil(K/128)] or [T][1]; w_scales float32
        [ceil(N/128)][ceil(K/128)]; out bf16 or f16 [T][N]. Rows may be strided (a8 and w8: by multiples of 16, from 16-byte aligned addresses)."""
        if not self.ctx:
            raise ValueError("the handle is closed")
        st = _matmul8(self.ctx.value, self.device, a8, a_scales, w8, w_scales, out, stream)
        if st:
            _check(st, "moe_matmul8_forward")

    def get_error(self) -> int:
        bits = ctypes.c_uint32(0)
        st = lib().moe_matmul8_get_error(self.ctx, ctypes.byref(bits))
        if st not in (MOE_OK, MOE_ERR_DEVICE_FLAG):
            _check(st, "moe_matmul8_get_error")
        return bits.value

    def device_bytes(self) -> int:
        return lib().moe_matmul8_device_bytes(self.ctx)

    def close(self) -> None:
        if self.ctx:
            lib().moe_matmul8_destroy(self.ctx)
            self.ctx = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedAttention:
    """Attention over a paged cache on one GPU (wraps a moe_attn_ctx: workspace and device
    error word). One host thread and one stream use a handle at a time."""

    def __init__(self, device: int = 0):
        self.device = device
        self.ctx = ctypes.c_void_p()
        _check(lib().moe_attn_create(device, ctypes.byref(self.ctx)), "moe_attn_create")

    def forward(self, q, k_cache, v_cache, block_table, q_start, kv_lens, out, scale: float, lse=None,
                max_new: int = 0, stream=None, tree=None) -> None:
        """out[n] = attention of q[n] over its request's keys up to its own position
        (moe_attn_forward), or with tree int32 [N][words] (tree_plan's mask) over the cached keys and those new
        tokens whose bits are set (moe_attn_forward_tree; a request with more than 32 * words new tokens is a
        plain chunk; tree shares no memory with out or lse). q, out [N][Hq][D]; caches [pages][P][Hkv][D] (any
        strides, D contiguous); block_table int32 [B][W], q_start int32 [B+1], kv_lens int32 [B]; lse
        float32 [N][Hq], contiguous, or None; max_new: the most new tokens of a request, if
        known (picks a variant)."""
        if not self.ctx:
            raise ValueError("the handle is closed")
        st = _attention(self.ctx.value, self.device, q, k_cache, v_cache, block_table, q_start, kv_lens, out, scale, lse,
                        max_new, stream, tree)
        if st:
            _check(st, "moe_attn_forward" if tree is None else "moe_attn_forward_tree")

    def get_error(self) -> int:
        bits = ctypes.c_uint32(0)
        st = lib().moe_attn_get_error(self.ctx, ctypes.byref(bits))
        if st not in (MOE_OK, MOE_ERR_DEVICE_FLAG):
            _check(st, "moe_attn_get_error")
        return bits.value

    def device_bytes(self) -> int:
        return lib().moe_attn_device_bytes(self.ctx)

    def close(self) -> None:
        if self.ctx:
            lib().moe_attn_destroy(self.ctx)
            self.ctx = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
