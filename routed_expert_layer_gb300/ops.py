"""The operators beside the expert layer (``include/moe_ops_gb300.h``): the residual norm, a
serving step's plan, rotary positions with the cache append, and paged attention. Outputs are
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


class PagedAttention:
    """Attention over a paged cache on one GPU (wraps a moe_attn_ctx: workspace and device
    error word). One host thread and one stream use a handle at a time."""

    def __init__(self, device: int = 0):
        self.device = device
        self.ctx = ctypes.c_void_p()
        _check(lib().moe_attn_create(device, ctypes.byref(self.ctx)), "moe_attn_create")

    def forward(self, q, k_cache, v_cache, block_table, q_start, kv_lens, out, scale: float, lse=None,
                max_new: int = 0, stream=None) -> None:
        """out[n] = attention of q[n] over its request's keys up to its own position
        (moe_attn_forward). q, out [N][Hq][D]; caches [pages][P][Hkv][D] (any strides, D
        contiguous); block_table int32 [B][W], q_start int32 [B+1], kv_lens int32 [B]; lse
        float32 [N][Hq], contiguous, or None; max_new: the most new tokens of a request, if
        known (picks a variant)."""
        if not self.ctx:
            raise ValueError("the handle is closed")
        st = _attention(self.ctx.value, self.device, q, k_cache, v_cache, block_table, q_start, kv_lens, out, scale, lse,
                        max_new, stream)
        if st:
            _check(st, "moe_attn_forward")

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
