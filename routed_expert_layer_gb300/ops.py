"""Binding of the operators beside the expert layer (``include/moe_ops_gb300.h``): the
residual norm, a serving step's plan, rotary positions with the cache append, and paged
attention. Argument marshalling and checks only; outputs are allocated by the caller, and
calls run on the current stream unless one is given. A wrong shape, type or device raises
ValueError before anything is enqueued; what the library refuses raises MoeError.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import MOE_DT_BF16, MOE_DT_F16, MOE_ERR_DEVICE_FLAG, MOE_OK, _check, lib

_DT = {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16}
# the argument structs, field for field as in the header (native sizes and alignment)
_NORM = struct.Struct("@8P5q5if").pack
_PLAN = struct.Struct("@11Pq5i").pack
_ROTARY = struct.Struct("@10P14q9if").pack
_ATTN = struct.Struct("@8P11q10if").pack
# torch.cuda.current_stream and current_device build objects and check initialisation on every call: 1.3 us
# of a call that takes 7; these are the functions under them, where this torch has them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_I32, _F32, _F64 = torch.int32, torch.float32, torch.float64


def _on(stream, dev: int) -> int:
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _device(x, what: str) -> int:
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{what}: expected a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{what}: expected a tensor on the current device, got cuda:{dev}")
    return dev


def _expect(name: str, t, shape: tuple, dtype, dev: int):
    """Check shape, type and device; the innermost dimension is contiguous. Returns the strides."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name}: expected {dtype} {list(shape)} on cuda:{dev}, got {t.dtype} {list(t.shape)} on "
                         f"{t.device}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: expected a contiguous innermost dimension")
    return st


def _ints(name: str, t, n: int, dev: int) -> int:
    """Check a contiguous int32 [n] tensor; returns its address."""
    if t.dtype is not _I32 or t.dim() != 1 or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous torch.int32 [{n}] on cuda:{dev}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    return t.data_ptr()


def _err(err, dev: int) -> int:
    if err is None:
        return 0
    if err.numel() != 1 or err.element_size() != 4 or err.get_device() != dev:
        raise ValueError("err: expected one 4-byte word on the device")
    return err.data_ptr()


def add_rmsnorm(x, weight, eps: float, out=None, residual=None, residual_out=None, out8=None, scales=None,
                group: int = 0, err=None, stream=None) -> None:
    """t = x + residual; residual_out = t; out = y = t / sqrt(mean(t^2) + eps) * weight;
    out8 = e4m3(y / scale) with scales[row] (group 0) or scales[row][block of 128] (group 128).

    x, residual, out, residual_out: bf16 or f16 [T][H] (rows may be strided); weight: [H] of
    that type or float32; out8: float8_e4m3fn or uint8 [T][H]; scales: float32, contiguous,
    [T][blocks]. residual_out may be residual (in place), out may be x."""
    dev = _device(x, "x")
    dt = _DT.get(x.dtype)
    if dt is None or x.dim() != 2:
        raise ValueError(f"x: expected bf16 or f16 [T][H], got {x.dtype} {list(x.shape)}")
    shape = x.shape
    T, H = shape
    xs = _expect("x", x, shape, x.dtype, dev)[0]
    w32 = weight.dtype is _F32
    _expect("weight", weight, (H,), _F32 if w32 else x.dtype, dev)
    rp = rs = op = os = rop = ros = o8p = o8s = sp = 0
    if residual is not None:
        rs = _expect("residual", residual, shape, x.dtype, dev)[0]
        rp = residual.data_ptr()
    if out is not None:
        os = _expect("out", out, shape, x.dtype, dev)[0]
        op = out.data_ptr()
    if residual_out is not None:
        ros = _expect("residual_out", residual_out, shape, x.dtype, dev)[0]
        rop = residual_out.data_ptr()
    if out8 is not None:
        if out8.element_size() != 1:
            raise ValueError(f"out8: expected float8_e4m3fn or uint8, got {out8.dtype}")
        o8s = _expect("out8", out8, shape, out8.dtype, dev)[0]
        o8p = out8.data_ptr()
        if scales is None:
            raise ValueError("scales: out8 needs scales")
        _expect("scales", scales, (T, -(-H // group) if group else 1), _F32, dev)
        if not scales.is_contiguous():
            raise ValueError("scales: expected a contiguous tensor")
        sp = scales.data_ptr()
    if T <= 1:  # one row has no row stride
        xs = rs = os = ros = o8s = H
    st = lib().moe_add_rmsnorm(_on(stream, dev), _NORM(x.data_ptr(), rp, weight.data_ptr(), op, rop, o8p, sp,
                                                       0 if err is None else _err(err, dev), xs, rs,
                                                       os, ros, o8s, T, H, dt, w32, group, eps))
    if st:
        _check(st, "moe_add_rmsnorm")


def paged_plan(ctx_lens, new_lens, block_table, free_pages, free_head, page_size: int, *, q_start, kv_lens, positions,
               slots, free_head_out, err=None, stream=None) -> None:
    """Plan one serving step on the device (moe_paged_plan): from ctx_lens and new_lens [B]
    the new pages (entered into block_table [B][W], taken from free_pages [F] at free_head
    [1]), q_start [B+1], kv_lens [B], positions and slots [N], and the new free_head_out [1].
    All int32. N may exceed the new tokens: the rest gets position 0 and slot -1."""
    dev = _device(ctx_lens, "ctx_lens")
    B = ctx_lens.numel()
    if block_table.dim() != 2:
        raise ValueError("block_table: expected [B][W]")
    W = block_table.shape[1]
    ts = _expect("block_table", block_table, (B, W), _I32, dev)[0] if B > 1 else W
    F, N = free_pages.numel(), positions.numel()
    st = lib().moe_paged_plan(_on(stream, dev), _PLAN(
        _ints("ctx_lens", ctx_lens, B, dev), _ints("new_lens", new_lens, B, dev), block_table.data_ptr(),
        _ints("free_pages", free_pages, F, dev), _ints("free_head", free_head, 1, dev),
        _ints("q_start", q_start, B + 1, dev), _ints("kv_lens", kv_lens, B, dev),
        _ints("positions", positions, N, dev), _ints("slots", slots, N, dev),
        _ints("free_head_out", free_head_out, 1, dev), _err(err, dev), ts, B, W, F, N, page_size))
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
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=_F64) / rot) / linear
    if blend is not None:
        factor, trained, slow, fast = blend
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f.to(device)


def _cache(name: str, t, dtype, dev: int):
    if t.dim() != 4:
        raise ValueError(f"{name}: expected [pages][page_size][heads][D]")
    return _expect(name, t, t.shape, dtype, dev)


def rotary_append(q, k, v, positions, slots, inv_freq, k_cache, v_cache, q_out=None, interleaved: bool = False,
                  mscale: float = 1.0, err=None, stream=None) -> None:
    """Rotate q [N][Hq][D] (into q_out, or in place) and k [N][Hkv][D], and append k and v to
    the paged caches [pages][P][Hkv][D] (any strides, D contiguous) at slots int32 [N]
    (-1: not appended); positions int32 [N]; inv_freq float64 [rot/2], rot <= D."""
    dev = _device(q, "q")
    dtype = q.dtype
    dt = _DT.get(dtype)
    if dt is None or q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"q, k: expected bf16 or f16 [N][heads][D], got {dtype} {list(q.shape)}, {list(k.shape)}")
    N, Hq, D = q.shape
    Hkv = k.shape[1]
    if q_out is None:
        q_out = q
    qs = _expect("q", q, q.shape, dtype, dev)
    ks = _expect("k", k, (N, Hkv, D), dtype, dev)
    vs = _expect("v", v, (N, Hkv, D), dtype, dev)
    os = _expect("q_out", q_out, q.shape, dtype, dev)
    kc = _cache("k_cache", k_cache, dtype, dev)
    vc = _cache("v_cache", v_cache, dtype, dev)
    pages, P, ch, cd = k_cache.shape
    if ch != Hkv or cd != D or v_cache.shape != k_cache.shape:
        raise ValueError(f"k_cache, v_cache: expected [pages][P][{Hkv}][{D}], got {list(k_cache.shape)}, "
                         f"{list(v_cache.shape)}")
    half = inv_freq.numel()
    _expect("inv_freq", inv_freq, (half,), _F64, dev)
    st = lib().moe_rotary_append(_on(stream, dev), _ROTARY(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        _ints("positions", positions, N, dev), _ints("slots", slots, N, dev), inv_freq.data_ptr(), _err(err, dev),
        qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], os[0], os[1], kc[0], kc[1], kc[2], vc[0], vc[1], vc[2],
        N, Hq, Hkv, D, 2 * half, P, pages, interleaved, dt, mscale))
    if st:
        _check(st, "moe_rotary_append")


class PagedAttention:
    """Attention over a paged cache on one GPU (wraps a moe_attn_ctx: workspace and device
    error word). One host thread and one stream use a handle at a time."""

    def __init__(self, device: int = 0):
        self.device = device
        self.ctx = ctypes.c_void_p()
        _check(lib().moe_attn_create(device, ctypes.byref(self.ctx)), "moe_attn_create")
        self._forward = lib().moe_attn_forward

    def forward(self, q, k_cache, v_cache, block_table, q_start, kv_lens, out, scale: float, lse=None,
                max_new: int = 0, stream=None) -> None:
        """out[n] = attention of q[n] over its request's keys up to its own position
        (moe_attn_forward). q, out [N][Hq][D]; caches [pages][P][Hkv][D] (any strides, D
        contiguous); block_table int32 [B][W], q_start int32 [B+1], kv_lens int32 [B]; lse
        float32 [N][Hq], contiguous, or None; max_new: the most new tokens of a request, if
        known (picks a variant)."""
        dev = self.device
        dtype = q.dtype
        dt = _DT.get(dtype)
        if dt is None or q.dim() != 3:
            raise ValueError(f"q: expected bf16 or f16 [N][Hq][D], got {dtype} {list(q.shape)}")
        shape = q.shape
        N, Hq, D = shape
        qs = _expect("q", q, shape, dtype, dev)
        os = _expect("out", out, shape, dtype, dev)
        kc = _cache("k_cache", k_cache, dtype, dev)
        vc = _cache("v_cache", v_cache, dtype, dev)
        pages, P, Hkv, cd = k_cache.shape
        if cd != D or v_cache.shape != k_cache.shape:
            raise ValueError(f"k_cache, v_cache: expected [pages][P][Hkv][{D}], got {list(k_cache.shape)}, "
                             f"{list(v_cache.shape)}")
        B = kv_lens.numel()
        if block_table.dim() != 2:
            raise ValueError("block_table: expected [B][W]")
        W = block_table.shape[1]
        ts = _expect("block_table", block_table, (B, W), _I32, dev)[0]
        if B == 1:
            ts = W
        lp = 0
        if lse is not None:
            _expect("lse", lse, (N, Hq), _F32, dev)
            if not lse.is_contiguous():
                raise ValueError("lse: expected a contiguous tensor")
            lp = lse.data_ptr()
        st = self._forward(self.ctx, _on(stream, dev), _ATTN(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), lp, block_table.data_ptr(),
            _ints("q_start", q_start, B + 1, dev), _ints("kv_lens", kv_lens, B, dev),
            qs[0], qs[1], os[0], os[1], kc[0], kc[1], kc[2], vc[0], vc[1], vc[2], ts,
            N, B, Hq, Hkv, D, P, pages, W, max_new, dt, scale))
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
