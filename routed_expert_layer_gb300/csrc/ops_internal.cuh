// Helpers shared by the operators beside the expert layer (ops.cu, attn.cu, tree.cu, matmul8.cu): 16-bit types,
// host-side checks, launches.
#pragma once

#include <cuda.h>

#include <cmath>
#include <new>

#include "../../include/moe_ops_gb300.h"
#include "moe_internal.cuh"

namespace moe {

constexpr uint32_t kErrPlan = MOE_OPS_ERR_PLAN;
constexpr uint32_t kErrIndex = MOE_OPS_ERR_INDEX;

// One 16-bit value, and two in a 32-bit word (low half first), to and from fp32.
template <int DT>
__device__ __forceinline__ float to_f32(uint16_t v) {
  if constexpr (DT == MOE_DT_BF16) return __uint_as_float((uint32_t)v << 16);
  return __half2float(__ushort_as_half(v));
}
template <int DT>
__device__ __forceinline__ uint16_t from_f32(float v) {
  if constexpr (DT == MOE_DT_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (DT == MOE_DT_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == MOE_DT_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two fp32 to e4m3, rounded to nearest even, beyond 448 saturated (low byte first).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// |v| as an unsigned integer: its order is that of the magnitudes, and a NaN is the largest.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

inline bool is_aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }

// Byte range a strided tensor of 16-bit elements spans: [n1][n2][n3], innermost contiguous.
struct Span {
  const char* lo;
  const char* hi;
};
inline Span span16(const void* p, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t n3) {
  const char* b = (const char*)p;
  return {b, b + 2 * ((n1 - 1) * s1 + (n2 - 1) * s2 + n3)};
}
inline bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) cudaSetDevice(dev);
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

constexpr int kMaxDevices = 64;
inline int current_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices ? dev : 0;
}

// SMs of the current device (a constant of the device, read once for each).
inline int sm_count() {
  static int known[kMaxDevices];
  const int dev = current_device();
  if (!known[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
    known[dev] = n;
  }
  return known[dev];
}

inline int shift_of(int p) {
  int s = 0;
  while ((1 << s) < p) ++s;
  return s;
}

// The driver's tensor-map encoder (host-only, so it may run during stream capture), or null.
typedef CUresult (*TensorMapFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline TensorMapFn tensor_map_fn() {
  static const TensorMapFn encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<TensorMapFn>(fn);
  }();
  return encode;
}

// Words of an output or input of a call, for finding outputs that share memory with another tensor of it.
struct Words {
  const void* p;
  int64_t n;
};
// Whether one of the first `outputs` tensors shares a word with another tensor.
inline bool shares_words(const Words* t, int outputs, int count) {
  for (int o = 0; o < outputs; ++o)
    for (int i = o + 1; i < count; ++i) {
      const uintptr_t x = (uintptr_t)t[o].p, y = (uintptr_t)t[i].p;
      if (x < y + 4 * t[i].n && y < x + 4 * t[o].n && t[o].n && t[i].n) return true;
    }
  return false;
}

// Programmatic dependent launch for the launches of one operator call.
struct OpsPdl {
  OpsPdl() { g_launch_pdl = true; }
  ~OpsPdl() { g_launch_pdl = false; }
};

}  // namespace moe
