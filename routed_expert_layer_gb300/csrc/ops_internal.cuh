// Helpers shared by the operators beside the expert layer (ops.cu, attn.cu): 16-bit types,
// host-side checks, launches.
#pragma once

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

// Programmatic dependent launch for the launches of one operator call.
struct OpsPdl {
  OpsPdl() { g_launch_pdl = true; }
  ~OpsPdl() { g_launch_pdl = false; }
};

}  // namespace moe
