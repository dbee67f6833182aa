// Operators beside the expert layer whose work is moving data: the residual norm, a serving
// step's plan, rotary positions with the cache append. Interfaces and formulas:
// include/moe_ops_gb300.h.
#include <algorithm>
#include <type_traits>

#include "ops_internal.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

// ---- residual addition + root-mean-square norm + 8-bit output ---------------------------------

struct NormParams {
  const uint16_t* x;
  const uint16_t* residual;
  const void* weight;
  uint16_t* out;
  uint16_t* residual_out;
  uint8_t* out8;
  float* scales;
  int64_t x_stride, residual_stride, out_stride, residual_out_stride, out8_stride;
  int T, H, weight_f32, group, n_blocks;
  float eps;
  uint32_t* err;
};

// A piece of 8, 4, 2 or 1 elements as it lies in memory.
template <int N>
using Piece = std::conditional_t<N == 8, uint4, std::conditional_t<N == 4, uint2, std::conditional_t<N == 2, uint32_t, uint16_t>>>;

template <int DT, int N>
__device__ __forceinline__ void unpack(const Piece<N>& w, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = to_f32<DT>(w);
  } else {
    uint32_t u[N / 2];
    if constexpr (N == 2) u[0] = w;
    else u[0] = w.x, u[1] = w.y;
    if constexpr (N == 8) u[2] = w.z, u[3] = w.w;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 f = unpack2<DT>(u[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

template <int DT, int N>
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&v)[N]) {
  if constexpr (N == 1) {
    *p = from_f32<DT>(v[0]);
  } else {
    Piece<N> w;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) reinterpret_cast<uint32_t*>(&w)[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<Piece<N>*>(p) = w;
  }
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// |v| as an unsigned integer: its order is that of the magnitudes, and a NaN is the largest.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The 8-bit output is y / s as y * (1 / s). Where s lies below fp32's normal range, 1 / s lies above its largest
// value: there both y and s are taken kLift times larger first.
constexpr float kLift = 0x1p64f;
__device__ __forceinline__ bool needs_lift(float s) { return s > 0.f && s < 0x1p-126f; }

// Reductions over the warps of one row (block row threadIdx.y); red has one word per warp.
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  float* r = red + threadIdx.y * nw;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < nw; ++i) v += r[i];
  return v;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  uint32_t* r = red + threadIdx.y * nw;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < nw; ++i) v = max(v, r[i]);
  return v;
}

// Three kernels, chosen by width and alignment. All read every input once: a thread holds its chunks of
// the row in registers between the sum of squares and the outputs. 8 or 9 bytes an element against
// some 10 operations: bound by memory.
//
// norm_staged_kernel (1024 < H <= 14336, 16-byte chunks): blocks stay and walk over the rows, the next
// rows' bytes come by bulk copies into two stages of shared memory, so the reduction's latency is
// not added to memory's, and the weights are loaded once per block. At T = 8192, H = 7168, bf16 with
// residual and 8-bit blocks: 87 us, 6.1 TB/s. Measured on the way: one row per block and register
// loads with 1, 2, 4, 8 chunks per thread 125, 114, 105, 117 us; walking with the next row's loads in
// registers 95 us; two blocks per SM with 2, 3, 4 stages 86.1, 87.1, 87.5 us, one block with six 111 us,
// three blocks of 224 threads 97 us. Single rows too: T = 1 2.4 us a launch in a graph (register loads 2.9). The limit is
// 896 threads of two pieces; T = 4096, H = 14336 without, with a row's and with blocks' 8-bit outputs: 81, 85, 82 us,
// norm_any_kernel in pairs 78, 99, 112. 1,024 threads would reach 16384, and are not built.
// norm_rows_kernel (H <= 1024, 16-byte chunks): several rows per block, one chunk per thread, the next
// rows' loads issued before this one's reduction; staging rows this short would cost a copy each. Both at
// T = 8192: H = 128 4.6 us (staged 6.3), 512 7.7 (8.4), 1024 13.4 (13.1); T = 1, H = 512 1.9 us (2.6).
// norm_any_kernel (chunks of 2 or 1 elements): what is wider than 14336, or whose width, stride or alignment is
// not a multiple of 8. T = 8192: H = 7170 bf16 with residual 78 us, 7169 with 8-bit blocks 212 us, bound by
// the number of its 1- and 2-byte accesses. Where all three can run, in elements, pairs and by the kernels above:
// H = 7168 200, 105, 87 us, H = 1024 23.2, 23.6, 13.3, T = 1 of 7168 5.6, 4.7, 3.3. Elements of rows wider than 16384
// (32 per thread of 1,024) are the one instance whose values do not fit its registers: some 500 bytes spill.

__device__ __forceinline__ uint4 load16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// The 8-bit output and scales of a row whose chunks are in t (|t| up to mx in this thread), by the whole block.
template <int NV>
__device__ __forceinline__ void write_8bit(const NormParams& p, int64_t row, bool live, float (&t)[NV][8],
                                           uint32_t mx, uint32_t* red) {
  const int tx = threadIdx.x, TX = blockDim.x, H = p.H;
  if (p.group == 0) {
    mx = row_max(mx, red);
    if (live && tx == 0) p.scales[row] = __uint_as_float(mx) / 448.f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (tx + i * TX) * 8;
    uint32_t m = mx;
    if (p.group) {  // 16 consecutive threads hold one block of 128 (threads past the row hold zeros)
      m = 0;
      if (e < H)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(t[i][j]));
#pragma unroll
      for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      if (live && e < H && (tx & 15) == 0) p.scales[row * p.n_blocks + (e >> 7)] = __uint_as_float(m) / 448.f;
    }
    if (!live || e >= H) continue;
    float s = __uint_as_float(m) / 448.f;
    if (needs_lift(s)) {
      s *= kLift;
#pragma unroll
      for (int j = 0; j < 8; ++j) t[i][j] *= kLift;
    }
    const float inv = s > 0.f ? 1.f / s : 1.f;  // zeros stay zeros; a NaN scale keeps its NaN values
    uint2 q;
    q.x = e4m3x2(t[i][0] * inv, t[i][1] * inv) | e4m3x2(t[i][2] * inv, t[i][3] * inv) << 16;
    q.y = e4m3x2(t[i][4] * inv, t[i][5] * inv) | e4m3x2(t[i][6] * inv, t[i][7] * inv) << 16;
    *reinterpret_cast<uint2*>(p.out8 + row * p.out8_stride + e) = q;
  }
}

template <int DT, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_rows_kernel(const NormParams p) {
  __shared__ float red_sum[2][32];
  __shared__ uint32_t red_max[2][32];
  pdl_entry();
  const int tx = threadIdx.x, TX = blockDim.x, H = p.H;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t first = (int64_t)blockIdx.x * blockDim.y;
  uint4 x[NV], r[NV], w[NV];
  const auto fetch = [&](int64_t at) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (tx + i * TX) * 8;
      if (at < p.T && e < H) {
        x[i] = *reinterpret_cast<const uint4*>(p.x + at * p.x_stride + e);
        if (p.residual) r[i] = *reinterpret_cast<const uint4*>(p.residual + at * p.residual_stride + e);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = r[i] = w[i] = make_uint4(0, 0, 0, 0);
  fetch(row);
  if (!p.weight_f32)
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((tx + i * TX) * 8 < H) w[i] = load16(reinterpret_cast<const uint16_t*>(p.weight) + (tx + i * TX) * 8);
  int turn = 0;
  for (int64_t r0 = first; r0 < p.T; r0 += step, row += step, turn ^= 1) {
    const bool live = row < p.T;
    float t[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (tx + i * TX) * 8;
      unpack<DT, 8>(x[i], t[i]);
      if (p.residual) {
        float a[8];
        unpack<DT, 8>(r[i], a);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[i][j] += a[j];
        if (p.residual_out && live && e < H) store_vec<DT, 8>(p.residual_out + row * p.residual_out_stride + e, t[i]);
      }
      if (live && e < H) {
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(t[i][j], t[i][j], ss);
      }
    }
    fetch(row + step);
    const float rs = rsqrtf(row_sum(ss, red_sum[turn]) / (float)H + p.eps);
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (tx + i * TX) * 8;
      float g[8];
      if (p.weight_f32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = e < H ? __ldg(reinterpret_cast<const float*>(p.weight) + e + j) : 0.f;
      } else {
        unpack<DT, 8>(w[i], g);
      }
      const bool in = live && e < H;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t[i][j] = in ? t[i][j] * rs * g[j] : 0.f;
        mx = max(mx, abs_bits(t[i][j]));
      }
      if (p.out && in) store_vec<DT, 8>(p.out + row * p.out_stride + e, t[i]);
    }
    if (p.out8) write_8bit<NV>(p, row, live, t, mx, red_max[turn]);
  }
}

constexpr int kNormStages = 2;

// One row per step, NV chunks per thread; thread 0 keeps the next rows' copies in flight. A stage is
// free for the next copy once the row's reduction has synchronised: every thread has read its part.
template <int DT, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_staged_kernel(const NormParams p) {
  extern __shared__ __align__(128) uint8_t staged[];  // [kNormStages][x row | residual row]
  __shared__ uint64_t full[kNormStages];
  __shared__ float red_sum[2][32];
  __shared__ uint32_t red_max[2][32];
  const int tx = threadIdx.x, H = p.H, TX = blockDim.x;
  const uint32_t row_bytes = (uint32_t)H * 2, stage_bytes = p.residual ? 2 * row_bytes : row_bytes;
  if (tx == 0) {
    for (int s = 0; s < kNormStages; ++s) ptx::mbar_init(&full[s], 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  pdl_entry();
  const auto copy = [&](int64_t row, int s) {
    uint8_t* d = staged + (size_t)s * stage_bytes;
    ptx::mbar_arrive_expect_tx(&full[s], stage_bytes);
    ptx::bulk_g2s(d, p.x + row * p.x_stride, row_bytes, &full[s]);
    if (p.residual) ptx::bulk_g2s(d + row_bytes, p.residual + row * p.residual_stride, row_bytes, &full[s]);
  };
  if (tx == 0)
    for (int s = 0; s < kNormStages; ++s) {
      const int64_t row = (int64_t)blockIdx.x + (int64_t)s * gridDim.x;
      if (row < p.T) copy(row, s);
    }
  uint4 w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i] = make_uint4(0, 0, 0, 0);
    const int e = (tx + i * TX) * 8;
    if (!p.weight_f32 && e < H) w[i] = load16(reinterpret_cast<const uint16_t*>(p.weight) + e);
  }
  uint32_t n = 0;
  bool ok = true;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, ++n) {
    const int s = n % kNormStages, turn = n & 1;
    ok = ptx::mbar_wait_quiet(&full[s], (n / kNormStages) & 1);
    const uint8_t* d = staged + (size_t)s * stage_bytes;
    float t[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tx + i * TX;
      const bool in = c * 8 < H;
      unpack<DT, 8>(in ? *reinterpret_cast<const uint4*>(d + c * 16) : make_uint4(0, 0, 0, 0), t[i]);
      if (p.residual && in) {
        float a[8];
        unpack<DT, 8>(*reinterpret_cast<const uint4*>(d + row_bytes + c * 16), a);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[i][j] += a[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(t[i][j], t[i][j], ss);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if ((tx & 31) == 0) red_sum[turn][tx >> 5] = ss;
    ok = __syncthreads_and(ok);
    if (!ok) break;  // a copy did not arrive within the limit
    if (tx == 0 && row + (int64_t)kNormStages * gridDim.x < p.T) copy(row + (int64_t)kNormStages * gridDim.x, s);
    ss = 0.f;
    for (int i = 0; i < TX >> 5; ++i) ss += red_sum[turn][i];
    const float rs = rsqrtf(ss / (float)H + p.eps);
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (tx + i * TX) * 8;
      if (e >= H) continue;
      if (p.residual_out) store_vec<DT, 8>(p.residual_out + row * p.residual_out_stride + e, t[i]);
      float g[8];
      if (p.weight_f32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = __ldg(reinterpret_cast<const float*>(p.weight) + e + j);
      } else {
        unpack<DT, 8>(w[i], g);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t[i][j] = t[i][j] * rs * g[j];
        mx = max(mx, abs_bits(t[i][j]));
      }
      if (p.out) store_vec<DT, 8>(p.out + row * p.out_stride + e, t[i]);
    }
    if (p.out8) write_8bit<NV>(p, row, true, t, mx, red_max[turn]);
  }
  if (!ok && tx == 0) {  // let the copies in flight land before the block's shared memory goes away
    if (p.err) atomicOr(p.err, ptx::kErrTimeout);
    for (uint32_t k = n; k < n + kNormStages; ++k)
      if ((int64_t)blockIdx.x + (int64_t)k * gridDim.x < p.T) ptx::mbar_wait_quiet(&full[k % kNormStages], (k / kNormStages) & 1);
  }
}

// The pieces of a row are VE elements, thread tx has pieces tx, tx + TX, ... (NV of them). TX is a constant, so a
// thread keeps one address per tensor, and no store stands between loads, which would wait for it.
template <int DT, int VE, int TX, int NV, int MINB>
__global__ void __launch_bounds__(TX < 256 ? 256 : TX, MINB) norm_any_kernel(const NormParams p) {
  __shared__ float red_sum[2][32];
  __shared__ uint32_t red_max[2][32];
  extern __shared__ uint32_t block_max[];  // with blocks of 128: [block rows][n_blocks] maxima, then 1 / scale
  pdl_entry();
  const int tx = threadIdx.x, n_pieces = p.H / VE;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const auto place = [&](int i) { return (tx + i * TX) * VE; };
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < p.T; r0 += step, turn ^= 1) {
    const bool live = r0 + threadIdx.y < p.T;
    const int64_t row = live ? r0 + threadIdx.y : p.T - 1;
    const int n = live ? n_pieces : 0;
    float t[NV][VE];
    {
      Piece<VE> a[NV];
      const uint16_t* x = p.x + row * p.x_stride;
#pragma unroll
      for (int i = 0; i < NV; ++i) a[i] = tx + i * TX < n ? *reinterpret_cast<const Piece<VE>*>(x + place(i)) : 0;
      if (p.residual) {
        Piece<VE> b[NV];
        const uint16_t* r = p.residual + row * p.residual_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) b[i] = tx + i * TX < n ? *reinterpret_cast<const Piece<VE>*>(r + place(i)) : 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float c[VE];
          unpack<DT, VE>(a[i], t[i]);
          unpack<DT, VE>(b[i], c);
#pragma unroll
          for (int j = 0; j < VE; ++j) t[i][j] += c[j];
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) unpack<DT, VE>(a[i], t[i]);
      }
    }
    if (p.residual_out) {
      uint16_t* o = p.residual_out + row * p.residual_out_stride;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (tx + i * TX < n) store_vec<DT, VE>(o + place(i), t[i]);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VE; ++j)
        ss = fmaf(t[i][j], t[i][j], ss);
    const float rs = rsqrtf(row_sum(ss, red_sum[turn]) / (float)p.H + p.eps);
    if (p.weight_f32) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VE; ++j)
          t[i][j] = t[i][j] * rs * (tx + i * TX < n ? __ldg(reinterpret_cast<const float*>(p.weight) + place(i) + j) : 0.f);
    } else {
      Piece<VE> a[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        a[i] = tx + i * TX < n ? *reinterpret_cast<const Piece<VE>*>(reinterpret_cast<const uint16_t*>(p.weight) + place(i)) : 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float c[VE];
        unpack<DT, VE>(a[i], c);
#pragma unroll
        for (int j = 0; j < VE; ++j) t[i][j] = t[i][j] * rs * c[j];
      }
    }
    if (p.out) {
      uint16_t* o = p.out + row * p.out_stride;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (tx + i * TX < n) store_vec<DT, VE>(o + place(i), t[i]);
    }
    if (!p.out8) continue;
    uint32_t* bm = block_max + threadIdx.y * p.n_blocks;
    float inv = 1.f;
    if (p.group == 0) {
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VE; ++j) mx = max(mx, tx + i * TX < n ? abs_bits(t[i][j]) : 0);
      const float s = __uint_as_float(row_max(mx, red_max[turn])) / 448.f;
      if (live && tx == 0) p.scales[row] = s;
      inv = s > 0.f ? 1.f / s : 1.f;  // zeros stay zeros; a NaN scale keeps its NaN values
      if (needs_lift(s)) {
        inv = 1.f / (s * kLift);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < VE; ++j) t[i][j] *= kLift;
      }
    } else {
      for (int b = tx; b < p.n_blocks; b += TX) bm[b] = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) {  // a warp's 32 pieces lie in one block of 128
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < VE; ++j) m = max(m, tx + i * TX < n ? abs_bits(t[i][j]) : 0);
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if ((tx & 31) == 0 && tx + i * TX < n) atomicMax(&bm[place(i) >> 7], m);
      }
      __syncthreads();
      for (int b = tx; b < p.n_blocks; b += TX) {
        const float s = __uint_as_float(bm[b]) / 448.f;
        if (live) p.scales[row * p.n_blocks + b] = s;
        // negative: the block's values are lifted
        bm[b] = __float_as_uint(needs_lift(s) ? -1.f / (s * kLift) : s > 0.f ? 1.f / s : 1.f);
      }
      __syncthreads();
    }
    uint8_t* o8 = p.out8 + row * p.out8_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (tx + i * TX >= n) continue;
      float k = inv;
      if (p.group) {
        k = __uint_as_float(bm[place(i) >> 7]);
        if (k < 0.f)
#pragma unroll
          for (int j = 0; j < VE; ++j) t[i][j] *= -kLift;
      }
      if constexpr (VE == 1) o8[place(i)] = (uint8_t)e4m3x2(t[i][0] * k, 0.f);
      else *reinterpret_cast<uint16_t*>(o8 + place(i)) = (uint16_t)e4m3x2(t[i][0] * k, t[i][1] * k);
    }
    if (p.group) __syncthreads();  // the next row's maxima take this one's place
  }
}

constexpr int kMaxDevices = 64;
int current_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices ? dev : 0;
}

// SMs of the current device (a constant of the device, read once for each).
int sm_count() {
  static int known[kMaxDevices];
  const int dev = current_device();
  if (!known[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
    known[dev] = n;
  }
  return known[dev];
}

template <int DT, int NV, int MAXT, int MINB>
cudaError_t launch_norm_rows(const NormParams& p, cudaStream_t s) {
  const int tx = ((p.H / 8 + NV - 1) / NV + 31) / 32 * 32;
  const int ry = std::max(1, 128 / tx);
  const int64_t blocks = ((int64_t)p.T + ry - 1) / ry;
  const int64_t resident = (int64_t)sm_count() * MINB * (MAXT / (tx * ry));
  return launch_pdl(norm_rows_kernel<DT, NV, MAXT, MINB>, dim3((unsigned)std::min(blocks, resident)), dim3(tx, ry), 0, s, p);
}

template <int DT, int NV, int MAXT, int MINB>
cudaError_t launch_norm_staged(const NormParams& p, cudaStream_t s) {
  const int tx = ((p.H / 8 + NV - 1) / NV + 31) / 32 * 32;
  const size_t smem = (size_t)kNormStages * p.H * (p.residual ? 4 : 2);
  static bool configured[kMaxDevices];  // the opt-in lasts for the process
  const int dev = current_device();
  if (!configured[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(norm_staged_kernel<DT, NV, MAXT, MINB>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kNormStages * MAXT * NV * 32);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const int per_sm = std::max(1, std::min(MINB * (MAXT / tx), (int)(233472 / (smem + 1024 + 768))));
  return launch_pdl(norm_staged_kernel<DT, NV, MAXT, MINB>, dim3((unsigned)std::min<int64_t>(p.T, (int64_t)sm_count() * per_sm)),
                    dim3(tx), smem, s, p);
}

template <int DT, int VE, int TX, int NV, int MINB>
cudaError_t launch_norm_any(const NormParams& p, cudaStream_t s) {
  constexpr int kRowsPerBlock = TX < 256 ? 256 / TX : 1;
  const size_t smem = p.out8 && p.group ? (size_t)kRowsPerBlock * p.n_blocks * 4 : 0;
  const int64_t blocks = ((int64_t)p.T + kRowsPerBlock - 1) / kRowsPerBlock;
  return launch_pdl(norm_any_kernel<DT, VE, TX, NV, MINB>, dim3((unsigned)std::min(blocks, (int64_t)sm_count() * MINB)),
                    dim3(TX, kRowsPerBlock), smem, s, p);
}

// Threads per row by the row's pieces: half or more of a thread's places are used. (H = 7169, T = 8192: 512 threads
// with 16 pieces, two blocks per SM 209 us; 1024 with 8, one block 267, two 227; 512 with 16, three blocks, spills, 251.)
template <int DT, int VE>
cudaError_t norm_any_by_size(const NormParams& p, cudaStream_t s) {
  const int n = p.H / VE;
  if (n <= 256) return launch_norm_any<DT, VE, 32, 8, 6>(p, s);
  if (n <= 1024) return launch_norm_any<DT, VE, 128, 8, 5>(p, s);
  if (n <= 2048) return launch_norm_any<DT, VE, 256, 8, 5>(p, s);
  if (n <= 4096) return launch_norm_any<DT, VE, 256, 16, 4>(p, s);
  if (n <= 8192) return launch_norm_any<DT, VE, 512, 16, 2>(p, s);
  if constexpr (VE == 1)
    if (n > 16384) return launch_norm_any<DT, VE, 1024, 32, 1>(p, s);
  return launch_norm_any<DT, VE, 1024, 16, 1>(p, s);
}

template <int DT>
cudaError_t norm_by_size(const NormParams& p, int ve, cudaStream_t s) {
  if (ve == 8) {
    if (p.H <= 1024) return launch_norm_rows<DT, 1, 128, 8>(p, s);
    if (p.H <= 8192) return launch_norm_staged<DT, 2, 512, 2>(p, s);
    if (p.H <= 14336) return launch_norm_staged<DT, 2, 896, 1>(p, s);
  }
  return ve == 1 ? norm_any_by_size<DT, 1>(p, s) : norm_any_by_size<DT, 2>(p, s);
}

// ---- a serving step's plan ---------------------------------------------------------------------

constexpr int kPlanThreads = 256;

// Every block scans the B requests for itself (each thread a run of consecutive ones), then
// takes its share of the tokens and of the new pages; a token or page finds its request by
// binary search in the scanned sums. A token's page is read from the table only where it
// was there before the call, so blocks do not depend on one another's writes. A chain of latencies bounds it, not
// bytes (0.4 MB at most): launch, lengths, scan, search, table. In a graph 53 requests 2.7 us, 1,021 with 43,848
// tokens, four requests per thread, 4.4 us.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const moe_paged_plan_args a, int p_shift) {
  __shared__ int32_t s_tok[MOE_PLAN_MAX_REQUESTS + 1];   // exclusive sums of new tokens
  __shared__ int32_t s_page[MOE_PLAN_MAX_REQUESTS + 1];  // exclusive sums of new pages
  __shared__ long long w_tok[kPlanThreads / 32], w_page[kPlanThreads / 32];
  __shared__ int s_bad;
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const int B = a.B, P = a.page_size;
  const int seg = (B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(B, tid * seg), b1 = min(B, b0 + seg);
  long long tok = 0, page = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const long long c = a.ctx_lens[b], n = a.new_lens[b];
    if (c < 0 || n < 0 || c + n > (long long)a.W * P) {
      bad = true;
      continue;
    }
    tok += n;
    page += ((c + n + P - 1) >> p_shift) - ((c + P - 1) >> p_shift);
  }
  if (bad) s_bad = 1;
  long long it = tok, ip = page;  // inclusive sums over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ut = __shfl_up_sync(0xFFFFFFFFu, it, o), up = __shfl_up_sync(0xFFFFFFFFu, ip, o);
    if (lane >= o) {
      it += ut;
      ip += up;
    }
  }
  if (lane == 31) {
    w_tok[warp] = it;
    w_page[warp] = ip;
  }
  __syncthreads();
  long long pt = 0, pp = 0, total_t = 0, total_p = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) {
      pt += w_tok[w];
      pp += w_page[w];
    }
    total_t += w_tok[w];
    total_p += w_page[w];
  }
  pt += it - tok;
  pp += ip - page;
  const long long head = a.free_head[0];
  bad = s_bad != 0 || total_t > a.N || head < 0 || head + total_p > a.F;
  if (!bad) {
    for (int b = b0; b < b1; ++b) {
      const int c = a.ctx_lens[b], n = a.new_lens[b];
      s_tok[b] = (int)pt;
      s_page[b] = (int)pp;
      if (blockIdx.x == 0) {
        a.q_start[b] = (int)pt;
        a.kv_lens[b] = c + n;
      }
      pt += n;
      pp += ((c + n + P - 1) >> p_shift) - ((c + P - 1) >> p_shift);
    }
    if (tid == 0) {
      s_tok[B] = (int)total_t;
      s_page[B] = (int)total_p;
    }
  } else if (blockIdx.x == 0) {
    for (int b = b0; b < b1; ++b) a.q_start[b] = a.kv_lens[b] = 0;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.q_start[B] = bad ? 0 : (int)total_t;
    a.free_head_out[0] = (int)(bad ? head : head + total_p);
    if (bad && a.err) atomicOr(a.err, kErrPlan);
  }
  __syncthreads();
  const int nt = bad ? 0 : (int)total_t, np = bad ? 0 : (int)total_p;
  auto find = [B](const int32_t* s, int v) {  // the last request whose sum is <= v
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s[mid] <= v) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  const int step = gridDim.x * kPlanThreads;
  for (int i = blockIdx.x * kPlanThreads + tid; i < a.N; i += step) {
    int pos = 0, slot = -1;
    if (i < nt) {
      const int b = find(s_tok, i), c = a.ctx_lens[b];
      pos = c + i - s_tok[b];
      const int col = pos >> p_shift, have = (int)(((long long)c + P - 1) >> p_shift);
      const int page_id = col < have ? a.block_table[b * a.table_stride + col]
                                     : a.free_pages[head + s_page[b] + col - have];
      const long long at = ((long long)page_id << p_shift) + (pos & (P - 1));
      if (page_id >= 0 && at < (1ll << 31)) slot = (int)at;
      else if (a.err) atomicOr(a.err, kErrIndex);
    }
    a.positions[i] = pos;
    a.slots[i] = slot;
  }
  for (int i = blockIdx.x * kPlanThreads + tid; i < np; i += step) {
    const int b = find(s_page, i);
    const int have = (int)(((long long)a.ctx_lens[b] + P - 1) >> p_shift);
    a.block_table[b * a.table_stride + have + i - s_page[b]] = a.free_pages[head + i];
  }
}

// ---- rotary positions and the cache append -----------------------------------------------------

constexpr int kRotaryThreads = 256;

// A rotary pair's turns per position as a 64-bit fraction of a turn: position * fraction mod 2^64 is the
// angle's, exactly, and costs an integer product (a 32-bit float angle would be off by 2^-24 of itself:
// a hundredth of a radian at position 10^5).
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
  double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);
}
__device__ __forceinline__ float2 turned(uint64_t fraction, int pos, float mscale) {
  const int32_t top = (int32_t)(((uint64_t)(int64_t)pos * fraction) >> 32);  // signed fraction of a turn
  float sn, cn;
  sincospif((float)top * (1.f / 2147483648.f), &sn, &cn);
  return make_float2(cn * mscale, sn * mscale);
}

// Where a token's k and v go: false if nowhere (slot -1, or outside the cache, which is reported).
__device__ __forceinline__ bool cache_row(const moe_rotary_args& a, int p_shift, int slot, int64_t& kc, int64_t& vc) {
  const bool ok = slot >= 0 && slot < (a.num_pages << p_shift);
  if (slot < -1 || (slot >= 0 && !ok)) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && a.err) atomicOr(a.err, kErrIndex);
  }
  const int64_t page = slot >> p_shift, row = slot & (a.page_size - 1);
  kc = page * a.kc_page + row * a.kc_row;
  vc = page * a.vc_page + row * a.vc_row;
  return ok;
}

// Pieces of PE elements (8: 16 bytes). A token's work is the same list of items for every token: a rotated piece (in the half
// layout with its partner half a rotary width away), a piece that passes, a piece of v. A thread
// works out its U items once and then walks over tokens: all its loads first, then the token's
// cosines and sines (shared by the heads; one exchange per token), then the products and stores.
// Where a part of a head, a stride or an address is no multiple of 8 elements, the pieces are 4 or 1 elements.
// Every element is read and written once, so memory bounds it: N = 8192, 96 + 2 x 8 heads of 128, bf16:
// 72.0 us, 6.5 TB/s, and 93 in pieces of 4, 296 of 1; with 104 of 128 rotated in halves, which need pieces of 4,
// 107. U items per thread and blocks per SM measured there: 4 and 3 72.0, 4 and 4 (spills)
// 87.5, 2 and 4 78.0, 2 and 6 77.4, 1 and 8 77.4 us; one item after another with two barriers per token 84 us. (1 and 8,
// and 2 and 6, which take tokens and calls of few items, spill 12 to 56 bytes too and are the faster there: N = 1531, 24 + 2 x 4
// heads of 64 4.8 us, with 4 and 3 6.3.)
template <int DT, bool INTER, int PE, int U, int MINB>
__global__ void __launch_bounds__(kRotaryThreads, MINB) rotary_kernel(const moe_rotary_args a, int p_shift) {
  constexpr bool kInPiece = INTER && PE > 1;  // both elements of a pair lie in the piece
  constexpr int kPairs = kInPiece ? PE / 2 : PE;
  // pair i sits at i + i / 8 * 2: pieces of 8 pairs are 80 bytes apart, so lanes on different pieces do not
  // meet in a bank
  __shared__ __align__(16) float2 cs[2][512 + 128];
  pdl_entry();
  const int tid = threadIdx.x, half = a.rot / 2;
  const int r_pieces = kInPiece ? a.rot / PE : half / PE, c_pieces = (a.D - a.rot) / PE, v_pieces = a.D / PE;
  const int h_pieces = r_pieces + c_pieces, heads = a.Hq + a.Hkv, n_rot = heads * h_pieces;
  const int partner = INTER ? 1 : half;  // from a pair's first element to its second
  int64_t from[U], to[U];
  int kind[U], pair[U];  // kind: 0 nothing, 1 q, 2 k, 3 v; pair: the piece's first rotary pair, or -1
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int it = ((int)blockIdx.x * U + u) * kRotaryThreads + tid;
    kind[u] = 0;
    pair[u] = -1;
    from[u] = to[u] = 0;
    if (it < n_rot) {
      const int h = it / h_pieces;
      int piece = it - h * h_pieces, at = piece * (INTER && PE == 1 ? 2 : PE);
      if (piece < r_pieces) pair[u] = piece * kPairs;
      else at = a.rot + (piece - r_pieces) * PE;
      kind[u] = h < a.Hq ? 1 : 2;
      from[u] = (h < a.Hq ? h * a.q_head : (h - a.Hq) * a.k_head) + at;
      to[u] = (h < a.Hq ? h * a.qo_head : (h - a.Hq) * a.kc_head) + at;
    } else if (it < n_rot + a.Hkv * v_pieces) {
      const int j = it - n_rot, h = j / v_pieces, at = (j - h * v_pieces) * PE;
      kind[u] = 3;
      from[u] = h * a.v_head + at;
      to[u] = h * a.vc_head + at;
    }
  }
  const uint64_t f0 = tid < half ? turn_fraction(a.inv_freq[tid]) : 0;
  int turn = 0;
  for (int n = blockIdx.y; n < a.N; n += gridDim.y, turn ^= 1) {
    int64_t kc, vc;
    const bool append = cache_row(a, p_shift, a.slots[n], kc, vc);
    const int pos = a.positions[n];
    Piece<PE> x[U], z[kInPiece ? 1 : U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kind[u] == 0 || (kind[u] > 1 && !append)) continue;
      const uint16_t* src = (kind[u] == 1   ? (const uint16_t*)a.q + n * a.q_tok
                             : kind[u] == 2 ? (const uint16_t*)a.k + n * a.k_tok
                                            : (const uint16_t*)a.v + n * a.v_tok) + from[u];
      x[u] = *reinterpret_cast<const Piece<PE>*>(src);
      if constexpr (!kInPiece)
        if (pair[u] >= 0) z[u] = *reinterpret_cast<const Piece<PE>*>(src + partner);
    }
    for (int i = tid; i < half; i += kRotaryThreads)
      cs[turn][i + (i >> 3) * 2] = turned(i == tid ? f0 : turn_fraction(a.inv_freq[i]), pos, a.mscale);
    __syncthreads();  // one per token: the next token's values go to the other buffer
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kind[u] == 0 || (kind[u] > 1 && !append)) continue;
      uint16_t* dst = (kind[u] == 1   ? (uint16_t*)a.q_out + n * a.qo_tok
                       : kind[u] == 2 ? (uint16_t*)a.k_cache + kc
                                      : (uint16_t*)a.v_cache + vc) + to[u];
      if (pair[u] < 0) {
        *reinterpret_cast<Piece<PE>*>(dst) = x[u];
        continue;
      }
      const float2* c = cs[turn] + pair[u] + (pair[u] >> 3) * 2;  // (a piece's pairs lie in one run of eight)
      float p[PE], y[PE];
      unpack<DT, PE>(x[u], p);
      if constexpr (kInPiece) {
#pragma unroll
        for (int j = 0; j < PE / 2; ++j) {
          y[2 * j] = p[2 * j] * c[j].x - p[2 * j + 1] * c[j].y;
          y[2 * j + 1] = p[2 * j] * c[j].y + p[2 * j + 1] * c[j].x;
        }
      } else {
        float q[PE], w[PE];
        unpack<DT, PE>(z[u], q);
#pragma unroll
        for (int j = 0; j < PE; ++j) {
          y[j] = p[j] * c[j].x - q[j] * c[j].y;
          w[j] = p[j] * c[j].y + q[j] * c[j].x;
        }
        store_vec<DT, PE>(dst + partner, w);
      }
      store_vec<DT, PE>(dst, y);
    }
  }
}

template <int DT, bool INTER, int PE, int U, int MINB>
cudaError_t launch_rotary_as(const moe_rotary_args& a, int groups, int p_shift, cudaStream_t s) {
  const int x = (groups + U - 1) / U;
  const int y = std::max(1, std::min(a.N, MINB * sm_count() / x));
  return launch_pdl(rotary_kernel<DT, INTER, PE, U, MINB>, dim3((unsigned)x, (unsigned)y), dim3(kRotaryThreads), 0, s, a, p_shift);
}

template <int DT, bool INTER, int PE>
cudaError_t launch_rotary_pieces(const moe_rotary_args& a, int p_shift, cudaStream_t s) {
  const int64_t rotated = INTER && PE > 1 ? a.rot / PE : a.rot / 2 / PE;  // pieces of a head
  const int64_t items = (int64_t)(a.Hq + a.Hkv) * (rotated + (a.D - a.rot) / PE) + (int64_t)a.Hkv * (a.D / PE);
  const int groups = (int)((items + kRotaryThreads - 1) / kRotaryThreads);
  // few tokens: a token's items over several blocks (N = 53: 2.6 us a launch in a graph against 3.6). Short pieces:
  // the same, for more bytes in flight (N = 8192, 104 of 128 rotated in halves: 107 us against 129 with 4 items)
  if constexpr (PE == 8) {
    if (groups > 1 && (int64_t)a.N * groups > 8 * sm_count())
      return groups == 2 ? launch_rotary_as<DT, INTER, PE, 2, 6>(a, groups, p_shift, s)
                         : launch_rotary_as<DT, INTER, PE, 4, 3>(a, groups, p_shift, s);
  }
  return launch_rotary_as<DT, INTER, PE, 1, 8>(a, groups, p_shift, s);
}

template <int DT, bool INTER>
cudaError_t launch_rotary(const moe_rotary_args& a, int pe, int p_shift, cudaStream_t s) {
  return pe == 8   ? launch_rotary_pieces<DT, INTER, 8>(a, p_shift, s)
         : pe == 4 ? launch_rotary_pieces<DT, INTER, 4>(a, p_shift, s)
                   : launch_rotary_pieces<DT, INTER, 1>(a, p_shift, s);
}

int shift_of(int p) {
  int s = 0;
  while ((1 << s) < p) ++s;
  return s;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_add_rmsnorm(void* stream, const moe_rmsnorm_args* a) {
  if (!a || a->T < 0) return MOE_ERR_INVALID_ARG;
  if (a->dtype != MOE_DT_BF16 && a->dtype != MOE_DT_F16) return MOE_ERR_INVALID_ARG;
  if (a->H < 1 || (a->group != 0 && a->group != 128) || !(a->eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (a->H > 32768) return MOE_ERR_UNSUPPORTED;
  if (a->T == 0) return MOE_OK;
  if (!a->x || !a->weight || (!a->out && !a->out8) || (!a->out8 != !a->scales)) return MOE_ERR_INVALID_ARG;
  if (a->residual_out && !a->residual) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(a->x, 2) || !is_aligned(a->residual, 2) || !is_aligned(a->out, 2) ||
      !is_aligned(a->residual_out, 2) || !is_aligned(a->weight, a->weight_f32 ? 4 : 2) || !is_aligned(a->scales, 4) || !is_aligned(a->err, 4))
    return MOE_ERR_INVALID_ARG;
  if (a->x_stride < a->H || (a->residual && a->residual_stride < a->H) || (a->out && a->out_stride < a->H) ||
      (a->residual_out && a->residual_out_stride < a->H) || (a->out8 && a->out8_stride < a->H))
    return MOE_ERR_INVALID_ARG;
  NormParams p;
  p.x = (const uint16_t*)a->x;
  p.residual = (const uint16_t*)a->residual;
  p.weight = a->weight;
  p.out = (uint16_t*)a->out;
  p.residual_out = (uint16_t*)a->residual_out;
  p.out8 = a->out8;
  p.scales = a->scales;
  p.x_stride = a->x_stride;
  p.residual_stride = a->residual_stride;
  p.out_stride = a->out_stride;
  p.residual_out_stride = a->residual_out_stride;
  p.out8_stride = a->out8_stride;
  p.T = a->T;
  p.H = a->H;
  p.weight_f32 = a->weight_f32;
  p.group = a->group;
  p.n_blocks = a->group ? (a->H + 127) / 128 : 1;
  p.eps = a->eps;
  p.err = a->err;
  // the widest piece that divides the width, the strides and the addresses: 8 elements, 2, or 1
  const auto fits = [&](int n) {
    const auto ok = [n](const void* q, int64_t stride, int size) { return !q || (is_aligned(q, n * size) && stride % n == 0); };
    return a->H % n == 0 && ok(a->x, a->x_stride, 2) && ok(a->residual, a->residual_stride, 2) && ok(a->out, a->out_stride, 2) &&
           ok(a->residual_out, a->residual_out_stride, 2) && ok(a->weight, 0, 2) && ok(a->out8, a->out8_stride, 1);
  };
  const int ve = fits(8) ? 8 : fits(2) ? 2 : 1;
  OpsPdl pdl;
  const cudaError_t e = a->dtype == MOE_DT_BF16 ? norm_by_size<MOE_DT_BF16>(p, ve, (cudaStream_t)stream)
                                                : norm_by_size<MOE_DT_F16>(p, ve, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_paged_plan(void* stream, const moe_paged_plan_args* a) {
  if (!a || !a->ctx_lens || !a->new_lens || !a->block_table || !a->free_head || !a->q_start || !a->kv_lens ||
      !a->free_head_out || (a->F > 0 && !a->free_pages))
    return MOE_ERR_INVALID_ARG;
  if (a->B < 1 || a->W < 1 || a->F < 0 || a->N < 0 || a->table_stride < a->W || !is_pow2(a->page_size))
    return MOE_ERR_INVALID_ARG;
  if (a->N > 0 && (!a->positions || !a->slots)) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {a->ctx_lens, a->new_lens, a->block_table, a->free_pages, a->free_head, a->q_start,
                        a->kv_lens,  a->positions, a->slots,      a->free_head_out, a->err};
  for (const void* q : ptrs)
    if (!is_aligned(q, 4)) return MOE_ERR_INVALID_ARG;
  if (a->B > MOE_PLAN_MAX_REQUESTS || (int64_t)a->W * a->page_size >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  // Every block reads the inputs again after others have begun to write: an output that shares a word with an
  // input, or with another output, would change positions, slots and table columns, or write past the table.
  struct {
    const void* p;
    int64_t words;
  } const t[] = {{a->block_table, (a->B - 1) * a->table_stride + a->W},
                 {a->q_start, (int64_t)a->B + 1},
                 {a->kv_lens, a->B},
                 {a->positions, a->N},
                 {a->slots, a->N},
                 {a->free_head_out, 1},
                 {a->err, a->err ? 1 : 0},  // outputs up to here
                 {a->ctx_lens, a->B},
                 {a->new_lens, a->B},
                 {a->free_pages, a->F},
                 {a->free_head, 1}};
  for (int o = 0; o < 7; ++o)
    for (int i = o + 1; i < 11; ++i) {
      const uintptr_t x = (uintptr_t)t[o].p, y = (uintptr_t)t[i].p;
      if (x < y + 4 * t[i].words && y < x + 4 * t[o].words && t[o].words && t[i].words) return MOE_ERR_INVALID_ARG;
    }
  const int blocks = (a->N + kPlanThreads - 1) / kPlanThreads;
  OpsPdl pdl;
  return launch_pdl(plan_kernel, dim3((unsigned)(blocks < 1 ? 1 : blocks > 304 ? 304 : blocks)), dim3(kPlanThreads),
                    0, (cudaStream_t)stream, *a, shift_of(a->page_size)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_rotary_append(void* stream, const moe_rotary_args* a) {
  if (!a || a->N < 0) return MOE_ERR_INVALID_ARG;
  if (a->dtype != MOE_DT_BF16 && a->dtype != MOE_DT_F16) return MOE_ERR_INVALID_ARG;
  if (a->Hq < 1 || a->Hkv < 1 || a->D < 2 || a->D % 2 || a->rot < 2 || a->rot > a->D || a->rot % 2 ||
      a->num_pages < 1 || !is_pow2(a->page_size))
    return MOE_ERR_INVALID_ARG;
  if (a->D > 1024 || (int64_t)a->num_pages * a->page_size >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)(a->Hq + 2 * (int64_t)a->Hkv) * a->D >= ((int64_t)1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (a->N == 0) return MOE_OK;
  const void* t16[] = {a->q, a->k, a->v, a->q_out, a->k_cache, a->v_cache};
  const int64_t strides[] = {a->q_tok,  a->q_head,  a->k_tok,  a->k_head, a->v_tok,   a->v_head, a->qo_tok,
                             a->qo_head, a->kc_page, a->kc_row, a->kc_head, a->vc_page, a->vc_row, a->vc_head};
  // the widest piece that divides the head's parts, the strides and the addresses: 8 elements, 4, or 1
  int pe = 8;
  const auto fits = [&](int64_t v) {
    if (v % pe) pe = v % 4 ? 1 : 4;
  };
  fits(a->D);
  fits(a->interleaved ? a->rot : a->rot / 2);
  for (const void* p : t16) {
    if (!p || !is_aligned(p, 2)) return MOE_ERR_INVALID_ARG;
    fits((int64_t)((uintptr_t)p / 2 % 8));
  }
  for (int64_t s : strides) {
    if (s < 0) return MOE_ERR_INVALID_ARG;
    fits(s);
  }
  if (!a->positions || !a->slots || !a->inv_freq || !is_aligned(a->positions, 4) || !is_aligned(a->slots, 4) ||
      !is_aligned(a->inv_freq, 8) || !is_aligned(a->err, 4))
    return MOE_ERR_INVALID_ARG;
  OpsPdl pdl;
  const int sh = shift_of(a->page_size);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e =
      a->dtype == MOE_DT_BF16
          ? (a->interleaved ? launch_rotary<MOE_DT_BF16, true>(*a, pe, sh, st) : launch_rotary<MOE_DT_BF16, false>(*a, pe, sh, st))
          : (a->interleaved ? launch_rotary<MOE_DT_F16, true>(*a, pe, sh, st) : launch_rotary<MOE_DT_F16, false>(*a, pe, sh, st));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
