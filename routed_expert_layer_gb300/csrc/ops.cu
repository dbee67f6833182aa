// Operators beside the expert layer whose work is moving data: the residual norm, a serving
// step's plan, rotary positions with the cache append. Interfaces and formulas:
// include/moe_ops_gb300.h.
#include "ops_internal.cuh"

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
};

template <int DT, int VEC>
__device__ __forceinline__ void load_vec(const uint16_t* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<DT>(u[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
    v[0] = to_f32<DT>(*p);
  }
}

template <int DT, int VEC>
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    uint4 w;
    w.x = pack2<DT>(v[0], v[1]);
    w.y = pack2<DT>(v[2], v[3]);
    w.z = pack2<DT>(v[4], v[5]);
    w.w = pack2<DT>(v[6], v[7]);
    *reinterpret_cast<uint4*>(p) = w;
  } else {
    *p = from_f32<DT>(v[0]);
  }
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// |v| as an unsigned integer: its order is that of the magnitudes, and a NaN is the largest.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

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

// One row per block row; thread x holds chunks x, x + blockDim.x, ... of VEC elements in
// registers, so every input is read once.
template <int DT, int VEC, int NV>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p) {
  __shared__ float red_sum[32];
  __shared__ uint32_t red_max[32];
  extern __shared__ uint32_t block_max[];  // VEC == 1 with blocks of 128: [block rows][n_blocks]
  pdl_entry();
  const int tx = threadIdx.x, TX = blockDim.x, H = p.H;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.T;
  float t[NV][VEC];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (tx + i * TX) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) t[i][j] = 0.f;
    if (live && e < H) {
      load_vec<DT, VEC>(p.x + row * p.x_stride + e, t[i]);
      if (p.residual) {
        float r[VEC];
        load_vec<DT, VEC>(p.residual + row * p.residual_stride + e, r);
#pragma unroll
        for (int j = 0; j < VEC; ++j) t[i][j] += r[j];
        if (p.residual_out) store_vec<DT, VEC>(p.residual_out + row * p.residual_out_stride + e, t[i]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss = fmaf(t[i][j], t[i][j], ss);
    }
  }
  const float rs = rsqrtf(row_sum(ss, red_sum) / (float)H + p.eps);
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (tx + i * TX) * VEC;
    if (live && e < H) {
      float w[VEC];
      if (p.weight_f32) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] = reinterpret_cast<const float*>(p.weight)[e + j];
      } else {
        load_vec<DT, VEC>(reinterpret_cast<const uint16_t*>(p.weight) + e, w);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        t[i][j] = t[i][j] * rs * w[j];
        mx = max(mx, abs_bits(t[i][j]));
      }
      if (p.out) store_vec<DT, VEC>(p.out + row * p.out_stride + e, t[i]);
    }
  }
  if (!p.out8) return;
  uint32_t* bm = block_max + threadIdx.y * p.n_blocks;
  if (p.group == 0) {
    mx = row_max(mx, red_max);
    if (live && tx == 0) p.scales[row] = __uint_as_float(mx) / 448.f;
  } else if constexpr (VEC == 1) {
    for (int b = tx; b < p.n_blocks; b += TX) bm[b] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = tx + i * TX;
      if (live && e < H) atomicMax(&bm[e >> 7], abs_bits(t[i][0]));
    }
    __syncthreads();
    for (int b = tx; live && b < p.n_blocks; b += TX) p.scales[row * p.n_blocks + b] = __uint_as_float(bm[b]) / 448.f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (tx + i * TX) * VEC;
    uint32_t m = mx;
    if (p.group) {
      if constexpr (VEC == 1) {
        m = e < H ? bm[e >> 7] : 0;
      } else {  // 16 consecutive threads hold one block of 128
        m = 0;
#pragma unroll
        for (int j = 0; j < VEC; ++j) m = max(m, abs_bits(t[i][j]));
#pragma unroll
        for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (live && e < H && (tx & 15) == 0) p.scales[row * p.n_blocks + (e >> 7)] = __uint_as_float(m) / 448.f;
      }
    }
    if (!live || e >= H) continue;
    const float s = __uint_as_float(m) / 448.f;
    const float inv = s > 0.f ? 1.f / s : 1.f;  // zeros stay zeros; a NaN scale keeps its NaN values
    uint8_t* o = p.out8 + row * p.out8_stride + e;
    if constexpr (VEC == 8) {
      uint2 w;
      w.x = e4m3x2(t[i][0] * inv, t[i][1] * inv) | e4m3x2(t[i][2] * inv, t[i][3] * inv) << 16;
      w.y = e4m3x2(t[i][4] * inv, t[i][5] * inv) | e4m3x2(t[i][6] * inv, t[i][7] * inv) << 16;
      *reinterpret_cast<uint2*>(o) = w;
    } else {
      *o = (uint8_t)e4m3x2(t[i][0] * inv, 0.f);
    }
  }
}

template <int DT, int VEC, int NV>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  const int chunks = (p.H + VEC - 1) / VEC;
  const int tx = ((chunks + NV - 1) / NV + 31) / 32 * 32;
  const int ry = tx >= 256 ? 1 : 256 / tx;
  const size_t smem = (VEC == 1 && p.out8 && p.group) ? (size_t)ry * p.n_blocks * 4 : 0;
  return launch_pdl(norm_kernel<DT, VEC, NV>, dim3((unsigned)((p.T + ry - 1) / ry)), dim3(tx, ry), smem, s, p);
}

template <int DT>
cudaError_t norm_by_size(const NormParams& p, bool vec, cudaStream_t s) {
  if (vec) {
    if (p.H <= 8 * 1024) return launch_norm<DT, 8, 1>(p, s);
    if (p.H <= 16 * 1024) return launch_norm<DT, 8, 2>(p, s);
    return launch_norm<DT, 8, 4>(p, s);
  }
  if (p.H <= 4 * 1024) return launch_norm<DT, 1, 4>(p, s);
  return launch_norm<DT, 1, 32>(p, s);
}

// ---- a serving step's plan ---------------------------------------------------------------------

constexpr int kPlanThreads = 256;

// Every block scans the B requests for itself (each thread a run of consecutive ones), then
// takes its share of the tokens and of the new pages; a token or page finds its request by
// binary search in the scanned sums. A token's page is read from the table only where it
// was there before the call, so blocks do not depend on one another's writes.
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

// VEC: 1 = one pair (or element) per item; 8 = 16-byte vectors.
template <int DT, int VEC, bool INTER>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const moe_rotary_args a, int p_shift) {
  __shared__ float2 cs[512];
  pdl_entry();
  const int half = a.rot / 2;
  // Angle in turns as a 64-bit fraction: pos * (inv_freq / 2 pi) mod 1 is an integer product.
  auto fraction = [&](int i) -> uint64_t {
    double t = a.inv_freq[i] * 0.15915494309189533577;
    t -= floor(t);
    return __double2ull_rn(t * 18446744073709551616.0);
  };
  uint64_t f0 = threadIdx.x < half ? fraction(threadIdx.x) : 0;
  const int n_slots = a.num_pages << p_shift;
  // items of a token: rotated heads (q then k) in pieces, then v heads in pieces
  const int r_pieces = INTER || VEC == 1 ? (VEC == 1 ? half : a.rot / 8) : half / 8;
  const int c_pieces = (a.D - a.rot) / (VEC == 1 ? 1 : 8);  // unrotated rest of a head
  const int v_pieces = a.D / (VEC == 1 ? 1 : 8);
  const int h_pieces = r_pieces + c_pieces;
  const int heads = a.Hq + a.Hkv;
  const int n_items = heads * h_pieces + a.Hkv * v_pieces;
  for (int n = blockIdx.x; n < a.N; n += gridDim.x) {
    const int pos = a.positions[n];
    for (int i = threadIdx.x; i < half; i += kRotaryThreads) {
      const uint64_t f = i == (int)threadIdx.x ? f0 : fraction(i);
      const int32_t top = (int32_t)(((uint64_t)(int64_t)pos * f) >> 32);  // signed fraction of a turn
      float sn, cn;
      sincospif((float)top * (1.f / 2147483648.f), &sn, &cn);
      cs[i] = make_float2(cn * a.mscale, sn * a.mscale);
    }
    const int slot = a.slots[n];
    const bool append = slot >= 0 && slot < n_slots;
    if ((slot < -1 || slot >= n_slots) && threadIdx.x == 0 && blockIdx.y == 0 && a.err) atomicOr(a.err, kErrIndex);
    const int64_t page = append ? slot >> p_shift : 0, prow = append ? slot & (a.page_size - 1) : 0;
    const uint16_t* q = (const uint16_t*)a.q + n * a.q_tok;
    const uint16_t* k = (const uint16_t*)a.k + n * a.k_tok;
    const uint16_t* v = (const uint16_t*)a.v + n * a.v_tok;
    uint16_t* qo = (uint16_t*)a.q_out + n * a.qo_tok;
    uint16_t* kc = (uint16_t*)a.k_cache + page * a.kc_page + prow * a.kc_row;
    uint16_t* vc = (uint16_t*)a.v_cache + page * a.vc_page + prow * a.vc_row;
    __syncthreads();
    for (int it = blockIdx.y * kRotaryThreads + threadIdx.x; it < n_items; it += gridDim.y * kRotaryThreads) {
      const uint16_t* src;
      uint16_t* dst;
      int piece;
      bool rotated = false, write = true;
      if (it < heads * h_pieces) {
        const int h = it / h_pieces;
        piece = it - h * h_pieces;
        if (h < a.Hq) {
          src = q + h * a.q_head;
          dst = qo + h * a.qo_head;
        } else {
          src = k + (h - a.Hq) * a.k_head;
          dst = kc + (h - a.Hq) * a.kc_head;
          write = append;
        }
        rotated = piece < r_pieces;
        if (!rotated) {
          src += a.rot;
          dst += a.rot;
          piece -= r_pieces;
        }
      } else {
        const int j = it - heads * h_pieces, h = j / v_pieces;
        piece = j - h * v_pieces;
        src = v + h * a.v_head;
        dst = vc + h * a.vc_head;
        write = append;
      }
      if (!write) continue;
      if (!rotated) {
        if constexpr (VEC == 8)
          *reinterpret_cast<uint4*>(dst + piece * 8) = *reinterpret_cast<const uint4*>(src + piece * 8);
        else
          dst[piece] = src[piece];
      } else if constexpr (VEC == 8 && INTER) {
        float x[8], y[8];
        load_vec<DT, 8>(src + piece * 8, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 c = cs[piece * 4 + j];
          y[2 * j] = x[2 * j] * c.x - x[2 * j + 1] * c.y;
          y[2 * j + 1] = x[2 * j] * c.y + x[2 * j + 1] * c.x;
        }
        store_vec<DT, 8>(dst + piece * 8, y);
      } else if constexpr (VEC == 8) {
        float x[8], z[8], y[8], w[8];
        load_vec<DT, 8>(src + piece * 8, x);
        load_vec<DT, 8>(src + half + piece * 8, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 c = cs[piece * 8 + j];
          y[j] = x[j] * c.x - z[j] * c.y;
          w[j] = x[j] * c.y + z[j] * c.x;
        }
        store_vec<DT, 8>(dst + piece * 8, y);
        store_vec<DT, 8>(dst + half + piece * 8, w);
      } else {
        const int i0 = INTER ? 2 * piece : piece, i1 = INTER ? 2 * piece + 1 : piece + half;
        const float x = to_f32<DT>(src[i0]), z = to_f32<DT>(src[i1]);
        const float2 c = cs[piece];
        dst[i0] = from_f32<DT>(x * c.x - z * c.y);
        dst[i1] = from_f32<DT>(x * c.y + z * c.x);
      }
    }
    __syncthreads();
  }
}

template <int DT>
cudaError_t launch_rotary(const moe_rotary_args& a, bool vec, int p_shift, cudaStream_t s) {
  const dim3 grid((unsigned)min(a.N, 65535)), block(kRotaryThreads);
  if (vec)
    return a.interleaved ? launch_pdl(rotary_kernel<DT, 8, true>, grid, block, 0, s, a, p_shift)
                         : launch_pdl(rotary_kernel<DT, 8, false>, grid, block, 0, s, a, p_shift);
  return a.interleaved ? launch_pdl(rotary_kernel<DT, 1, true>, grid, block, 0, s, a, p_shift)
                       : launch_pdl(rotary_kernel<DT, 1, false>, grid, block, 0, s, a, p_shift);
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
      !is_aligned(a->residual_out, 2) || !is_aligned(a->weight, a->weight_f32 ? 4 : 2) || !is_aligned(a->scales, 4))
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
  const auto ok16 = [](const void* q, int64_t stride) { return !q || (is_aligned(q, 16) && stride % 8 == 0); };
  const bool vec = a->H % 8 == 0 && ok16(a->x, a->x_stride) && ok16(a->residual, a->residual_stride) &&
                   ok16(a->out, a->out_stride) && ok16(a->residual_out, a->residual_out_stride) &&
                   is_aligned(a->weight, 16) && (!a->out8 || (is_aligned(a->out8, 8) && a->out8_stride % 8 == 0));
  OpsPdl pdl;
  const cudaError_t e = a->dtype == MOE_DT_BF16 ? norm_by_size<MOE_DT_BF16>(p, vec, (cudaStream_t)stream)
                                                : norm_by_size<MOE_DT_F16>(p, vec, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_paged_plan(void* stream, const moe_paged_plan_args* a) {
  if (!a || !a->ctx_lens || !a->new_lens || !a->block_table || !a->free_pages || !a->free_head || !a->q_start ||
      !a->kv_lens || !a->free_head_out || a->free_head == a->free_head_out)
    return MOE_ERR_INVALID_ARG;
  if (a->B < 1 || a->W < 1 || a->F < 0 || a->N < 0 || a->table_stride < a->W || !is_pow2(a->page_size))
    return MOE_ERR_INVALID_ARG;
  if (a->N > 0 && (!a->positions || !a->slots)) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {a->ctx_lens, a->new_lens, a->block_table, a->free_pages, a->free_head, a->q_start,
                        a->kv_lens,  a->positions, a->slots,      a->free_head_out, a->err};
  for (const void* q : ptrs)
    if (!is_aligned(q, 4)) return MOE_ERR_INVALID_ARG;
  if (a->B > MOE_PLAN_MAX_REQUESTS || (int64_t)a->W * a->page_size >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
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
  bool vec = a->D % 8 == 0 && a->rot % (a->interleaved ? 8 : 16) == 0;
  for (const void* p : t16) {
    if (!p || !is_aligned(p, 2)) return MOE_ERR_INVALID_ARG;
    vec = vec && is_aligned(p, 16);
  }
  for (int64_t s : strides) {
    if (s < 0) return MOE_ERR_INVALID_ARG;
    vec = vec && s % 8 == 0;
  }
  if (!a->positions || !a->slots || !a->inv_freq || !is_aligned(a->positions, 4) || !is_aligned(a->slots, 4) ||
      !is_aligned(a->inv_freq, 8) || !is_aligned(a->err, 4))
    return MOE_ERR_INVALID_ARG;
  OpsPdl pdl;
  const int sh = shift_of(a->page_size);
  const cudaError_t e = a->dtype == MOE_DT_BF16 ? launch_rotary<MOE_DT_BF16>(*a, vec, sh, (cudaStream_t)stream)
                                                : launch_rotary<MOE_DT_F16>(*a, vec, sh, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
