// Attention of new tokens over a paged cache (interface and formula: include/moe_ops_gb300.h).
//
// One warp per (token, query head): an online softmax over the keys the token sees, fp32
// scores, sums and accumulators. The last visible key bounds the loop, so keys a row does
// not see are never read.
#include "ops_internal.cuh"

struct moe_attn_ctx {
  int device = 0;
  int sm_count = 0;
  uint32_t* err = nullptr;
};

namespace moe {
namespace {

struct AttnParams {
  moe_attn_args a;
  int p_shift;
  float scale_log2;
  uint32_t* err;
};

template <int DT, int D>
__global__ void __launch_bounds__(128) attn_rows_kernel(const AttnParams p) {
  constexpr int E = D / 32;
  pdl_entry();
  const moe_attn_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (int64_t)a.N * a.Hq) return;
  const int n = (int)(item / a.Hq), h = (int)(item - (int64_t)n * a.Hq), g = h / (a.Hq / a.Hkv);
  int lo = 0, hi = a.B;  // the last request that starts at or before n
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= n) lo = mid;
    else hi = mid;
  }
  const int s0 = a.q_start[lo], s1 = a.q_start[lo + 1];
  if (n < s0 || n >= s1) return;
  if (s0 < 0 || s1 > a.N) {
    if (lane == 0) atomicOr(p.err, kErrIndex);
    return;
  }
  const int kv = a.kv_lens[lo];
  const int64_t seen = (int64_t)kv - (s1 - s0) + (n - s0) + 1;  // keys this row sees
  const int len = seen < 0 ? 0 : (int)seen;
  float q[E], o[E] = {};
  const uint16_t* qp = (const uint16_t*)a.q + n * a.q_tok + h * a.q_head + lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) q[i] = to_f32<DT>(qp[i]);
  float m = -INFINITY, l = 0.f;
  bool bad = false;
  for (int j = 0; j < len; ++j) {
    const int col = j >> p.p_shift, row = j & (a.page_size - 1);
    const int page = col < a.W ? a.block_table[lo * a.table_stride + col] : -1;
    const bool ok = page >= 0 && page < a.num_pages;
    bad |= !ok;
    const uint16_t* kp = (const uint16_t*)a.k_cache + page * a.kc_page + row * a.kc_row + g * a.kc_head + lane * E;
    const uint16_t* vp = (const uint16_t*)a.v_cache + page * a.vc_page + row * a.vc_row + g * a.vc_head + lane * E;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], ok ? to_f32<DT>(kp[i]) : 0.f, s);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(s - mn);
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * f + w * (ok ? to_f32<DT>(vp[i]) : 0.f);
    m = mn;
  }
  if (bad && lane == 0) atomicOr(p.err, kErrIndex);
  uint16_t* op = (uint16_t*)a.out + n * a.out_tok + h * a.out_head + lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) op[i] = from_f32<DT>(len > 0 ? o[i] / l : 0.f);
  if (a.lse && lane == 0) a.lse[(int64_t)n * a.Hq + h] = len > 0 ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

int attn_check(const moe_attn_args* a) {
  if (!a || a->N < 0 || a->B < 1 || a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv || a->num_pages < 1 || a->W < 1 ||
      a->max_new < 0 || !is_pow2(a->page_size) || a->table_stride < a->W)
    return MOE_ERR_INVALID_ARG;
  if (a->dtype != MOE_DT_BF16 && a->dtype != MOE_DT_F16) return MOE_ERR_INVALID_ARG;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return MOE_ERR_INVALID_ARG;
  if ((a->D != 64 && a->D != 128) || a->Hq / a->Hkv > 128 || a->page_size < 16 || a->page_size > 1024 ||
      (int64_t)a->W * a->page_size >= ((int64_t)1 << 31) || (int64_t)a->N * a->Hq >= ((int64_t)1 << 31))
    return MOE_ERR_UNSUPPORTED;
  if (a->N == 0) return MOE_OK;
  const void* t16[] = {a->q, a->k_cache, a->v_cache, a->out};
  for (const void* p : t16)
    if (!p || !is_aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  const int64_t strides[] = {a->q_tok,   a->q_head, a->out_tok, a->out_head, a->kc_page,
                             a->kc_row, a->kc_head, a->vc_page, a->vc_row,   a->vc_head};
  for (int64_t s : strides)
    if (s < 0 || s % 8 || s >= ((int64_t)1 << 38)) return MOE_ERR_INVALID_ARG;
  const void* t32[] = {a->block_table, a->q_start, a->kv_lens};
  for (const void* p : t32)
    if (!p || !is_aligned(p, 4)) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(a->lse, 4)) return MOE_ERR_INVALID_ARG;
  if (overlap(span16(a->q, a->N, a->q_tok, a->Hq, a->q_head, a->D),
              span16(a->out, a->N, a->out_tok, a->Hq, a->out_head, a->D)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_attn_create(int device, moe_attn_ctx** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess) return MOE_ERR_CUDA;
  if (device < 0 || device >= ndev) return MOE_ERR_INVALID_ARG;
  cudaDeviceProp prop;
  if (cudaGetDeviceProperties(&prop, device) != cudaSuccess) return MOE_ERR_CUDA;
  if (!(prop.major == 10 && prop.minor == 3)) return MOE_ERR_UNSUPPORTED;
  DeviceGuard g(device);
  moe_attn_ctx* c = new (std::nothrow) moe_attn_ctx();
  if (!c) return MOE_ERR_OOM;
  c->device = device;
  c->sm_count = prop.multiProcessorCount;
  if (cudaMalloc(&c->err, 256) != cudaSuccess) {
    cudaGetLastError();
    delete c;
    return MOE_ERR_OOM;
  }
  if (cudaMemset(c->err, 0, 256) != cudaSuccess) {
    cudaFree(c->err);
    delete c;
    return MOE_ERR_CUDA;
  }
  *out = c;
  return MOE_OK;
}

int moe_attn_forward(moe_attn_ctx* ctx, void* stream, const moe_attn_args* a) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  const int st = attn_check(a);
  if (st != MOE_OK || a->N == 0) return st;
  DeviceGuard g(ctx->device);
  AttnParams p;
  p.a = *a;
  p.p_shift = __builtin_ctz((unsigned)a->page_size);
  p.scale_log2 = a->scale * 1.44269504088896340736f;
  p.err = ctx->err;
  const dim3 grid((unsigned)(((int64_t)a->N * a->Hq + 3) / 4)), block(128);
  OpsPdl pdl;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (a->dtype == MOE_DT_BF16)
    e = a->D == 64 ? launch_pdl(attn_rows_kernel<MOE_DT_BF16, 64>, grid, block, 0, s, p)
                   : launch_pdl(attn_rows_kernel<MOE_DT_BF16, 128>, grid, block, 0, s, p);
  else
    e = a->D == 64 ? launch_pdl(attn_rows_kernel<MOE_DT_F16, 64>, grid, block, 0, s, p)
                   : launch_pdl(attn_rows_kernel<MOE_DT_F16, 128>, grid, block, 0, s, p);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_attn_get_error(moe_attn_ctx* ctx, uint32_t* bits) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  DeviceGuard g(ctx->device);
  uint32_t v = 0;
  if (cudaDeviceSynchronize() != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaMemcpy(&v, ctx->err, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaMemset(ctx->err, 0, sizeof(v)) != cudaSuccess) return MOE_ERR_CUDA;
  if (bits) *bits = v;
  return v ? MOE_ERR_DEVICE_FLAG : MOE_OK;
}

int64_t moe_attn_device_bytes(const moe_attn_ctx* ctx) { return ctx ? 256 : 0; }

int moe_attn_destroy(moe_attn_ctx* ctx) {
  if (!ctx) return MOE_OK;
  DeviceGuard g(ctx->device);
  cudaFree(ctx->err);
  delete ctx;
  return MOE_OK;
}

}  // extern "C"
