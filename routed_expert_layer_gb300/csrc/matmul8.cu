// 8-bit projections: values to e4m3 with block scales, and the product of e4m3 activations and weights
// (interfaces and formulas: include/moe_ops_gb300.h).
#include <algorithm>

#include <cuda_fp8.h>

#include "ops_internal.cuh"
#include "tc_ptx.cuh"

struct moe_matmul8_ctx {
  int device = 0;
  int sm_count = 0;
  void* mem = nullptr;
  size_t bytes = 0;
  uint32_t* err = nullptr;
};

namespace moe {

namespace {

// ---- quantisation ------------------------------------------------------------------------------

// One block per block of values, read twice.
template <int DT>
__global__ void __launch_bounds__(256) quantize_kernel(const moe_quantize8_args a, int group) {
  __shared__ uint32_t s_max[8];
  pdl_entry();
  const int tid = threadIdx.x, nb = (a.H + group - 1) / group;
  const int64_t total = (int64_t)((a.T + a.rows - 1) / a.rows) * nb;
  for (int64_t at = blockIdx.x; at < total; at += gridDim.x) {
    const int64_t br = at / nb;
    const int bc = (int)(at - br * nb), c0 = bc * group, width = min(group, a.H - c0);
    const int64_t r0 = br * a.rows;
    const int height = (int)min((int64_t)a.rows, a.T - r0), n = height * width;
    uint32_t m = 0;
    for (int i = tid; i < n; i += 256) {
      const int r = i / width, c = i - r * width;
      m = max(m, abs_bits(to_f32<DT>(((const uint16_t*)a.x)[(r0 + r) * a.x_stride + c0 + c])));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((tid & 31) == 0) s_max[tid >> 5] = m;
    __syncthreads();
    m = 0;
    for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
    __syncthreads();
    const float s = __uint_as_float(m) / 448.f;
    if (tid == 0) a.scales[at] = s;
    for (int i = tid; i < n; i += 256) {
      const int r = i / width, c = i - r * width;
      const float v = to_f32<DT>(((const uint16_t*)a.x)[(r0 + r) * a.x_stride + c0 + c]);
      a.out8[(r0 + r) * a.out8_stride + c0 + c] = (uint8_t)e4m3x2(m ? v / s : 0.f, 0.f);
    }
  }
}

// ---- product -----------------------------------------------------------------------------------

constexpr int kTile = 64;

// 64 x 64 outputs per block, 4 x 4 per thread, values as fp32 in shared memory.
template <int DT>
__global__ void __launch_bounds__(256) matmul8_kernel(const moe_matmul8_args a) {
  __shared__ float sa[32][kTile + 1], sw[32][kTile + 1];
  pdl_entry();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * kTile;
  for (int64_t t0 = (int64_t)blockIdx.y * kTile; t0 < a.T; t0 += (int64_t)gridDim.y * kTile) {
    float acc[4][4] = {};
    for (int k0 = 0, kb = 0; k0 < a.K; k0 += 128, ++kb) {
      float part[4][4] = {};
      for (int k1 = k0; k1 < min(k0 + 128, a.K); k1 += 32) {
        __syncthreads();
        for (int i = tid; i < kTile * 32; i += 256) {
          const int r = i >> 5, c = i & 31;
          const bool in = k1 + c < a.K;
          __nv_fp8_e4m3 x, w;
          x.__x = in && t0 + r < a.T ? a.a8[(t0 + r) * a.a8_stride + k1 + c] : 0;
          w.__x = in && n0 + r < a.N ? a.w8[(n0 + r) * a.w8_stride + k1 + c] : 0;
          sa[c][r] = (float)x;
          sw[c][r] = (float)w;
        }
        __syncthreads();
        for (int c = 0; c < 32; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sa[c][ty * 4 + i], sw[c][tx + 16 * j], part[i][j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + ty * 4 + i;
        const float as = t < a.T ? a.a_scales[t * a.a_scales_stride + (a.a_blocks > 1 ? kb : 0)] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t n = n0 + tx + 16 * j;
          const float ws = n < a.N ? a.w_scales[(n >> 7) * a.w_scales_stride + kb] : 0.f;
          acc[i][j] = fmaf(part[i][j], as * ws, acc[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + ty * 4 + i, n = n0 + tx + 16 * j;
        if (t < a.T && n < a.N) ((uint16_t*)a.out)[t * a.out_stride + n] = from_f32<DT>(acc[i][j]);
      }
  }
}

// Bytes a strided [rows][width] tensor spans.
Span span2(const void* p, int64_t rows, int64_t stride, int64_t width, int size) {
  const char* b = (const char*)p;
  return {b, b + size * ((rows - 1) * stride + width)};
}

bool clear_error(const moe_matmul8_ctx* c) {
  return cudaMemset(c->mem, 0, 256) == cudaSuccess && cudaStreamSynchronize(cudaStreamLegacy) == cudaSuccess;
}

int matmul8_check(const moe_matmul8_args* a) {
  if (!a || a->T < 0 || a->N < 0 || a->K < 16 || a->K % 16 || (a->dtype != MOE_DT_BF16 && a->dtype != MOE_DT_F16))
    return MOE_ERR_INVALID_ARG;
  const int blocks = (a->K + 127) / 128;
  if (a->a_blocks != blocks && a->a_blocks != 1) return MOE_ERR_INVALID_ARG;
  if (a->T == 0 || a->N == 0) return MOE_OK;
  if (!a->a8 || !a->w8 || !a->a_scales || !a->w_scales || !a->out || !is_aligned(a->a8, 16) || !is_aligned(a->w8, 16) ||
      !is_aligned(a->a_scales, 4) || !is_aligned(a->w_scales, 4) || !is_aligned(a->out, 2))
    return MOE_ERR_INVALID_ARG;
  const int64_t wb = ((int64_t)a->N + 127) / 128;
  const auto short_rows = [](int64_t rows, int64_t stride, int64_t width) { return rows > 1 && stride < width; };
  if (short_rows(a->T, a->a8_stride, a->K) || short_rows(a->N, a->w8_stride, a->K) || short_rows(a->T, a->out_stride, a->N) ||
      short_rows(a->T, a->a_scales_stride, a->a_blocks) || short_rows(wb, a->w_scales_stride, blocks) ||
      (a->T > 1 && a->a8_stride % 16) || (a->N > 1 && a->w8_stride % 16))
    return MOE_ERR_INVALID_ARG;
  const Span out = span2(a->out, a->T, a->out_stride, a->N, 2);
  if (overlap(out, span2(a->a8, a->T, a->a8_stride, a->K, 1)) || overlap(out, span2(a->w8, a->N, a->w8_stride, a->K, 1)) ||
      overlap(out, span2(a->a_scales, a->T, a->a_scales_stride, a->a_blocks, 4)) ||
      overlap(out, span2(a->w_scales, wb, a->w_scales_stride, blocks, 4)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_quantize8(void* stream, const moe_quantize8_args* a) {
  if (!a || a->T < 0 || a->H < 1 || (a->dtype != MOE_DT_BF16 && a->dtype != MOE_DT_F16)) return MOE_ERR_INVALID_ARG;
  if (!(a->group == 128 && (a->rows == 1 || a->rows == 128)) && !(a->group == 0 && a->rows == 1)) return MOE_ERR_INVALID_ARG;
  if (a->T == 0) return MOE_OK;
  if (!a->x || !a->out8 || !a->scales || !is_aligned(a->x, 2) || !is_aligned(a->scales, 4)) return MOE_ERR_INVALID_ARG;
  if (a->T > 1 && (a->x_stride < a->H || a->out8_stride < a->H)) return MOE_ERR_INVALID_ARG;
  const int group = a->group ? a->group : a->H;
  const int64_t blocks = (((int64_t)a->T + a->rows - 1) / a->rows) * (((int64_t)a->H + group - 1) / group);
  const Span x = span2(a->x, a->T, a->x_stride, a->H, 2), o = span2(a->out8, a->T, a->out8_stride, a->H, 1);
  const Span s = span2(a->scales, 1, 0, blocks, 4);
  if (overlap(x, o) || overlap(x, s) || overlap(o, s)) return MOE_ERR_INVALID_ARG;
  OpsPdl pdl;
  const dim3 grid((unsigned)std::min<int64_t>(blocks, (int64_t)8 * sm_count()));
  const cudaError_t e = a->dtype == MOE_DT_BF16
                            ? launch_pdl(quantize_kernel<MOE_DT_BF16>, grid, dim3(256), 0, (cudaStream_t)stream, *a, group)
                            : launch_pdl(quantize_kernel<MOE_DT_F16>, grid, dim3(256), 0, (cudaStream_t)stream, *a, group);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_matmul8_create(int device, moe_matmul8_ctx** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess) return MOE_ERR_CUDA;
  if (device < 0 || device >= ndev) return MOE_ERR_INVALID_ARG;
  cudaDeviceProp prop;
  if (cudaGetDeviceProperties(&prop, device) != cudaSuccess) return MOE_ERR_CUDA;
  if (!(prop.major == 10 && prop.minor == 3)) return MOE_ERR_UNSUPPORTED;
  DeviceGuard g(device);
  moe_matmul8_ctx* c = new (std::nothrow) moe_matmul8_ctx();
  if (!c) return MOE_ERR_OOM;
  c->device = device;
  c->sm_count = prop.multiProcessorCount;
  c->bytes = 256;
  if (cudaMalloc(&c->mem, c->bytes) != cudaSuccess) {
    cudaGetLastError();
    delete c;
    return MOE_ERR_OOM;
  }
  c->err = (uint32_t*)c->mem;
  if (!clear_error(c)) {
    cudaGetLastError();
    cudaFree(c->mem);
    delete c;
    return MOE_ERR_CUDA;
  }
  *out = c;
  return MOE_OK;
}

int moe_matmul8_forward(moe_matmul8_ctx* ctx, void* stream, const moe_matmul8_args* a) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  const int st = matmul8_check(a);
  if (st != MOE_OK || a->T == 0 || a->N == 0) return st;
  DeviceGuard g(ctx->device);
  OpsPdl pdl;
  const dim3 grid((unsigned)((a->N + kTile - 1) / kTile), (unsigned)std::min((a->T + kTile - 1) / kTile, 65535));
  const cudaError_t e = a->dtype == MOE_DT_BF16
                            ? launch_pdl(matmul8_kernel<MOE_DT_BF16>, grid, dim3(256), 0, (cudaStream_t)stream, *a)
                            : launch_pdl(matmul8_kernel<MOE_DT_F16>, grid, dim3(256), 0, (cudaStream_t)stream, *a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_matmul8_get_error(moe_matmul8_ctx* ctx, uint32_t* bits) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  DeviceGuard g(ctx->device);
  uint32_t v = 0;
  if (cudaDeviceSynchronize() != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaMemcpy(&v, ctx->err, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return MOE_ERR_CUDA;
  if (v && !clear_error(ctx)) return MOE_ERR_CUDA;
  if (bits) *bits = v;
  return v ? MOE_ERR_DEVICE_FLAG : MOE_OK;
}

int64_t moe_matmul8_device_bytes(const moe_matmul8_ctx* ctx) { return ctx ? (int64_t)ctx->bytes : 0; }

int moe_matmul8_destroy(moe_matmul8_ctx* ctx) {
  if (!ctx) return MOE_OK;
  DeviceGuard g(ctx->device);
  cudaFree(ctx->mem);
  delete ctx;
  return MOE_OK;
}

}  // extern "C"
