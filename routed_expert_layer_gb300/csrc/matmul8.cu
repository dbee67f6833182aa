// 8-bit projections: values to e4m3 with block scales, and the product of e4m3 activations and weights
// (interfaces and formulas: include/moe_ops_gb300.h).
#include <algorithm>
#include <type_traits>

#include "ops_internal.cuh"
#include "tc_ptx.cuh"

struct moe_matmul8_ctx {
  int device = 0;
  int sm_count = 0;
  void* mem = nullptr;
  size_t bytes = 0;
  size_t head_bytes = 0;  // error word and tickets
  uint32_t* err = nullptr;
  int32_t* tickets = nullptr;
  float* parts = nullptr;
};

namespace moe {

namespace {

// ---- quantisation ------------------------------------------------------------------------------

// Three kernels by the shape of a block, each with 16-byte loads where widths, strides and addresses allow it and single
// elements where not. Every value is read once and held in registers between the maximum and its quotient (rows wider than
// 32,768, or than 4,096 where they go by single elements, and unaligned 128 x 128 blocks are read again), so memory bounds them: 3 bytes
// an element.

// x / s, as division rounds it. Where s is neither tiny nor huge: Markstein's correction of q = x * (1 / s) by its remainder,
// two operations more than the product, instead of some ten. (The remainder is taken as q s - x: of a zero it is +0,
// and -0 * (1 / s) added to q keeps q's sign, where x - q s of x = -0 would turn -0 into +0.)
struct Quotient {
  float s, r;
  bool plain;
  __device__ __forceinline__ explicit Quotient(float scale) : s(scale), r(1.f / scale), plain(!(scale >= 0x1p-60f && scale < 0x1p100f)) {}
  template <bool PLAIN>
  __device__ __forceinline__ float at(float x) const {
    if constexpr (PLAIN) return s == 0.f ? 0.f : x / s;
    const float q = x * r;
    return fmaf(fmaf(q, s, -x), -r, q);
  }
  __device__ __forceinline__ uint8_t operator()(float x) const {
    return (uint8_t)(plain ? e4m3x2(at<true>(x), 0.f) : e4m3x2(at<false>(x), 0.f));
  }
  template <int DT, bool PLAIN>
  __device__ __forceinline__ uint2 piece(const uint4& w) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<DT>(u[i]);
      q[i] = e4m3x2(at<PLAIN>(f.x), at<PLAIN>(f.y));
    }
    return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
  }
  template <int DT>
  __device__ __forceinline__ uint2 piece(const uint4& w) const {  // 8 elements
    return plain ? piece<DT, true>(w) : piece<DT, false>(w);
  }
};

// Largest magnitudes, as 16-bit patterns without their signs: their order is that of the magnitudes, and a NaN is the largest.
__device__ __forceinline__ uint32_t top_bits(uint16_t w) { return w & 0x7FFFu; }
__device__ __forceinline__ uint32_t top_bits(const uint4& w) {
  const uint32_t k = 0x7FFF7FFFu, m = __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
  return max(m & 0xFFFFu, m >> 16);
}
template <int DT>
__device__ __forceinline__ float scale_of(uint32_t top) { return to_f32<DT>((uint16_t)top) / 448.f; }

// Blocks of 128 of a row: 8 lanes with two pieces of 8 elements each (or 32 with 4 single ones), two blocks in flight. The
// scale's two divisions are a lane's, so 16 elements share them. 8192 x 12288, bf16: 56 us, 5.4 TB/s; with one block in flight
// 63, four 74 us.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const moe_quantize8_args a, int nb) {
  constexpr int kLanes = WIDE ? 8 : 32, kAtOnce = 2, kEach = WIDE ? 2 : 4, kApart = WIDE ? 64 : 32;  // pieces of a lane, elements between
  using W = std::conditional_t<WIDE, uint4, uint16_t>;
  pdl_entry();
  const int lane = threadIdx.x & (kLanes - 1);
  const int64_t total = (int64_t)a.T * nb, step = (int64_t)gridDim.x * (256 / kLanes);
  const uint16_t* x = (const uint16_t*)a.x;
  // (the loop is the same for a warp's lanes: exchanges in it need them all)
  for (int64_t b0 = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / 32 * (32 / kLanes); b0 < total; b0 += kAtOnce * step) {
    W w[kAtOnce][kEach];
    int64_t row[kAtOnce];
    int at[kAtOnce];
    bool in[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t b = b0 + (threadIdx.x & 31) / kLanes + u * step;
      in[u] = b < total;
      row[u] = ((b | nb) >> 32) == 0 ? (uint32_t)b / (uint32_t)nb : b / nb;
      at[u] = (int)(b - row[u] * nb) * 128 + lane * (WIDE ? 8 : 1);
      const uint16_t* from = x + row[u] * a.x_stride + at[u];
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (in[u] && at[u] + kApart * i < a.H) w[u][i] = *reinterpret_cast<const W*>(from + kApart * i);
        else w[u][i] = W{};
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        m = max(m, top_bits(w[u][i]));
      }
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      if (!in[u]) continue;
      const float s = scale_of<DT>(m);
      const Quotient by(s);
      if (lane == 0) a.scales[row[u] * nb + (at[u] >> 7)] = s;
      uint8_t* to = a.out8 + row[u] * a.out8_stride + at[u];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (at[u] + kApart * i >= a.H) continue;
        if constexpr (WIDE) *reinterpret_cast<uint2*>(to + kApart * i) = by.piece<DT>(w[u][i]);
        else to[kApart * i] = by(to_f32<DT>(w[u][i]));
      }
    }
  }
}

// The largest of the block's values (of a warp's, where rows are a warp's).
__device__ __forceinline__ uint32_t threads_max(uint32_t m, bool one_warp, uint32_t* red) {
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (one_warp) return m;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = (threadIdx.x & 31) < blockDim.x >> 5 ? red[threadIdx.x & 31] : 0;
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  __syncthreads();
  return m;
}

// Whole rows: a row per block, or per warp (blockDim.y of them). 8192 x 12288, bf16: 64 us, 4.7 TB/s; 8192 x 12289, by single elements and read
// twice, 197 us.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(1024) quantize_rows_kernel(const moe_quantize8_args a) {
  constexpr int kHeld = 4, kPiece = WIDE ? 8 : 1;
  __shared__ uint32_t red[32];
  pdl_entry();
  const int tx = threadIdx.x, TX = blockDim.x, n = a.H / kPiece;
  for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < a.T; row += (int64_t)gridDim.x * blockDim.y) {
    const uint16_t* x = (const uint16_t*)a.x + row * a.x_stride;
    uint8_t* out = a.out8 + row * a.out8_stride;
    const auto load = [&](int i) {
      if constexpr (WIDE) return reinterpret_cast<const uint4*>(x)[i];
      else return x[i];
    };
    decltype(load(0)) held[kHeld];
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (tx + u * TX < n) held[u] = load(tx + u * TX);
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (tx + u * TX < n) m = max(m, top_bits(held[u]));
    for (int i = tx + kHeld * TX; i < n; i += TX) m = max(m, top_bits(load(i)));
    const float s = scale_of<DT>(threads_max(m, TX == 32, red));
    const Quotient by(s);
    if (tx == 0) a.scales[row] = s;
    const auto store = [&](int i, const auto& w) {
      if constexpr (WIDE) reinterpret_cast<uint2*>(out)[i] = by.piece<DT>(w);
      else out[i] = by(to_f32<DT>(w));
    };
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (tx + u * TX < n) store(tx + u * TX, held[u]);
    for (int i = tx + kHeld * TX; i < n; i += TX) store(i, load(i));
  }
}

// Blocks of 128 x 128: one per thread block, 8 pieces of 8 elements per thread. 14336 x 7168, bf16: 52 us, 5.9 TB/s.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const moe_quantize8_args a, int nb) {
  __shared__ uint32_t red[32];
  pdl_entry();
  const int tid = threadIdx.x;
  const int64_t total = (((int64_t)a.T + 127) / 128) * nb;
  for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
    const int64_t r0 = b / nb * 128;
    const int c0 = (int)(b % nb) * 128, height = (int)min((int64_t)128, a.T - r0), width = min(128, a.H - c0);
    const uint16_t* x = (const uint16_t*)a.x + r0 * a.x_stride + c0;
    uint8_t* out = a.out8 + r0 * a.out8_stride + c0;
    uint32_t m = 0;
    if constexpr (WIDE) {
      const int c = (tid & 15) * 8, r = tid >> 4;
      uint4 w[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        w[u] = make_uint4(0, 0, 0, 0);
        if (r + 16 * u < height && c < width) w[u] = *reinterpret_cast<const uint4*>(x + (r + 16 * u) * a.x_stride + c);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) m = max(m, top_bits(w[u]));
      const float s = scale_of<DT>(threads_max(m, false, red));
      const Quotient by(s);
      if (tid == 0) a.scales[b] = s;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (r + 16 * u < height && c < width)
          *reinterpret_cast<uint2*>(out + (r + 16 * u) * a.out8_stride + c) = by.piece<DT>(w[u]);
    } else {
      const int c = tid & 127, r = tid >> 7;
      for (int y = r; y < height; y += 2)
        if (c < width) m = max(m, top_bits(x[y * a.x_stride + c]));
      const float s = scale_of<DT>(threads_max(m, false, red));
      const Quotient by(s);
      if (tid == 0) a.scales[b] = s;
      for (int y = r; y < height; y += 2)
        if (c < width) out[y * a.out8_stride + c] = by(to_f32<DT>(x[y * a.x_stride + c]));
    }
  }
}

template <int DT, bool WIDE>
cudaError_t quantize(const moe_quantize8_args& a, cudaStream_t s) {
  const int nb = (a.H + 127) / 128;
  const int64_t resident = (int64_t)8 * sm_count();  // blocks of 256 threads
  if (a.rows == 128)
    return launch_pdl(quantize_tiles_kernel<DT, WIDE>, dim3((unsigned)std::min(((int64_t)a.T + 127) / 128 * nb, resident)), dim3(256),
                      0, s, a, nb);
  if (a.group == 128) {
    constexpr int kPerBlock = WIDE ? 32 : 8;
    return launch_pdl(quantize_blocks_kernel<DT, WIDE>,
                      dim3((unsigned)std::min(((int64_t)a.T * nb + kPerBlock - 1) / kPerBlock, resident)), dim3(256), 0, s, a, nb);
  }
  // the fewest threads that hold a row in four pieces each
  const int n = a.H / (WIDE ? 8 : 1), tx = n <= 128 ? 32 : n <= 1024 ? 256 : n <= 2048 ? 512 : 1024, ry = tx == 32 ? 8 : 1;
  return launch_pdl(quantize_rows_kernel<DT, WIDE>, dim3((unsigned)std::min(((int64_t)a.T + ry - 1) / ry, resident * 256 / (tx * ry))),
                    dim3(tx, ry), 0, s, a);
}

// ---- product -----------------------------------------------------------------------------------
//
// D (128 x BN per CTA, tokens in tensor memory's lanes) = A8 W8^T of one block of 128 along K, on the tensor cores; the
// epilogue warps multiply it by the block's two scales into fp32 registers while the next block's product
// is computed into another part of tensor memory: acc += (a_scale w_scale) D, one operation an element. The tensor cores take
// no fp32 scales of 128, and rounding them to powers of two would change the values.
//
// Two instances. One CTA takes 128 rows of W8 and 128 tokens: up to 128 tokens the weights are read once, streamed. A pair of
// CTAs takes 256 tokens and 256 rows of W8; its MMA reads each CTA's half of W8's rows from that CTA's shared memory, so each
// CTA loads 128 rows of A8 and 128 of W8 for 128 x 256 outputs. matmul8_plan estimates both.
//
// Work. A unit is a block of 128 of a tile. Whole rounds of tiles over all CTAs (or pairs) go tile by tile; the tiles
// left over, all of a small product, are laid on one axis of units and cut into stretches. The
// pieces of a tile go through the workspace and the warp that finishes last adds them in K's order (so results
// do not depend on which one that was), for its own 32 rows and its columns: no warp waits for another.
//
// Warps. 0: TMA (a stage: a unit's rows of A8 and W8). 1: issues the MMAs (of a pair: the first CTA's). 2, 3: bring the scales
// of 8 units at a time to shared memory (rows of scales are read along K, the epilogue wants them down the rows). 4..11:
// epilogue, a thread per row, half of the tile's columns each.
//
// Measured (bf16; the weights of a call not in L2). 8192 x 14336 x 7168 (tokens, outputs, K): 721 to 738 us, 2.3 PFLOP/s, 1.2
// times the bf16 rate. A pair's unit takes some 1,050 cycles where its products alone take 521 and its copies 660 (the copies
// with one MMA in four and no epilogue); without the loads of tensor memory 842: TMA's writes, the MMAs' operands, the
// epilogue's loads and every look at a barrier share the SM's memories, and no unit of it is full (tensor pipe 51 %, issue 41 %).
// 53 x 14336 x 7168: 21.3 us, 4.9 TB/s; 1 x 7168 x 12288 20.6 us. Their 112 CTAs stream at 5.9 to 6.6 TB/s beside some 4 us for the start
// and the end (53 tokens, 14,336 outputs, K of 3,584, 7,168, 14,336 and 28,672: 12.7, 21.3, 37.1 and 69.3 us); before
// two units were handed over at once, a unit's chain of accesses to shared memory bound them (each some 150 cycles while
// copies and MMAs keep it busy).
// On the way, 4096 x 14336 x 7168 (361 us then): every arrival on the other CTA released at cluster scope, which waits for the
// thread's stores, 1033; addresses spilled in the units' loop 384; steps of 128 columns with half a warp's columns in each 510;
// scalar products 392; one lane polling for its warp 424. 53 x 14336 x 7168 (23.9 then): weights in the lanes and tokens in the columns 31 us
// (a scale per column comes from shared memory; one token 25.1, then 26.9); tiles of 96 rows of W8, so that 150 CTAs work, 28.8;
// the next unit's scales read early 26.8.

using namespace ptx;

constexpr int kChunk = 8;       // units whose scales are fetched at a time
constexpr int kParked = 48;     // bytes of an epilogue warp's parked place
constexpr int kScaleRow = 132;  // a unit's row scales in shared memory: 128, and 4 so that lanes on 8 units meet in no bank

struct MatmulParams {
  moe_matmul8_args a;
  int kb;                  // units of a tile
  int m_tiles, n_tiles;
  int whole;               // tiles in whole rounds
  int units, cuts;         // units of the tiles left, stretches they are cut into
  int snap;                // a cut so near to a tile's border is moved there
  int stages, a_rows;      // rows of A8 in a stage
  int tma_out;             // out can be written by TMA
  uint32_t* err;
  int32_t* tickets;        // [tiles left][CG][warps], zero between calls
  float* parts;            // [CTAs][2] partial results: [warps][128 columns / 4][32 rows][4]
};

template <int CG_, int BN_, int DT_>
struct MatmulCfg {
  static constexpr int CG = CG_, BN = BN_, DT = DT_;
  static constexpr int kEpi = 8;                   // epilogue warps: 32 rows and half of the columns each
  static constexpr int kCols = BN / 2;
  static constexpr int kThreads = 128 + 32 * kEpi;
  static constexpr int kBlocks = BN / 128;         // blocks of W8's scales in a tile
  static constexpr int kBufs = 4;                  // products of 128 columns in tensor memory
  // Units whose products are handed to the epilogue at once. A look at a barrier costs it some 150 cycles, so where tensor
  // memory holds four units it is every other (53 x 14336 x 7168: 21.3 us for 23.9).
  static constexpr int kGroup = CG == 1 ? 2 : 1;
  static constexpr int kDeep = kBufs / kBlocks / kGroup;  // groups in tensor memory
  static constexpr int kPart = 128 * BN;
  static constexpr int kB = 128 * 128;             // bytes of W8 in a stage: 128 rows per CTA
  static_assert(BN == 128 * CG, "each CTA of a tile loads 128 rows of W8");
  static constexpr int kStaging = kEpi * 4096;
  static constexpr int kMaxStages = 12;
  static constexpr double kUnitUs = CG == 1 ? 0.30 : 0.54;  // a unit's time on the SM
  static constexpr int kScales = kChunk * (kScaleRow + BN / 128);  // floats of a chunk's scales
  // Shared memory. What the epilogue uses lies at constant places: addresses cost it no registers, and a spilled one in the
  // units' loop costs more than the arithmetic there.
  static constexpr int kScalesAt = 512, kParkedAt = kScalesAt + 2 * kScales * 4;
  static constexpr int kStagingAt = (kParkedAt + kParked * kEpi + 1023) / 1024 * 1024, kStagesAt = kStagingAt + kStaging;
  static constexpr int kFixed = 1024 + kStagesAt;
  // Registers: 384 threads of 168. Of a pair's kernel the first 128 give theirs up: 88 for them and 208 for the epilogue.
  static constexpr bool kMoveRegs = CG == 2;
};
constexpr int kSmemLimit = 232448;

struct Cuts {
  int units, cuts, snap, kb;
  __device__ __forceinline__ int at(int c) const {  // where stretch c starts
    if (c >= cuts) return units;
    const int u = units * c / cuts, in = u % kb;  // (below 2^31: K <= 2^20)
    return in <= snap ? u - in : kb - in <= snap ? u + kb - in : u;
  }
  // The stretches that hold a tile's first and last unit, by a whole warp: 8 lanes look at the stretches around each.
  __device__ __forceinline__ void owners(int tile, int& first, int& last) const {
    const int lane = threadIdx.x & 31, u = (lane & 8) ? (tile + 1) * kb - 1 : tile * kb;
    const int from = (int)((float)u * ((float)cuts / (float)units)) - 3, c = from + (lane & 7);
    const uint32_t begun = __ballot_sync(0xFFFFFFFFu, lane < 16 && c < cuts && (c <= 0 || at(c) <= u));
    first = __shfl_sync(0xFFFFFFFFu, from, 0) + __popc(begun & 0xFFu) - 1;
    last = __shfl_sync(0xFFFFFFFFu, from, 8) + __popc(begun & 0xFF00u) - 1;
  }
};

// The pieces of a CTA (or pair): whole tiles, then its stretch of the tiles left.
struct Walk {
  int tile, k0, k1;  // the piece
  int next_whole, u, u_end, step;
  __device__ __forceinline__ Walk(const MatmulParams& p, const Cuts& c, int id, int n) : next_whole(id), step(n) {
    u = c.at(id);
    u_end = c.at(id + 1);
  }
  __device__ __forceinline__ bool next(const MatmulParams& p) {
    if (next_whole < p.whole) {
      tile = next_whole;
      next_whole += step;
      k0 = 0;
      k1 = p.kb;
      return true;
    }
    if (u >= u_end) return false;
    const int t = u / p.kb;
    tile = p.whole + t;
    k0 = u - t * p.kb;
    k1 = min(p.kb, k0 + u_end - u);
    u += k1 - k0;
    return true;
  }
  // Tiles are ordered in bands of kBand rows of tiles, column by column: CTAs at work at the same time share rows and columns.
  __device__ __forceinline__ void place(const MatmulParams& p, int& m, int& n) const {
    constexpr int kBand = 8;
    const int band = tile / (kBand * p.n_tiles), height = min(kBand, p.m_tiles - band * kBand);
    const int in = tile - band * kBand * p.n_tiles;
    n = in / height;
    m = band * kBand + in - n * height;
  }
};

// mbar_wait by a whole warp, with one answer for all its lanes. (Its first look costs 15 cycles; mbar_wait_suspended's takes
// 94 for a barrier that is ready, and a unit's 512 cycles of products see several waits in a row.)
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint32_t* err) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, err));
}

__device__ __forceinline__ int load_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// c + a * b, two at a time in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    matmul8_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                   const __grid_constant__ CUtensorMap map_o, const __grid_constant__ MatmulParams p) {
  constexpr int CG = C::CG, BN = C::BN, DT = C::DT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  // the MMA reads 128 rows of A8 from a stage's start, whatever the stage holds: rows past a_rows are other
  // stages' and end in lanes that nobody reads
  const int a_bytes = p.a_rows * 128;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem);
  uint64_t *full = bar, *empty = full + C::kMaxStages, *acc_full = empty + C::kMaxStages, *acc_empty = acc_full + C::kBufs;
  uint64_t *scale_full = acc_empty + C::kBufs, *scale_empty = scale_full + 2, *drain = scale_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  float* scales = reinterpret_cast<float*>(smem + C::kScalesAt);  // [2][kChunk][kScaleRow | kBlocks]
  uint8_t* sa = smem + C::kStagesAt;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::kBufs; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 8);  // 4 warps of both CTAs, or 8 of one
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&scale_full[s], 2);
      mbar_init(&scale_empty[s], C::kEpi);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane < 3) prefetch_map(lane == 0 ? &map_a : lane == 1 ? &map_w : &map_o);
  if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, 512);
  tc_fence_before();
  if constexpr (CG == 1) __syncthreads();
  else cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const Cuts cuts{p.units, p.cuts, p.snap, p.kb};
  const int id = (int)(blockIdx.x / CG);
  Walk w(p, cuts, id, (int)(gridDim.x / CG));
  bool ok = true;
  int m, n;
  // While the kernel before this one ends, the first stages' weights come as far as L2 (which stays right whoever writes them).
  if (warp == 0 && elect_one()) {
    Walk ahead = w;
    if (ahead.next(p)) {
      ahead.place(p, m, n);
      for (int k = ahead.k0; k < min(ahead.k1, ahead.k0 + p.stages); ++k)
        for (int h = 0; h < C::kBlocks; ++h) prefetch_2d(&map_w, k * 128, n * BN + (int)rank * (128 / CG) + h * 128);
    }
  }
  __syncwarp();
  pdl_entry();

  if (warp >= 4) {
    if constexpr (C::kMoveRegs) regs_up<208>();
    const int e = warp - 4, quarter = warp & 3, part = e >> 2, block = CG == 1 ? 0 : part;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    uint8_t* stage = smem + C::kStagingAt + e * 4096;
    uint32_t groups = 0, chunks = 0;  // passed so far: their buffers and parities
    const uint32_t first_empty = CG == 1 ? 0 : cluster_addr(acc_empty, 0);
    const auto free_acc = [&](uint32_t at) {
      if constexpr (CG == 1) mbar_arrive(&acc_empty[at]);
      else mbar_arrive_cluster(first_empty + at * 8);
    };
    // the place on the work is out of the registers while units are added up
    struct Parked {
      Walk w;
      int first, last;  // the stretches of a cut tile's first and last piece
    };
    Parked* const parked = reinterpret_cast<Parked*>(smem + C::kParkedAt + e * kParked);
    static_assert(sizeof(Parked) <= kParked, "space of a parked place");
    while (ok && w.next(p)) {
      w.place(p, m, n);
      const bool live = (m * CG + (int)rank) * 128 + quarter * 32 < p.a.T;
      const int count = w.k1 - w.k0;
      int first = id, last = id;
      if (count < p.kb) cuts.owners(w.tile - p.whole, first, last);
      if (lane == 0) *parked = Parked{w, first, last};
      float2 acc[C::kCols / 2];
#pragma unroll
      for (int i = 0; i < C::kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int k = 0; k < count; k += C::kGroup, ++groups) {
        const int x = k & (kChunk - 1), bar_at = groups % C::kDeep * C::kBlocks + block;
        if (x == 0) ok = wait_warp(&scale_full[chunks & 1], chunks >> 1 & 1, p.err);
        const float* sc = scales + (chunks & 1) * C::kScales;
        // The product of the scales first, as the interface says it. (The sum times one scale after the other, in chunks where that product
        // leaves fp32's range, costs every call a look at each chunk: 8192 x 14336 x 7168 765 us for 722, 1 x 7168 x 12288 21.0 for 20.6.)
        float s[C::kGroup];
#pragma unroll
        for (int u = 0; u < C::kGroup; ++u)
          s[u] = sc[(x + u) * kScaleRow + quarter * 32 + lane] * sc[kChunk * kScaleRow + (x + u) * C::kBlocks + block];
        ok = ok && wait_warp(&acc_full[bar_at], groups / C::kDeep & 1, p.err);
        if (!ok) break;
        tc_fence_after();
        const auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) free_acc(bar_at);
        };
        if (live) {
          const uint32_t from = tmem + lane_base + bar_at * C::kGroup * 128 + (CG == 1 ? part * C::kCols : 0);
          const auto add_units = [&](auto n) {
            constexpr int kPer = C::kCols / 32, kAll = decltype(n)::value * kPer;  // chunks of 32 columns
            const auto at = [&](int c) { return from + c / kPer * 128 + c % kPer * 32; };
            float2 s2[C::kGroup];
#pragma unroll
            for (int u = 0; u < C::kGroup; ++u) s2[u] = make_float2(s[u], s[u]);
            uint32_t v[2][32];  // a load runs under the arithmetic of the one before
            tmem_ld32(from, v[0]);
#pragma unroll
            for (int c = 0; c < kAll; ++c) {
              tmem_wait_ld32(v[c & 1]);
              if (c + 1 < kAll) tmem_ld32(at(c + 1), v[(c + 1) & 1]);
              else release();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float2& sum = acc[c % kPer * 16 + i];
                sum = fma2(make_float2(__uint_as_float(v[c & 1][2 * i]), __uint_as_float(v[c & 1][2 * i + 1])), s2[c / kPer], sum);
              }
            }
          };
          if (C::kGroup == 1 || k + 1 < count) add_units(std::integral_constant<int, C::kGroup>());
          else add_units(std::integral_constant<int, 1>());
        } else {
          release();
        }
        if (x == kChunk - C::kGroup || k + C::kGroup >= count) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&scale_empty[chunks & 1]);
          ++chunks;
        }
      }
      if (!ok) break;
      __syncwarp();
      w = parked->w;
      first = parked->first;
      const int pieces = parked->last - first + 1;
      __syncwarp();
      if (!live) continue;
      w.place(p, m, n);
      const int row0 = (m * CG + (int)rank) * 128 + quarter * 32, col0 = n * BN + part * C::kCols;
      if (count < p.kb) {  // a piece: the last to finish adds the tile's pieces
        const int index = id - first;
        const auto part_of = [&](int i) {  // the i-th piece: a stretch's piece at a tile's start, or its other one
          return reinterpret_cast<float4*>(p.parts + ((int64_t)((first + i) * CG + (int)rank) * 2 + (i == 0 ? 1 : 0)) * C::kPart) +
                 e * (C::kCols * 8) + lane;
        };
        int32_t* ticket = p.tickets + ((w.tile - p.whole) * CG + (int)rank) * C::kEpi + e;
        const auto add = [&](int i, bool to_sum) {
          const float4* from = part_of(i);
#pragma unroll
          for (int c = 0; c < C::kCols / 4; c += 16) {
            float4 v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __ldcg(from + (c + j) * 32);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float2 &a = acc[2 * (c + j)], &b = acc[2 * (c + j) + 1];
              a = to_sum ? make_float2(a.x + v[j].x, a.y + v[j].y) : make_float2(v[j].x, v[j].y);
              b = to_sum ? make_float2(b.x + v[j].z, b.y + v[j].w) : make_float2(v[j].z, v[j].w);
            }
          }
        };
        int done = 0;
        // Where the others are done already, this piece need not be written: looked up where no more work waits for this
        // warp. (In the sum's order it has to be one of the first two, which may change places.)
        if (lane == 0 && index < 2 && w.u >= w.u_end) done = load_acquire(ticket);
        done = __shfl_sync(0xFFFFFFFFu, done, 0);
        __syncwarp();  // what lane 0 has acquired is the warp's
        if (done == pieces - 1) {
          for (int i = 0; i < pieces; ++i)
            if (i != index) add(i, true);
        } else {
          float4* mine = part_of(index);
          if (row0 + lane < p.a.T)
#pragma unroll
            for (int c = 0; c < C::kCols / 4; ++c)
              mine[c * 32] = make_float4(acc[2 * c].x, acc[2 * c].y, acc[2 * c + 1].x, acc[2 * c + 1].y);
          __threadfence();
          __syncwarp();
          if (lane == 0) done = atomicAdd(ticket, 1);
          if (__shfl_sync(0xFFFFFFFFu, done, 0) != pieces - 1) continue;
          __threadfence();
          add(0, false);
          for (int i = 1; i < pieces; ++i) add(i, true);
        }
        if (lane == 0) *ticket = 0;
      }
      // 64 columns at a time through shared memory: a row of 128 bytes per lane, 16-byte pieces swizzled by row
#pragma unroll
      for (int h = 0; h < C::kCols / 64; ++h) {
        const int col = col0 + h * 64;
        if (col >= p.a.N) break;
        if (lane == 0) bulk_wait_read();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2* f = acc + h * 32 + j * 4;
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
              make_uint4(pack2<DT>(f[0].x, f[0].y), pack2<DT>(f[1].x, f[1].y), pack2<DT>(f[2].x, f[2].y), pack2<DT>(f[3].x, f[3].y));
        }
        if (p.tma_out) {
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&map_o, stage, col, row0);
            bulk_commit();
          }
        } else {
          __syncwarp();
          uint16_t* out = (uint16_t*)p.a.out + (int64_t)row0 * p.a.out_stride + col;
          const int rows = min(32, p.a.T - row0), cols = min(64, p.a.N - col);
          for (int r = 0; r < rows; ++r, out += p.a.out_stride)
#pragma unroll
            for (int x = 0; x < 64; x += 32) {
              const int at = x + lane;
              if (at < cols) out[at] = *reinterpret_cast<const uint16_t*>(stage + r * 128 + (((at >> 3) ^ (r & 7)) << 4) + (at & 7) * 2);
            }
        }
      }
    }
    if (lane == 0) bulk_wait_read();  // shared memory goes away
    __syncwarp();
  } else {
    if constexpr (C::kMoveRegs) regs_down<88>();
    uint8_t* sw = sa + (size_t)p.stages * a_bytes;
    if (warp == 0) {
      if (elect_one()) {
        uint32_t s = 0, turn = 0;
        while (ok && w.next(p)) {
          w.place(p, m, n);
          const int row = (m * CG + (int)rank) * 128, col = n * BN + (int)rank * (128 / CG);
          for (int k = w.k0; k < w.k1; ++k) {
            ok = mbar_wait(&empty[s], turn ^ 1u, p.err);
            if (!ok) break;
            if constexpr (CG == 1) {
              mbar_arrive_expect_tx(&full[s], a_bytes + C::kB);
              tma_2d(sw + s * C::kB, &map_w, k * 128, col, &full[s]);
              tma_2d(sa + s * a_bytes, &map_a, k * 128, row, &full[s]);
            } else {
              // both CTAs' bytes are counted where the MMAs are issued
              if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (a_bytes + C::kB));
              const uint32_t to = cluster_addr(&full[s], 0);
              tma_2d_pair(sw + s * C::kB, &map_w, k * 128, col, to);
              tma_2d_pair(sw + s * C::kB + C::kB / 2, &map_w, k * 128, col + 128, to);
              tma_2d_pair(sa + s * a_bytes, &map_a, k * 128, row, to);
            }
            if (++s == (uint32_t)p.stages) s = 0, turn ^= 1u;
          }
        }
        if (!ok) {  // copies in flight land long before this, and before shared memory goes away
          const uint64_t t0 = globaltimer();
          while (globaltimer() - t0 < 2000000) {
          }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (rank == 0 && elect_one()) {
        constexpr uint32_t kId = idesc_e4m3(128 * CG, 128);
        const uint64_t da = desc_sw128(smem_u32(sa)), dw = desc_sw128(smem_u32(sw));
        uint32_t s = 0, turn = 0, buf = 0, buf_turn = 0;
        while (ok && w.next(p)) {
          for (int k = w.k0; k < w.k1; k += C::kGroup) {
#pragma unroll
            for (int u = 0; u < C::kGroup; ++u) {
              if (u && k + u >= w.k1) break;
              ok = ok && mbar_wait(&full[s], turn, p.err);
              const uint64_t a = da + ((uint32_t)(s * a_bytes) >> 4), b = dw + ((uint32_t)(s * C::kB) >> 4);
#pragma unroll
              for (int h = 0; h < C::kBlocks; ++h) {
                if (u == 0) ok = ok && mbar_wait(&acc_empty[buf + h], buf_turn ^ 1u, p.err);
                if (!ok) break;
                tc_fence_after();
                const uint32_t to = tmem + ((buf + h) * C::kGroup + u) * 128;
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_f8_ss<CG>(to, a + j * 2, b + h * (C::kB >> 5) + j * 2, kId, j > 0);
                if (h + 1 == C::kBlocks) mma_commit_cg<CG>(&empty[s]);
                if (C::kGroup == 1) mma_commit_cg<CG>(&acc_full[buf + h]);
              }
              if (!ok) break;
              if (++s == (uint32_t)p.stages) s = 0, turn ^= 1u;
            }
            if (!ok) break;
            if (C::kGroup > 1) mma_commit_cg<CG>(&acc_full[buf]);
            buf += C::kBlocks;
            if (buf == C::kDeep * C::kBlocks) buf = 0, buf_turn ^= 1u;
          }
        }
        mma_commit_cg<CG>(drain);  // every MMA issued, and every arrival on the other CTA's barriers, is through
      }
      __syncwarp();
      if (rank == 0) mbar_wait(drain, 0, p.err);
    } else {
      uint32_t buf = 0, turn = 0;
      const int x = lane & (kChunk - 1), y = lane / kChunk;  // unit and row of a lane
      constexpr int kRows = 32 / kChunk;
      const int row_first = (warp - 2) * 64 + y;  // each of the two warps takes 64 rows
      while (ok && w.next(p)) {
        w.place(p, m, n);
        const int row0 = (m * CG + (int)rank) * 128, rows = min(128, p.a.T - row0), block0 = n * C::kBlocks;
        for (int k = w.k0; k < w.k1; k += kChunk) {
          ok = wait_warp(&scale_empty[buf], turn ^ 1u, p.err);
          if (!ok) break;
          float* to = scales + buf * C::kScales + x * kScaleRow;
          const bool in = k + x < w.k1;
          const float* from = p.a.a_scales + (int64_t)row0 * p.a.a_scales_stride + (p.a.a_blocks > 1 ? k + x : 0);
          float v[64 / kRows];
#pragma unroll
          for (int i = 0; i < 64 / kRows; ++i) {
            const int r = row_first + i * kRows;
            v[i] = in && r < rows ? __ldg(from + r * p.a.a_scales_stride) : 0.f;
          }
#pragma unroll
          for (int i = 0; i < 64 / kRows; ++i) to[row_first + i * kRows] = v[i];
          if (warp == 2 && y < C::kBlocks)
            scales[buf * C::kScales + kChunk * kScaleRow + x * C::kBlocks + y] =
                in && block0 + y <= (p.a.N - 1) >> 7 ? __ldg(p.a.w_scales + (block0 + y) * p.a.w_scales_stride + k + x) : 0.f;
          __syncwarp();
          if (lane == 0) mbar_arrive(&scale_full[buf]);
          if (++buf == 2) buf = 0, turn ^= 1u;
        }
      }
    }
  }
  tc_fence_before();
  if constexpr (CG == 1) __syncthreads();
  else cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    // The arrival of the last commit on the second CTA's barrier, before its shared memory goes away. The first CTA has seen its own, so
    // this takes no time; waited for instead of the work, it would give up in a product that runs for longer than a wait may.
    // (The rank is read again: kept in its register until here, 8192 x 14336 x 7168 takes 760 us instead of 728.)
    if (CG > 1 && cluster_rank() != 0) mbar_wait(drain, 0, p.err);
    __syncwarp();
    tmem_dealloc_cg<CG>(tmem, 512);
  }
}

// A matrix [rows][width] of 1- or 2-byte elements in boxes of box_rows x 128 bytes with 128-byte swizzle.
bool make_map2(CUtensorMap* map, const void* base, CUtensorMapDataType type, int size, int64_t rows, int64_t width,
               int64_t stride, int box_rows) {
  const TensorMapFn encode = tensor_map_fn();
  if (!encode) return false;
  const cuuint64_t d[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  // the stride of a single row is never used; TMA still wants a valid one
  const cuuint64_t s[1] = {(cuuint64_t)(rows == 1 ? (width * size + 15) / 16 * 16 : stride * size)};
  const cuuint32_t b[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows}, e[2] = {1, 1};
  return encode(map, type, 2, const_cast<void*>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
bool matmul8_configure() {
  return cudaFuncSetAttribute(matmul8_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) == cudaSuccess;
}

// How a product is shared out: tiles in whole rounds over the CTAs (or pairs), and the stretches into which the units of the
// tiles left over are cut: every tile into the same number of pieces, or all units into as many stretches as there are CTAs,
// whose borders then lie inside tiles. The estimates, in us, are of this card: a unit takes what its products do or, of weights
// that stream from memory, its bytes' share; the pieces of a tile are written and read again; and a stretch that goes on in
// a second tile stalls for its first piece's way out. (517 x 1811 x 7152: 75 tiles of single CTAs in two pieces each 19.8 us,
// 24 of pairs in three 24.1; 256 x 14336 x 7168 33.5 and 36.7; 4096 x 14336 x 7168 395 and 363.)
struct MatmulPlan {
  int64_t m_tiles, n_tiles;
  int most, left, cuts;
  double us;
};
template <class C>
MatmulPlan matmul8_plan(const moe_matmul8_args& a, int sm_count) {
  MatmulPlan p;
  p.m_tiles = ((int64_t)a.T + 128 * C::CG - 1) / (128 * C::CG);
  p.n_tiles = ((int64_t)a.N + C::BN - 1) / C::BN;
  p.most = sm_count / C::CG;
  const int64_t tiles = p.m_tiles * p.n_tiles, kb = (a.K + 127) / 128;
  p.left = (int)(tiles % p.most);
  p.us = (double)(tiles / p.most * kb) * C::kUnitUs;
  p.cuts = 0;
  if (p.left == 0) return p;
  const int64_t units = p.left * kb;
  const auto cost = [&](int64_t cuts) {
    const double stretch = (double)((units + cuts - 1) / cuts);
    const double each = std::max(C::kUnitUs, (double)(cuts * C::CG) * C::kB / (double)p.m_tiles / 6.5e6);
    const bool inside = cuts % p.left != 0;
    const double pieces = inside ? (double)kb / stretch + 1 : (double)(cuts / p.left);
    return stretch * each + (pieces > 1 ? 2.0 + 0.6 * pieces : 0.0) + (inside ? 2.5 : 0.0);
  };
  p.cuts = p.left;
  for (int64_t cuts = 2 * p.left; cuts <= p.most && cuts <= units; cuts += p.left)
    if (cost(cuts) < cost(p.cuts)) p.cuts = (int)cuts;
  if (units >= p.most && cost(p.most) < cost(p.cuts)) p.cuts = p.most;
  p.us += cost(p.cuts);
  return p;
}

template <class C>
int matmul8_launch(const moe_matmul8_ctx* ctx, const moe_matmul8_args& a, const MatmulPlan& plan, cudaStream_t stream) {
  MatmulParams p;
  p.a = a;
  p.kb = (a.K + 127) / 128;
  const int64_t tiles = plan.m_tiles * plan.n_tiles;  // (2^30 at most: matmul8_check)
  p.m_tiles = (int)plan.m_tiles;
  p.n_tiles = (int)plan.n_tiles;
  p.whole = (int)tiles - plan.left;
  p.units = plan.left * p.kb;
  p.cuts = plan.cuts;
  p.snap = p.cuts ? p.units / p.cuts / 16 : 0;
  p.a_rows = (int)std::min<int64_t>(128, (a.T + 7) / 8 * 8);
  p.stages = std::min(C::kMaxStages, (kSmemLimit - C::kFixed) / (p.a_rows * 128 + C::kB));
  p.tma_out = is_aligned(a.out, 16) && (a.T == 1 || a.out_stride % 8 == 0);
  p.err = ctx->err;
  p.tickets = ctx->tickets;
  p.parts = ctx->parts;
  CUtensorMap ma, mw, mo = {};
  if (!make_map2(&ma, a.a8, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.T, a.K, a.a8_stride, p.a_rows) ||
      !make_map2(&mw, a.w8, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.N, a.K, a.w8_stride, 128 / C::CG) ||
      (p.tma_out && !make_map2(&mo, a.out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.T, a.N, a.out_stride, 32)))
    return MOE_ERR_CUDA;
  const int ctas = (p.whole ? plan.most : p.cuts) * C::CG;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = C::CG;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kFixed + (size_t)p.stages * (p.a_rows * 128 + C::kB);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = C::CG > 1 ? 2 : 1;
  void* args[] = {&ma, &mw, &mo, &p};
  return cudaLaunchKernelExC(&cfg, (const void*)matmul8_kernel<C>, args) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int DT>
using StreamMatmul = MatmulCfg<1, 128, DT>;
template <int DT>
using PairMatmul = MatmulCfg<2, 256, DT>;

template <int DT>
int matmul8_by_rows(const moe_matmul8_ctx* ctx, const moe_matmul8_args& a, cudaStream_t s) {
  const MatmulPlan one = matmul8_plan<StreamMatmul<DT>>(a, ctx->sm_count), two = matmul8_plan<PairMatmul<DT>>(a, ctx->sm_count);
  if (a.T <= 128 || one.us < two.us) return matmul8_launch<StreamMatmul<DT>>(ctx, a, one, s);
  return matmul8_launch<PairMatmul<DT>>(ctx, a, two, s);
}

// Bytes a strided [rows][width] tensor spans.
Span span2(const void* p, int64_t rows, int64_t stride, int64_t width, int size) {
  const char* b = (const char*)p;
  return {b, b + size * ((rows - 1) * stride + width)};
}

// Clears the error word and the tickets, and waits for it (streams need not wait for the default one).
bool clear_head(const moe_matmul8_ctx* c) {
  return cudaMemset(c->mem, 0, c->head_bytes) == cudaSuccess && cudaStreamSynchronize(cudaStreamLegacy) == cudaSuccess;
}

int matmul8_check(const moe_matmul8_args* a) {
  if (!a || a->T < 0 || a->N < 0 || a->K < 16 || a->K % 16 || (a->dtype != MOE_DT_BF16 && a->dtype != MOE_DT_F16))
    return MOE_ERR_INVALID_ARG;
  const int blocks = (a->K + 127) / 128;
  if (a->a_blocks != blocks && a->a_blocks != 1) return MOE_ERR_INVALID_ARG;
  const int64_t wb = ((int64_t)a->N + 127) / 128;
  if (a->K > 1 << 20 || a->T > 1 << 30 || a->N > 1 << 30 || ((int64_t)a->T + 127) / 128 * wb > 1 << 30)
    return MOE_ERR_UNSUPPORTED;
  if (a->T == 0 || a->N == 0) return MOE_OK;
  if (!a->a8 || !a->w8 || !a->a_scales || !a->w_scales || !a->out || !is_aligned(a->a8, 16) || !is_aligned(a->w8, 16) ||
      !is_aligned(a->a_scales, 4) || !is_aligned(a->w_scales, 4) || !is_aligned(a->out, 2))
    return MOE_ERR_INVALID_ARG;
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
  if (a->H > 1 << 30) return MOE_ERR_UNSUPPORTED;
  if (a->T == 0) return MOE_OK;
  if (!a->x || !a->out8 || !a->scales || !is_aligned(a->x, 2) || !is_aligned(a->scales, 4)) return MOE_ERR_INVALID_ARG;
  if (a->T > 1 && (a->x_stride < a->H || a->out8_stride < a->H)) return MOE_ERR_INVALID_ARG;
  const int group = a->group ? a->group : a->H;
  const int64_t blocks = (((int64_t)a->T + a->rows - 1) / a->rows) * (((int64_t)a->H + group - 1) / group);
  const Span x = span2(a->x, a->T, a->x_stride, a->H, 2), o = span2(a->out8, a->T, a->out8_stride, a->H, 1);
  const Span s = span2(a->scales, 1, 0, blocks, 4);
  if (overlap(x, o) || overlap(x, s) || overlap(o, s)) return MOE_ERR_INVALID_ARG;
  OpsPdl pdl;
  const auto fits = [&](int64_t rows, int64_t stride) { return rows == 1 || stride % 8 == 0; };
  const bool wide = a->H % 8 == 0 && is_aligned(a->x, 16) && is_aligned(a->out8, 8) && fits(a->T, a->x_stride) && fits(a->T, a->out8_stride);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = a->dtype == MOE_DT_BF16 ? (wide ? quantize<MOE_DT_BF16, true>(*a, st) : quantize<MOE_DT_BF16, false>(*a, st))
                                                : (wide ? quantize<MOE_DT_F16, true>(*a, st) : quantize<MOE_DT_F16, false>(*a, st));
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
  // error word | tickets (of each tile left over, its CTAs' epilogue warps) | partial results (two per CTA)
  c->head_bytes = (256 + (size_t)c->sm_count * PairMatmul<0>::kEpi * 4 + 255) / 256 * 256;
  c->bytes = c->head_bytes + 2 * (size_t)c->sm_count * sizeof(float) * PairMatmul<0>::kPart;
  if (cudaMalloc(&c->mem, c->bytes) != cudaSuccess) {
    cudaGetLastError();
    delete c;
    return MOE_ERR_OOM;
  }
  c->err = (uint32_t*)c->mem;
  c->tickets = (int32_t*)((char*)c->mem + 256);
  c->parts = (float*)((char*)c->mem + c->head_bytes);
  if (!clear_head(c) || !matmul8_configure<StreamMatmul<MOE_DT_BF16>>() || !matmul8_configure<StreamMatmul<MOE_DT_F16>>() ||
      !matmul8_configure<PairMatmul<MOE_DT_BF16>>() || !matmul8_configure<PairMatmul<MOE_DT_F16>>()) {
    cudaGetLastError();
    cudaFree(c->mem);
    delete c;
    return MOE_ERR_CUDA;
  }
  *out = c;
  return MOE_OK;
}

int moe_matmul8_forward(moe_matmul8_ctx* ctx, void* stream, const moe_matmul8_args* a) {
  const int st = matmul8_check(a);
  if (st == MOE_OK && !ctx) return MOE_ERR_INVALID_ARG;
  if (st != MOE_OK || a->T == 0 || a->N == 0) return st;
  DeviceGuard g(ctx->device);
  return a->dtype == MOE_DT_BF16 ? matmul8_by_rows<MOE_DT_BF16>(ctx, *a, (cudaStream_t)stream)
                                 : matmul8_by_rows<MOE_DT_F16>(ctx, *a, (cudaStream_t)stream);
}

int moe_matmul8_get_error(moe_matmul8_ctx* ctx, uint32_t* bits) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  DeviceGuard g(ctx->device);
  uint32_t v = 0;
  if (cudaDeviceSynchronize() != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaMemcpy(&v, ctx->err, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return MOE_ERR_CUDA;
  if (v && !clear_head(ctx)) return MOE_ERR_CUDA;
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
