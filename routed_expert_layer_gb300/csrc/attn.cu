// Attention of new tokens over a paged cache (interface and formula: include/moe_ops_gb300.h),
// on the tensor cores.
//
//   S = Q K^T (rows: a tile's (token, query head) pairs of one key head; columns: keys)
//   P = exp2(scale log2(e) (S - m)), l = sum of P, O = P V, out = O / l
// with m the running row maximum. One pass over the keys; S, P and O live in tensor memory.
//
// Rows. The G = Hq / Hkv query heads that share a key head are packed with the tokens: row r
// of a tile is token r / G, head r % G, TPT = tokens per tile of 128 rows. An item is one
// (request, key head, QT tiles): all its rows read the same keys.
//
// Work. The items, in the order request, key head, tile, lie on one axis on which an item is
// as long as the keys it reads plus a constant for its start and end. Every CTA takes an
// equal stretch of the axis, whatever mix of chunk lengths and contexts the call has; an item
// that crosses a boundary is computed in pieces whose (m, l, O) go through the workspace, and
// the CTA that finishes an item's last piece joins them in key order, many pieces in runs first (so the
// result does not depend on which one that was). The axis is laid out from the lengths by every CTA itself.
//
// Warps. 0: TMA producer (Q, K and V tiles by page; a page that does not exist is an
// out-of-range coordinate, which TMA fills with zeros). 1: issues the MMAs. 2, 3: clean V
// tiles that hold keys some row must not see: rows past the last visible key become zeros,
// and values that are not finite become zeros and their token is noted, so 0 * inf never
// reaches a row that does not see them; rows that do see one add it in the end. 4..: softmax,
// one group of four warps per tile, one thread per row. A row's O is only rescaled when its
// maximum grew by more than 2^8 since the last rescaling: until then P just exceeds 1, by at
// most 2^8, which neither the fp32 sums nor P's 16-bit floating point notice.
//
// P is rounded to the type of the cache for the second product (the tensor cores take no
// other); l sums the unrounded values. f16 ends 2^-24 below 1, where the many small weights of a long
// context beside one large one would vanish from O and not from l: there P is taken 2^7 times larger, so that
// the largest, 2^8 of the lazy maximum included, is 2^15 and what is lost lies below 2^-32 of a row's
// largest weight. O and l carry the factor alike; only the logarithm of l has to shed it.
//
// Two instances per head width, chosen by the most rows a request can have (max_new, or all of N):
// up to one tile's tokens, or more.
//   One row tile, 64 keys per step, two CTAs per SM: decoding and a few draft tokens stream the cache, so one
//   CTA's softmax and items' ends hide behind the other's loads. 128 requests of 500 to 7,500 keys, 96 heads
//   over 8 of 128, bf16: 315 to 329 us, 6.4 to 6.6 TB/s, bound by memory (two row tiles: 341).
//   Two row tiles, 128 keys per step, one CTA per SM: every K and V tile is used twice, and one tile's
//   products run under the other's softmax. A chunk of 4,096 tokens over 16,384 keys, the same heads:
//   1.76 ms in a short run, 1.88 to 1.99 ms under the power limit, 1.45 to 1.64 PFLOP/s (one row tile: 2.58). 32
//   requests of 11 tokens, one more than a tile has, over 4,000 keys: 116 us against 183; of 10 107 and 111. Bound
//   by the chain of a row tile's step: softmax 1,550 cycles (512 of them the exponentials' at 4 per instruction),
//   handing over 200, and the MMAs after the last weights 1,040, of which each row tile's half overlaps the other's.
// Measured on the way, same chunk: a thread chosen by lane number instead of elect.sync issues an MMA every 85
// cycles instead of 45 (2.47 ms); a row split over two warps 2.28 ms (the exchange costs what the shorter
// rows gain); one issuing thread per row tile 2.08 ms; waiting for the next tiles between the two row
// tiles' MMAs 2.27 ms (a wait behind queued MMAs lets the pipe run dry); the exponential in 16 bits is no
// faster; a second S tile per row tile with one row tile per CTA 440 us against 326 for decoding; output rows
// staged through shared memory 1.99 ms.
#include <algorithm>
#include <cstdlib>
#include <numeric>

#include "ops_internal.cuh"
#include "tc_ptx.cuh"

struct moe_attn_ctx {
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

using namespace ptx;

namespace {

constexpr int kRows = 128;          // rows of a tile (TMEM lanes)
constexpr int kRuns = 128;          // runs of requests whose cost sums a CTA keeps
// A CTA's least share of the axis (in keys): more CTAs than that are not worth a join. One row tile: five requests
// of up to 595 keys, 24 heads over 4 of 64: 128 11.2, 192 11.1 to 11.5, 256 13.3 us; one of 11,385 keys and 48
// heads 30.9 with 128, 26.2 with 192. Two row tiles: three chunks of up to 1,147, two heads of 128: 192 32.1,
// 384 29.4, 512 28.9 us; two chunks of 127 12.2, 15.7 and 12.0, and 17.9 with 768.
template <int QT>
constexpr int kMinStretch = QT == 1 ? 192 : 512;
// Where a CTA's share is less than twice this, items up to this long are not split. Two row tiles: 27 chunks of 205
// over 24 to 192 keys: 512 30.7, 896 23.9, 1280 23.8 us; one of 41 over 3,000 keys 18.1, 18.1 and 12.8; with 1792
// four chunks of 2,729 take 69.5 us instead of 59.7. One row tile: 768 makes the five requests above 13.5 us.
template <int QT>
constexpr int kWhole = QT == 1 ? 512 : 1280;
// What the start and end of an item of so many rows cost, in keys. With one row tile they partly hide behind the
// other CTA of the SM: 49 requests of 211 to 1,693 keys, 12 heads over 2 of 128: 128 23.5, 176 21.6, 224 21.2,
// 384 21.7 us; the five requests above 11.5, 11.1, 11.6, 11.9; eight of 52 to 417 12.3, 13.5, 13.6, 14.4. With two,
// O's way out and the join of a full tile cost as much as some keys: 28 decoding requests and 5 prompts: a fixed
// 128 82.2, 384 77.9, 640 79.9, 256 and the rows 73.8, and twice the rows 76.2 us.
template <int QT>
__device__ __forceinline__ int item_cost(int rows) { return QT == 1 ? 176 : 256 + rows; }
constexpr int kNoteSlots = 8;       // pieces whose notes of non-finite tokens are kept (> V stages + 2)
constexpr float kRescaleLog2 = 8.f;
template <int DT>
constexpr float kLiftLog2 = DT == MOE_DT_F16 ? 7.f : 0.f;  // P and l are 2^kLiftLog2 times the weights (bf16 has fp32's range)

struct AttnParams {
  moe_attn_args a;
  int p_shift;
  int G;           // query heads per key head
  int tpt;         // tokens per tile
  int box_tok;     // tokens per Q box
  float scale_log2;
  uint32_t* err;
  int32_t* tickets;  // [CTAs][QT][3], zero between calls: finished pieces (or runs) of the split item that starts in
                     // the CTA, of that item's first run, and of the run of an earlier item that starts in the CTA
  float* parts;      // [2 CTAs][QT] partial results: O [D/4][128][4], m [128], l [128], m and l of a joined run
};

template <int DT_, int D_, int QT_, int BN_, int NK_, int NV_>
struct AttnCfg {
  static constexpr int DT = DT_, D = D_, QT = QT_, BN = BN_, NK = NK_, NV = NV_;
  static constexpr int kThreads = 128 + 128 * QT;
  static constexpr int kCtasPerSm = QT == 1 ? 2 : 1;
  static constexpr int kBlk = BN * 128;          // 64 elements of every key of a tile
  static constexpr int kTile = D / 64 * kBlk;
  static constexpr int kQBlk = kRows * 128;
  static constexpr int kQ = D / 64 * kQBlk;
  static constexpr size_t kSmem = 1024 + (size_t)QT * kQ + (size_t)(NK + NV) * kTile + kRuns * 8 + 1024 + 64 * 4 * QT + 64;
  static constexpr uint32_t cols() {
    uint32_t c = 32;
    while (c < (uint32_t)(QT * (BN + D))) c <<= 1;
    return c;
  }
  static constexpr uint32_t kCols = cols();
  static constexpr int kPart = kRows * (D + 4);  // floats of one partial result
  static_assert(NV + 2 < kNoteSlots, "notes of a piece outlive the pieces that can be loaded behind it");
};

// Quotient of non-negative values; the axis usually fits in 32 bits, where a division is several times faster.
__device__ __forceinline__ int64_t div_floor(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// The axis and the calling CTA's stretch [x0, x1) of it: CTA c of n starts at c * (total / n) + min(c, total % n).
struct Axis {
  int64_t each, x0, x1, whole;
  int n, extra;
  __device__ __forceinline__ int64_t start(int c) const { return c * each + min(c, extra); }
  __device__ __forceinline__ int owner(int64_t x) const {  // the CTA whose stretch holds x
    const int64_t wide = extra * (each + 1);
    return (int)(x < wide ? div_floor(x, each + 1) : extra + div_floor(x - wide, each));
  }
};

// One request's share of the axis, and the position of an item on it.
struct Work {
  int b, h, i;             // request, key head, tile group
  int n_new, ctx, q0;      // new tokens, cached tokens before them (negative: rows without keys), first row of q
  int n_items;             // tile groups
  int fixed;               // an item's start and end, in keys
  int64_t head_cost;       // cost of one key head of the request
  int64_t base, at, cost;  // axis: start of the head, start and length of the item

  template <int QT>
  __device__ __forceinline__ bool load(const AttnParams& p, int request) {  // false: rows outside q, or keys past the table
    b = request;
    const int s = p.a.q_start[b], e = p.a.q_start[b + 1], most = p.a.W << p.p_shift, len = p.a.kv_lens[b];
    const int kv = min(max(len, 0), most);
    const bool ok = s >= 0 && e <= p.a.N && e >= s;
    n_new = ok ? e - s : 0;
    q0 = s;
    ctx = kv - n_new;
    const int st = QT * p.tpt;
    n_items = (n_new + st - 1) / st;
    const int64_t n = n_items;
    fixed = item_cost<QT>(min(n_new, st) * p.G);
    head_cost = n * (fixed + max(ctx, 0)) + st * (n * (n - 1) / 2) + n_new;
    return ok && len <= most;
  }
  template <int QT>
  __device__ __forceinline__ void set_item(const AttnParams& p, int64_t before) {
    at = base + before;
    cost = fixed + max(ctx, 0) + min((i + 1) * QT * p.tpt, n_new);
  }
  // The item at x, by a whole warp (every lane gets it).
  template <int QT>
  __device__ __forceinline__ void seek(const AttnParams& p, const int64_t* runs, int seg, int64_t x) {
    static_assert(kRuns == 128, "four runs per lane");
    const int lane = threadIdx.x & 31;
    int lo = 4 * (__popc(__ballot_sync(0xFFFFFFFFu, runs[4 * lane] <= x)) - 1);  // the last run that starts at or before x
    lo += __popc(__ballot_sync(0xFFFFFFFFu, runs[lo + (lane & 3)] <= x) & 15) - 1;
    int64_t acc = runs[lo];
    int r = lo * seg;
    load<QT>(p, r);
    while (x - acc >= (int64_t)p.a.Hkv * head_cost && r + 1 < p.a.B) {
      acc += (int64_t)p.a.Hkv * head_cost;
      load<QT>(p, ++r);
    }
    h = (int)div_floor(x - acc, head_cost);
    base = acc + h * head_cost;
    const int64_t rest = x - base, each = fixed + max(ctx, 0), st = QT * p.tpt;
    int hi = n_items;
    lo = 0;
    while (hi - lo > 1) {  // the last group that starts at or before rest
      const int64_t mid = (lo + hi) >> 1;
      if (mid * each + st * (mid * (mid + 1) / 2) <= rest) lo = (int)mid;
      else hi = (int)mid;
    }
    i = lo;
    set_item<QT>(p, i * each + st * ((int64_t)i * (i + 1) / 2));
  }
  template <int QT>
  __device__ __forceinline__ void next(const AttnParams& p) {
    if (i + 1 < n_items) {
      const int64_t before = at - base + cost;
      ++i;
      set_item<QT>(p, before);
      return;
    }
    i = 0;
    base += head_cost;
    if (++h == p.a.Hkv) {
      h = 0;
      do load<QT>(p, b + 1);
      while (n_items == 0 && b + 1 < p.a.B);
    }
    set_item<QT>(p, 0);
  }
};

// The part of an item that is a CTA's. A boundary between two stretches counts as the item's start
// where it lies in the item's first tile or before, and anywhere in an item that is not split.
template <int QT, int BN>
struct Piece {
  int t0, t1;      // tiles of BN keys
  int tq1[QT];     // the end for each row tile (its own last visible key)
  int kv_end;      // keys visible to the item's last row
  int first_lim;   // keys visible to its first row
  int64_t first_part;  // the length of axis in which a boundary counts as the start
  bool none;       // nothing of the item is this CTA's
  bool split;
  __device__ __forceinline__ Piece(const AttnParams& p, const Work& w, const Axis& ax) {
    const int tok = w.i * QT * p.tpt;
    kv_end = max(0, w.ctx + min(tok + QT * p.tpt, w.n_new));
    first_lim = w.ctx + tok + 1;
    const int nt = (kv_end + BN - 1) / BN;
    first_part = w.cost <= max(ax.whole, (int64_t)w.fixed + BN) ? w.cost : w.fixed + BN;
    int64_t lo = max(ax.x0 - w.at, (int64_t)0), hi = min(ax.x1 - w.at, w.cost);
    if (lo < first_part) lo = 0;
    if (hi < first_part) hi = 0;
    none = hi == 0;
    split = lo > 0 || hi < w.cost;
    t0 = (int)min((int64_t)nt, max(lo - w.fixed, (int64_t)0) / BN);
    t1 = none ? t0 : hi == w.cost ? nt : (int)min((int64_t)nt, max(hi - w.fixed, (int64_t)0) / BN);
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      const int end = tok + q * p.tpt < w.n_new ? max(0, w.ctx + min(tok + (q + 1) * p.tpt, w.n_new)) : 0;
      tq1[q] = min(t1, (end + BN - 1) / BN);
    }
  }
  __device__ __forceinline__ bool tiles() const { return t1 > t0; }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}

__device__ __forceinline__ void max32(const uint32_t* v, float (&mx)[4]) {
#pragma unroll
  for (int k = 0; k < 32; k += 2)
    mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
}
// 32 scores to weights exp2(s * scale + off), packed to the 16-bit type in v[0..15]; added to sum.
template <int DT>
__device__ __forceinline__ void exp32(uint32_t* v, float2 scale, float2 off, float2 (&sum)[2]) {
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    const float2 x = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), scale, off);
    const float2 e = make_float2(ex2(x.x), ex2(x.y));
    sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], e);
    v[k / 2] = pack2<DT>(e.x, e.y);
  }
}

// ln of a row's sum of exp(scale * score), from its maximum and its sum of weights.
template <int DT>
__device__ __forceinline__ float log_sum(float m, float l, float scale_log2) {
  return l == 0.f ? -INFINITY : (m * scale_log2 + (log2f(l) - kLiftLog2<DT>)) * 0.69314718055994530942f;
}

template <int DT>
__device__ __forceinline__ bool not_finite(uint32_t half) {  // one 16-bit value
  constexpr uint32_t e = DT == MOE_DT_BF16 ? 0x7F80u : 0x7C00u;
  return (half & e) == e;
}

// mbar_wait by a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_suspended(bar, parity, err));
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtasPerSm)
    attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const __grid_constant__ AttnParams p) {
  constexpr int D = C::D, QT = C::QT, BN = C::BN, NK = C::NK, NV = C::NV, DT = C::DT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sq = smem;
  uint8_t* sk = sq + QT * C::kQ;
  uint8_t* sv = sk + NK * C::kTile;
  int64_t* runs = reinterpret_cast<int64_t*>(sv + NV * C::kTile);
  uint64_t* bar = reinterpret_cast<uint64_t*>(runs + kRuns);
  uint64_t *kfull = bar, *kempty = kfull + NK, *vfull = kempty + NK, *vempty = vfull + NV, *vclean = vempty + NV;
  uint64_t *qfull = vclean + NV, *qempty = qfull + 1, *oempty = qempty + 1, *drain = oempty + 1;
  uint64_t *sfull = drain + 1, *pfull = sfull + QT, *ofull = pfull + 2 * QT, *group = ofull + QT;
  int64_t* warp_sum = reinterpret_cast<int64_t*>(group + QT);      // [4]
  uint32_t* notes = reinterpret_cast<uint32_t*>(warp_sum + 4);     // [kNoteSlots][2][8]
  uint32_t* tmem_slot = notes + kNoteSlots * 16;
  int* group_flag = reinterpret_cast<int*>(tmem_slot + 1);         // [QT]
  // the softmax warps' place on the axis, out of their registers while they work on tiles
  Work* parked = reinterpret_cast<Work*>(reinterpret_cast<uint8_t*>(bar) + 1024);
  static_assert(sizeof(Work) <= 64, "space of a parked place");
  Axis* parked_axis = reinterpret_cast<Axis*>(reinterpret_cast<uint8_t*>(parked) + 64 * 4 * QT);
  static_assert(sizeof(Axis) <= 64, "space of the parked axis");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NK; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 1);
      mbar_init(&vclean[s], 2);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    mbar_init(oempty, 4 * QT);
    mbar_init(drain, 1);
    for (int q = 0; q < QT; ++q) {
      mbar_init(&sfull[q], 1);
      mbar_init(&pfull[2 * q], 4);
      mbar_init(&pfull[2 * q + 1], 4);
      mbar_init(&ofull[q], 1);
      mbar_init(&group[q], 4);
    }
    fence_mbar_init();
  }
  if (warp == 0 && lane < 3) prefetch_map(lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v);
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_entry();

  // the axis: thread t < kRuns sums the costs of a run of requests
  const int B = p.a.B, seg = (B + kRuns - 1) / kRuns;
  int64_t mine = 0, upto = 0;
  if (warp < kRuns / 32) {
    for (int b = threadIdx.x * seg; b < min(B, (int)(threadIdx.x + 1) * seg); ++b) {
      Work one{};
      if (!one.load<QT>(p, b) && blockIdx.x == 0) atomicOr(p.err, kErrIndex);
      mine += (int64_t)p.a.Hkv * one.head_cost;
    }
    upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += u;
    }
    if (lane == 31) warp_sum[warp] = upto;
  }
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int k = 0; k < kRuns / 32; ++k) {
    if (k == warp) runs[threadIdx.x] = total + upto - mine;
    total += warp_sum[k];
  }
  __syncthreads();
  Axis ax;
  ax.n = (int)max((int64_t)1, min((int64_t)gridDim.x, total / kMinStretch<QT>));
  ax.each = div_floor(total, ax.n);
  ax.extra = (int)(total - ax.each * ax.n);
  ax.whole = ax.each <= 2 * kWhole<QT> ? kWhole<QT> : 0;
  ax.x0 = ax.x1 = 0;
  if (blockIdx.x < ax.n) {
    ax.x0 = ax.start(blockIdx.x);
    ax.x1 = ax.start(blockIdx.x + 1);
  }
  if (threadIdx.x == 0) *parked_axis = ax;
  __syncthreads();
  Work w{};
  if (ax.x0 < ax.x1) w.seek<QT>(p, runs, seg, ax.x0);
  bool more = ax.x0 < ax.x1, ok = true;
  auto advance = [&] {
    more = ok && w.at + w.cost < ax.x1;
    if (more) w.next<QT>(p);
  };

  if (warp == 0) {
    // ---- producer: the warp walks together, lanes load and copy one page each ----
    const int P = p.a.page_size, pages = P >= BN ? 1 : BN / P;
    const int rows = P >= BN ? BN : P;  // keys per box
    uint32_t kn = 0, vn = 0, qn = 0;
    while (more) {
      const Piece<QT, BN> pc(p, w, ax);
      if (pc.tiles()) {
        if (!warp_wait(qempty, (qn & 1) ^ 1u, p.err)) {
          ok = false;
          break;
        }
        ++qn;
        if (lane == 0) {
          const int box_bytes = p.box_tok * p.G * 128;
          int boxes[QT], n = 0;
#pragma unroll
          for (int q = 0; q < QT; ++q) {
            const int tok = (w.i * QT + q) * p.tpt;
            boxes[q] = pc.tq1[q] > pc.t0 ? (min(p.tpt, w.n_new - tok) + p.box_tok - 1) / p.box_tok : 0;
            n += boxes[q];
          }
          mbar_arrive_expect_tx(qfull, (uint32_t)(n * (D / 64) * box_bytes));
          for (int q = 0; q < QT; ++q)
            for (int x = 0; x < boxes[q]; ++x)
              for (int d = 0; d < D / 64; ++d)
                tma_3d(sq + q * C::kQ + d * C::kQBlk + x * box_bytes, &map_q, d * 64, w.h * p.G,
                       w.q0 + (w.i * QT + q) * p.tpt + x * p.box_tok, qfull);
        }
        __syncwarp();
        const int32_t* table = p.a.block_table + w.b * p.a.table_stride;
        // pages are looked up 32 at a time, the next 32 while these are copied
        const auto inside = [&](int col) { return ((int64_t)col << p.p_shift) < pc.kv_end; };  // (the table holds kv_end)
        const auto look_up = [&](int col) { return inside(col + lane) ? table[col + lane] : 0; };
        const auto checked = [&](int col, int page) {  // num_pages: nothing there, TMA fills with zeros
          if (!inside(col + lane)) return p.a.num_pages;
          if (page >= 0 && page < p.a.num_pages) return page;
          atomicOr(p.err, kErrIndex);
          return p.a.num_pages;
        };
        int col0 = (int)(((int64_t)pc.t0 * BN) >> p.p_shift);
        int ids = checked(col0, look_up(col0)), ids_next = look_up(col0 + 32);
        for (int t = pc.t0; t < pc.t1 && ok; ++t) {
          int at = (int)(((int64_t)t * BN) >> p.p_shift) - col0;
          if (at >= 32) {
            col0 += 32;
            at -= 32;
            ids = checked(col0, ids_next);
            ids_next = look_up(col0 + 32);
          }
          const int id = __shfl_sync(0xFFFFFFFFu, ids, (at + lane) & 31);  // lanes below `pages`: the tile's pages
          const int row = P >= BN ? (t * BN) & (P - 1) : 0;
          const int ks = (int)(kn % NK), vs = (int)(vn % NV);
          ok = warp_wait(&kempty[ks], ((kn / NK) & 1) ^ 1u, p.err);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&kfull[ks], C::kTile);
          __syncwarp();
          if (lane < pages)
#pragma unroll
            for (int d = 0; d < D / 64; ++d)
              tma_4d(sk + ks * C::kTile + d * C::kBlk + lane * rows * 128, &map_k, d * 64, row, w.h, id, &kfull[ks]);
          ++kn;
          ok = warp_wait(&vempty[vs], ((vn / NV) & 1) ^ 1u, p.err);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&vfull[vs], C::kTile);
          __syncwarp();
          if (lane < pages)
#pragma unroll
            for (int d = 0; d < D / 64; ++d)
              tma_4d(sv + vs * C::kTile + d * C::kBlk + lane * rows * 128, &map_v, d * 64, row, w.h, id, &vfull[vs]);
          ++vn;
        }
      }
      advance();
    }
    if (!ok) {  // copies already issued land before the CTA's shared memory goes away
      if (qn) warp_wait(qfull, (qn - 1) & 1, p.err);
      for (uint32_t j = kn > NK ? kn - NK : 0; j < kn; ++j) warp_wait(&kfull[j % NK], (j / NK) & 1, p.err);
      for (uint32_t j = vn > NV ? vn - NV : 0; j < vn; ++j) warp_wait(&vfull[j % NV], (j / NV) & 1, p.err);
    }
  } else if (warp == 1) {
    // ---- MMA issuer. The MMAs of one thread run in the order of issue: P(t) is read before S(t + 1) is
    // written over it, and what a commit reports includes every MMA before it. ----
    if (elect_one()) {
      constexpr uint32_t kIdS = idesc_16(DT == MOE_DT_BF16, false, kRows, BN);
      constexpr uint32_t kIdO = idesc_16(DT == MOE_DT_BF16, true, kRows, D);
      uint32_t kn = 0, vn = 0, pn = 0, on[QT] = {};
      // descriptors of the first tiles; the address field (16-byte units) of the others is further on
      const uint64_t dq = desc_sw128(smem_u32(sq)), dk = desc_sw128(smem_u32(sk));
      const uint64_t dv = desc_sw128_mn(smem_u32(sv), C::kBlk);
      const auto issue_s = [&](int q) {
        const uint64_t d = dk + ((kn % NK) * C::kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16_ss(tmem + q * BN, dq + ((q * C::kQ + (kk >> 2) * C::kQBlk + (kk & 3) * 32) >> 4),
                     d + (((kk >> 2) * C::kBlk + (kk & 3) * 32) >> 4), kIdS, kk > 0);
        mma_commit(&sfull[q]);
      };
      const auto wait_k = [&] { return mbar_wait_suspended(&kfull[kn % NK], (kn / NK) & 1, p.err); };
      const auto wait_v = [&](uint32_t n) { return mbar_wait_suspended(&vclean[n % NV], (n / NV) & 1, p.err); };
      while (more) {
        const Piece<QT, BN> pc(p, w, ax);
        if (pc.tiles()) {
          ok = mbar_wait_suspended(qfull, pn & 1, p.err) && wait_k();
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < QT; ++q)
            if (pc.t0 < pc.tq1[q]) issue_s(q);
          mma_commit(&kempty[kn % NK]);
          ++kn;
          const bool one = pc.t0 + 1 == pc.t1;
          if (one) mma_commit(qempty);
          ok = wait_v(vn) && (one || wait_k()) && mbar_wait_suspended(oempty, (pn & 1) ^ 1u, p.err);
          for (int t = pc.t0; t < pc.t1 && ok; ++t) {
            const bool last = t + 1 == pc.t1;
            const uint64_t d = dv + ((vn % NV) * C::kTile >> 4);
#pragma unroll
            for (int q = 0; q < QT; ++q) {
              if (t < pc.tq1[q]) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // half of the keys can start while the other is computed
                  ok = ok && mbar_wait_suspended(&pfull[2 * q + half], on[q] & 1, p.err);
                  if (!ok) break;
                  tc_fence_after();
#pragma unroll
                  for (int j = 0; j < BN / 32; ++j) {
                    const int kk = half * (BN / 32) + j;
                    mma_f16_ts(tmem + QT * BN + q * D, tmem + q * BN + kk * 8, d + (kk * 2048 >> 4), kIdO,
                               t > pc.t0 || kk > 0);
                  }
                }
                if (!ok) break;
                ++on[q];
                if (t + 1 < pc.tq1[q]) issue_s(q);
                else mma_commit(&ofull[q]);
              }
              if (q + 1 < QT) continue;
              mma_commit(&vempty[vn % NV]);
              if (!last) {
                mma_commit(&kempty[kn % NK]);
                if (t + 2 == pc.t1) mma_commit(qempty);
              }
            }
            ++vn;
            if (!last) {
              ++kn;
              ok = ok && wait_v(vn);
              if (ok && t + 2 < pc.t1) ok = wait_k();
            }
          }
          if (!ok) break;
          // a row tile without keys in this piece passes it at the MMAs' pace too
#pragma unroll
          for (int q = 0; q < QT; ++q)
            if (pc.tq1[q] <= pc.t0) mma_commit(&ofull[q]);
          ++pn;
        }
        advance();
      }
      mma_commit(drain);  // every MMA issued has completed before TMEM is released
      mbar_wait_suspended(drain, 0, p.err);
    }
  } else if (warp < 4) {
    // ---- V tiles that hold keys some row must not see ----
    const int cw = warp - 2;
    uint32_t vn = 0, pn = 0;
    while (more) {
      const Piece<QT, BN> pc(p, w, ax);
      if (pc.tiles()) {
        uint32_t* note = notes + (pn % kNoteSlots) * 16 + cw * 8;
        if (lane < 8) note[lane] = 0;
        __syncwarp();
        for (int t = pc.t0; t < pc.t1; ++t, ++vn) {
          const int vs = (int)(vn % NV);
          ok = warp_wait(&vfull[vs], (vn / NV) & 1, p.err);
          if (!ok) break;
          if ((int64_t)(t + 1) * BN > pc.first_lim) {
            for (int c = cw * 32 + lane; c < BN; c += 64) {
              const int64_t key = (int64_t)t * BN + c;
              if (key < pc.first_lim) continue;
              const bool unseen = key >= pc.kv_end;
              bool odd = false;
#pragma unroll
              for (int d = 0; d < D / 64; ++d)
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  // every lane starts at another 16 bytes of its row: no two share a bank
                  uint4* u = reinterpret_cast<uint4*>(sv + vs * C::kTile + d * C::kBlk + c * 128 + ((x + lane) & 7) * 16);
                  if (unseen) {
                    *u = make_uint4(0, 0, 0, 0);
                    continue;
                  }
                  uint4 val = *u;
                  uint32_t* word = reinterpret_cast<uint32_t*>(&val);
                  bool hit = false;
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    if (not_finite<DT>(word[k])) word[k] &= 0xFFFF0000u, hit = true;
                    if (not_finite<DT>(word[k] >> 16)) word[k] &= 0x0000FFFFu, hit = true;
                  }
                  if (hit) *u = val;
                  odd |= hit;
                }
              const int rel = (int)(key - pc.first_lim);  // < QT * tpt <= 256
              if (odd) atomicOr(&note[rel >> 5], 1u << (rel & 31));
            }
            fence_proxy_async();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&vclean[vs]);
        }
        if (!ok) break;
        ++pn;
      }
      advance();
    }
  } else {
    // ---- softmax: thread = row r of tile q ----
    constexpr int kHalf = BN / 2;
    const int q = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane, rt = r / p.G, rh = r - rt * p.G;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_base + q * BN, to = tmem + lane_base + QT * BN + q * D;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t sn = 0, on = 0, pn = 0, gn = 0;
    const auto group_sync = [&] {  // the tile's warps
      __syncwarp();
      if (lane == 0) mbar_arrive(&group[q]);
      ok = warp_wait(&group[q], gn++ & 1, p.err) && ok;
    };
    Work* const place = reinterpret_cast<Work*>(reinterpret_cast<uint8_t*>(parked) + 64 * (warp - 4));
    while (more) {
      int t0, t_end, lim, tile_lim;
      bool live, warp_live;
      {
        const Piece<QT, BN> pc(p, w, ax);
        if (pc.none) {
          advance();
          continue;
        }
        const int tok = (w.i * QT + q) * p.tpt, n_tok = min(p.tpt, w.n_new - tok);
        t0 = pc.t0;
        t_end = q == 0 ? pc.tq1[0] : pc.tq1[QT - 1];
        live = rt < n_tok;
        warp_live = quarter * 32 < n_tok * p.G;
        lim = w.ctx + tok + rt + 1;   // keys this row sees (live rows)
        tile_lim = w.ctx + tok + 1;   // keys every row of the tile sees
      }
      __syncwarp();
      if (lane == 0) *place = w;
      __syncwarp();
      float m = -INFINITY, l = 0.f;
      for (int t = t0; t < t_end; ++t) {
        ok = warp_wait(&sfull[q], sn & 1, p.err);
        if (!ok) break;
        ++sn;
        tc_fence_after();
        if (warp_live) {
          const int64_t key0 = (int64_t)t * BN;
          if (key0 + BN > tile_lim) {  // hide keys in place: few tiles need it, so it is kept out of the code of the others
            const int see = (int)max(min((int64_t)lim - key0, (int64_t)BN), (int64_t)0);
#pragma unroll 1
            for (int c = 0; c < BN; c += 32) {
              uint32_t v[32];
              tmem_ld32(ts + c, v);
              tmem_wait_ld32(v);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (c + k >= see) v[k] = 0xFF800000u;  // -inf
              tmem_st32(ts + c, v);
            }
            tmem_wait_st();
          }
          uint32_t s[BN];
          const auto load_s = [&] {
#pragma unroll
            for (int c = 0; c < BN; c += 32) tmem_ld32(ts + c, s + c);
          };
          load_s();
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < BN; c += 32) {
            tmem_wait_ld32(s + c);
            max32(s + c, mx);
          }
          const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
          if (t == t0) {
            m = top;
          } else {
            const bool grow = live && (top - m) * p.scale_log2 > kRescaleLog2;
            if (__any_sync(0xFFFFFFFFu, grow)) {
              // S(t) is complete, so is the product of tile t - 1 that was issued before it
              const float f = grow ? ex2((m - top) * p.scale_log2) : 1.f;
              if (grow) m = top;
              l *= f;
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(to + c, o);
                tmem_wait_ld32(o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st32(to + c, o);
                tmem_wait_st();
              }
              load_s();  // again, so that its registers need not be kept over the loop above
#pragma unroll
              for (int c = 0; c < BN; c += 32) tmem_wait_ld32(s + c);
            }
          }
          const float off = m == -INFINITY ? 0.f : fmaf(-m, p.scale_log2, kLiftLog2<DT>);
          float2 sum[2] = {};
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // the MMAs can start on the first half of the weights
#pragma unroll
            for (int c = half * kHalf; c < (half + 1) * kHalf; c += 32) {
              exp32<DT>(s + c, sc2, make_float2(off, off), sum);
              tmem_st16(ts + c / 2, s + c);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[2 * q + half]);
          }
          sum[0] = add2(sum[0], sum[1]);
          l += sum[0].x + sum[0].y;
        } else {
          if (lane == 0) mbar_arrive(&pfull[2 * q]);
          if (lane == 0) mbar_arrive(&pfull[2 * q + 1]);
        }
      }
      if (!ok) break;
      // ---- the piece's result: to out, or to the workspace where the item is split ----
      const bool any = t0 < t_end;
      w = *place;
      const Piece<QT, BN> pc(p, w, *parked_axis);
      const int tok = (w.i * QT + q) * p.tpt;       // the tile's first token
      const int n_tok = min(p.tpt, w.n_new - tok);  // its tokens (<= 0: no such tile)
      if (pc.tiles()) {
        ok = warp_wait(&ofull[q], on & 1, p.err);
        if (!ok) break;
        ++on;
        tc_fence_after();
      }
      int first = 0, pieces = 1;
      float* part = nullptr;
      if (pc.split) {
        first = parked_axis->owner(w.at + pc.first_part - 1);
        pieces = parked_axis->owner(w.at + w.cost - 1) - first + 1;
        part = p.parts + (size_t)((2 * blockIdx.x + (first == (int)blockIdx.x ? 1 : 0)) * QT + q) * C::kPart;
      }
      const int64_t n_row = (int64_t)w.q0 + tok + rt;
      const int head = w.h * p.G + rh;
      const int64_t out_at = n_row * p.a.out_tok + (int64_t)head * p.a.out_head;
      if (warp_live) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const volatile uint32_t* note = notes + (pn % kNoteSlots) * 16;
        // does any clean warp's note say that a token was not finite?
        const bool noted = any && (int64_t)pc.t1 * BN > pc.first_lim && __any_sync(0xFFFFFFFFu, lane < 16 && note[lane & 15]);
        if (any || !pc.split) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            if (any) {
              __syncwarp();
              tmem_ld32(to + c, o);
              tmem_wait_ld32(o);
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = 0;
            }
            if (noted && live) {  // add what the cleaning took out, where this row sees it
#pragma unroll 1
              for (int rel = 0; rel < lim - pc.first_lim; ++rel) {
                if (!((note[rel >> 5] | note[8 + (rel >> 5)]) >> (rel & 31) & 1)) continue;
                const int key = pc.first_lim + rel, col = key >> p.p_shift;
                const int id = p.a.block_table[w.b * p.a.table_stride + col];
                const uint16_t* v = (const uint16_t*)p.a.v_cache + id * p.a.vc_page +
                                    (key & (p.a.page_size - 1)) * p.a.vc_row + w.h * p.a.vc_head + c;
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (not_finite<DT>(v[k])) o[k] = __float_as_uint(__uint_as_float(o[k]) + to_f32<DT>(v[k]));
              }
            }
            if (pc.split) {
              if (live)
#pragma unroll
                for (int k = 0; k < 32; k += 4)  // lanes are neighbours
                  *reinterpret_cast<uint4*>(part + ((c + k) / 4 * kRows + r) * 4) =
                      make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            } else {
              if (live)
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                  uint4 y;
                  uint32_t* u = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
                  for (int x = 0; x < 4; ++x)
                    u[x] = pack2<DT>(__uint_as_float(o[k + 2 * x]) * inv, __uint_as_float(o[k + 2 * x + 1]) * inv);
                  *reinterpret_cast<uint4*>((uint16_t*)p.a.out + out_at + c + k) = y;
                }
            }
          }
        }
        if (live) {
          if (pc.split) {
            part[kRows * D + r] = m;
            part[kRows * (D + 1) + r] = l;
          } else if (p.a.lse) {
            p.a.lse[n_row * p.a.Hq + head] = log_sum<DT>(m, l, p.scale_log2);
          }
        }
      }
      if (pc.tiles()) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(oempty);
        ++pn;
      }
      if (pc.split && n_tok > 0) {
        // Pieces are joined by the last to finish; many of them in two levels, runs of `fan` neighbours by each
        // run's last, then the runs by the last run's: a join waits for one L2 access per few pieces. (One request of
        // 60,000 keys, 96 heads over 8 of 128: 57 us, in one level 67; of 16,000 26.7 and 34; of 11,385 keys and four
        // tokens, 48 heads over 4 of 64, 26 and 49. Up to 16 pieces one level: five of 6,000 keys 17.7 us, two 19.2.)
        const int rows = n_tok * p.G, fan = pieces > 16 && pieces <= 64 ? 8 : 16;
        bool whole = pieces <= fan;  // this join ends the item
        int base = whole ? 0 : ((int)blockIdx.x - first) / fan * fan, step = 1;
        int count = whole ? pieces : min(fan, pieces - base);
        while (true) {
          int32_t* ticket = p.tickets + ((first + base) * QT + q) * 3 + (whole ? 0 : base == 0 ? 1 : 2);
          __threadfence();
          group_sync();
          if (ok && r == 0) group_flag[q] = atomicAdd(ticket, 1) == count - 1;
          group_sync();
          if (!ok || *(volatile int*)&group_flag[q] == 0) break;
          __threadfence();
          if (r == 0) *ticket = 0;
          const auto piece_at = [&](int k) {
            const int x = base + k * step;
            return p.parts + (size_t)((2 * (first + x) + (x == 0 ? 1 : 0)) * QT + q) * C::kPart;
          };
          const int stat = kRows * (step > 1 ? D + 2 : D);  // where m and l are
          float* run = piece_at(0);                         // where a run's result goes
          const auto row_out = [&](int row, int64_t& n, int& hd) {  // token and head of a row of the tile
            const int t = row / p.G;
            n = (int64_t)w.q0 + tok + t;
            hd = w.h * p.G + row - t * p.G;
          };
          const auto row_stat = [&](int row, float top, float sum) {
            if (!whole) {
              run[kRows * (D + 2) + row] = top;
              run[kRows * (D + 3) + row] = sum;
            } else if (p.a.lse) {
              int64_t n;
              int hd;
              row_out(row, n, hd);
              p.a.lse[n * p.a.Hq + hd] = log_sum<DT>(top, sum, p.scale_log2);
            }
          };
          // Two ways through the loads: four columns of a row per thread and eight pieces at once, or lane = row, each
          // warp a quarter of the columns and two pieces at once. The one with fewer rounds.
          constexpr int kAtOnce = 8;
          if ((rows * (D / 4) + kRows - 1) / kRows * ((count + kAtOnce - 1) / kAtOnce) <= (rows + 31) / 32 * ((count + 1) / 2)) {
            for (int x = r; x < rows * (D / 4); x += kRows) {
              const int c = x / rows, row = x - c * rows;  // neighbours on neighbouring rows
              float top = -INFINITY, sum = 0.f;
              float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
              for (int k = 0; k < count; k += kAtOnce) {
                float mk[kAtOnce], lk[kAtOnce];
                float4 o[kAtOnce];
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                  const float* pt = piece_at(min(k + u, count - 1));
                  mk[u] = __ldcg(pt + stat + row);
                  lk[u] = k + u < count ? __ldcg(pt + stat + kRows + row) : 0.f;
                  o[u] = __ldcg(reinterpret_cast<const float4*>(pt) + c * kRows + row);
                }
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                  if (lk[u] == 0.f) continue;  // the row saw nothing in this piece; its O may not be written
                  const float nt = fmaxf(top, mk[u]);
                  const float f0 = ex2((top - nt) * p.scale_log2), f = ex2((mk[u] - nt) * p.scale_log2);
                  top = nt;
                  sum = sum * f0 + lk[u] * f;
                  acc.x = acc.x * f0 + o[u].x * f;
                  acc.y = acc.y * f0 + o[u].y * f;
                  acc.z = acc.z * f0 + o[u].z * f;
                  acc.w = acc.w * f0 + o[u].w * f;
                }
              }
              if (c == 0) row_stat(row, top, sum);
              if (!whole) {
                reinterpret_cast<float4*>(run)[c * kRows + row] = acc;
                continue;
              }
              const float inv = sum == 0.f ? 0.f : 1.f / sum;
              int64_t n;
              int hd;
              row_out(row, n, hd);
              *reinterpret_cast<uint2*>((uint16_t*)p.a.out + n * p.a.out_tok + (int64_t)hd * p.a.out_head + 4 * c) =
                  make_uint2(pack2<DT>(acc.x * inv, acc.y * inv), pack2<DT>(acc.z * inv, acc.w * inv));
            }
          } else {
            for (int r0 = 0; r0 < rows; r0 += 32) {
              constexpr int kCols4 = D / 16;
              const int row = min(r0 + lane, rows - 1);
              float top = -INFINITY, sum = 0.f;
              float4 acc[kCols4];
#pragma unroll
              for (int j = 0; j < kCols4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
              for (int k = 0; k < count; k += 2) {
                float mk[2], lk[2];
                float4 o[2][kCols4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const float* pt = piece_at(min(k + u, count - 1));
                  mk[u] = __ldcg(pt + stat + row);
                  lk[u] = k + u < count ? __ldcg(pt + stat + kRows + row) : 0.f;
#pragma unroll
                  for (int j = 0; j < kCols4; ++j)
                    o[u][j] = __ldcg(reinterpret_cast<const float4*>(pt) + (quarter * kCols4 + j) * kRows + row);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  if (lk[u] == 0.f) continue;  // the row saw nothing in this piece; its O may not be written
                  const float nt = fmaxf(top, mk[u]);
                  const float f0 = ex2((top - nt) * p.scale_log2), f = ex2((mk[u] - nt) * p.scale_log2);
                  top = nt;
                  sum = sum * f0 + lk[u] * f;
#pragma unroll
                  for (int j = 0; j < kCols4; ++j) {
                    acc[j].x = acc[j].x * f0 + o[u][j].x * f;
                    acc[j].y = acc[j].y * f0 + o[u][j].y * f;
                    acc[j].z = acc[j].z * f0 + o[u][j].z * f;
                    acc[j].w = acc[j].w * f0 + o[u][j].w * f;
                  }
                }
              }
              __syncwarp();  // lanes past the last row have read its values, which it may now replace
              if (r0 + lane >= rows) continue;
              if (quarter == 0) row_stat(row, top, sum);
              if (!whole) {
#pragma unroll
                for (int j = 0; j < kCols4; ++j) reinterpret_cast<float4*>(run)[(quarter * kCols4 + j) * kRows + row] = acc[j];
                continue;
              }
              const float inv = sum == 0.f ? 0.f : 1.f / sum;
              int64_t n;
              int hd;
              row_out(row, n, hd);
              uint16_t* out = (uint16_t*)p.a.out + n * p.a.out_tok + (int64_t)hd * p.a.out_head + quarter * (D / 4);
#pragma unroll
              for (int j = 0; j < kCols4; j += 2)
                *reinterpret_cast<uint4*>(out + 4 * j) =
                    make_uint4(pack2<DT>(acc[j].x * inv, acc[j].y * inv), pack2<DT>(acc[j].z * inv, acc[j].w * inv),
                               pack2<DT>(acc[j + 1].x * inv, acc[j + 1].y * inv),
                               pack2<DT>(acc[j + 1].z * inv, acc[j + 1].w * inv));
            }
          }
          if (whole) break;
          whole = true;
          count = (pieces + fan - 1) / fan;
          step = fan;
          base = 0;
        }
        if (!ok) break;
      }
      w = *place;
      ax = *parked_axis;
      advance();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int DT, int D>
using StreamCfg = AttnCfg<DT, D, 1, 64, 2, 2>;
template <int DT, int D>
using ChunkCfg = AttnCfg<DT, D, 2, 128, 2, 2>;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A tensor of 16-bit elements read in boxes with 128-byte swizzle; dims innermost first,
// strides (elements) of the outer dimensions. Host-only, so it may run during stream capture.
bool make_map(CUtensorMap* map, const void* base, int dt, int rank, const int64_t* dims, const int64_t* strides,
              const int* box) {
  static const EncodeTiledFn encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<EncodeTiledFn>(fn);
  }();
  if (!encode) return false;
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], e[4];
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    b[i] = (cuuint32_t)box[i];
    e[i] = 1;
    // the stride of a dimension of one is never used; TMA still wants a valid one
    if (i) s[i - 1] = (cuuint64_t)(dims[i] == 1 ? dims[0] : strides[i - 1]) * 2;
  }
  return encode(map, dt == MOE_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                (cuuint32_t)rank, const_cast<void*>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
cudaError_t attn_configure() {
  return cudaFuncSetAttribute(attn_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
}

template <class C>
int attn_launch(const moe_attn_ctx* ctx, const AttnParams& p, cudaStream_t s) {
  const moe_attn_args& a = p.a;
  CUtensorMap mq, mk, mv;
  const int64_t qd[3] = {a.D, a.Hq, a.N}, qs[2] = {a.q_head, a.q_tok};
  const int qb[3] = {64, p.G, p.box_tok};
  const int64_t cd[4] = {a.D, a.page_size, a.Hkv, a.num_pages};
  const int64_t ks[3] = {a.kc_row, a.kc_head, a.kc_page}, vs[3] = {a.vc_row, a.vc_head, a.vc_page};
  const int cb[4] = {64, a.page_size < C::BN ? a.page_size : C::BN, 1, 1};
  if (!make_map(&mq, a.q, a.dtype, 3, qd, qs, qb) || !make_map(&mk, a.k_cache, a.dtype, 4, cd, ks, cb) ||
      !make_map(&mv, a.v_cache, a.dtype, 4, cd, vs, cb))
    return MOE_ERR_CUDA;
  return launch_pdl(attn_kernel<C>, dim3((unsigned)(ctx->sm_count * C::kCtasPerSm)), dim3(C::kThreads), C::kSmem, s,
                    mq, mk, mv, p) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

template <int DT, int D>
int attn_by_rows(const moe_attn_ctx* ctx, const AttnParams& p, cudaStream_t s) {
  const int64_t most = p.a.max_new > 0 ? std::min(p.a.max_new, p.a.N) : p.a.N;
  if (most <= p.tpt) return attn_launch<StreamCfg<DT, D>>(ctx, p, s);
  return attn_launch<ChunkCfg<DT, D>>(ctx, p, s);
}

// Clears the error word and the tickets. cudaMemset does not wait, and streams that do not wait for the default one
// could use the handle before it ran: so this does.
bool clear_head(const moe_attn_ctx* c) {
  return cudaMemset(c->mem, 0, c->head_bytes) == cudaSuccess && cudaStreamSynchronize(cudaStreamLegacy) == cudaSuccess;
}

// Whether q and out share an element. Tensors of the same strides whose spans meet may still lie beside each other (as
// halves of a row or of a head, or in every other row): then element (n, h, d) of out is one of q's where their distance
// is dn tokens, dh heads and dd elements, each less than the tensor has.
bool shares_elements(const moe_attn_args* a) {
  if (!overlap(span16(a->q, a->N, a->q_tok, a->Hq, a->q_head, a->D), span16(a->out, a->N, a->out_tok, a->Hq, a->out_head, a->D)))
    return false;
  if ((a->N > 1 && a->q_tok != a->out_tok) || (a->Hq > 1 && a->q_head != a->out_head)) return true;
  const int64_t apart = ((const char*)a->out - (const char*)a->q) / 2;
  for (int64_t dh = 1 - a->Hq; dh < a->Hq; ++dh) {
    const int64_t rest = apart - (a->Hq > 1 ? dh * a->q_head : 0);
    const int64_t most = a->N - 1, near = most ? std::max(-most, std::min(most, rest / a->q_tok)) : 0;
    for (int64_t dn = near - 1; dn <= near + 1; ++dn)
      if (std::abs(dn) <= most && std::abs(rest - (most ? dn * a->q_tok : 0)) < a->D) return true;
  }
  return false;
}

int attn_check(const moe_attn_args* a) {
  if (!a || a->N < 0 || a->B < 0 || a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv || a->num_pages < 1 || a->W < 1 ||
      a->max_new < 0 || !is_pow2(a->page_size) || a->table_stride < a->W)
    return MOE_ERR_INVALID_ARG;
  if (a->dtype != MOE_DT_BF16 && a->dtype != MOE_DT_F16) return MOE_ERR_INVALID_ARG;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return MOE_ERR_INVALID_ARG;
  if ((a->D != 64 && a->D != 128) || a->Hq / a->Hkv > 128 || a->page_size < 16 || a->page_size > 1024 ||
      (int64_t)a->W * a->page_size >= ((int64_t)1 << 30) || (int64_t)a->N * a->Hq >= ((int64_t)1 << 31))
    return MOE_ERR_UNSUPPORTED;
  if (a->N == 0 || a->B == 0) return MOE_OK;
  const void* t16[] = {a->q, a->k_cache, a->v_cache, a->out};
  for (const void* p : t16)
    if (!p || !is_aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  const int64_t strides[] = {a->q_tok,   a->q_head, a->out_tok, a->out_head, a->kc_page,
                             a->kc_row, a->kc_head, a->vc_page, a->vc_row,   a->vc_head};
  const int64_t extents[] = {a->N, a->Hq, a->N, a->Hq, a->num_pages, a->page_size, a->Hkv, a->num_pages, a->page_size,
                             a->Hkv};
  for (int i = 0; i < 10; ++i) {
    const int64_t s = strides[i];
    // (the stride of a dimension of one is never used)
    if (s < 0 || s >= ((int64_t)1 << 38) || (extents[i] > 1 && (s == 0 || s % 8))) return MOE_ERR_INVALID_ARG;
  }
  const void* t32[] = {a->block_table, a->q_start, a->kv_lens};
  for (const void* p : t32)
    if (!p || !is_aligned(p, 4)) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(a->lse, 4)) return MOE_ERR_INVALID_ARG;
  if (shares_elements(a)) return MOE_ERR_INVALID_ARG;
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
  // error word | tickets (three per CTA and row tile) | partial results (two per CTA and row tile)
  const size_t most = 2 * (size_t)c->sm_count;
  const size_t head = (256 + most * 3 * 4 + 255) / 256 * 256;
  c->head_bytes = head;
  c->bytes = head + 2 * most * sizeof(float) * StreamCfg<0, 128>::kPart;
  if (cudaMalloc(&c->mem, c->bytes) != cudaSuccess) {
    cudaGetLastError();
    delete c;
    return MOE_ERR_OOM;
  }
  c->err = (uint32_t*)c->mem;
  c->tickets = (int32_t*)((char*)c->mem + 256);
  c->parts = (float*)((char*)c->mem + head);
  if (!clear_head(c) || attn_configure<StreamCfg<0, 64>>() != cudaSuccess ||
      attn_configure<StreamCfg<0, 128>>() != cudaSuccess || attn_configure<StreamCfg<1, 64>>() != cudaSuccess ||
      attn_configure<StreamCfg<1, 128>>() != cudaSuccess || attn_configure<ChunkCfg<0, 64>>() != cudaSuccess ||
      attn_configure<ChunkCfg<0, 128>>() != cudaSuccess || attn_configure<ChunkCfg<1, 64>>() != cudaSuccess ||
      attn_configure<ChunkCfg<1, 128>>() != cudaSuccess) {
    cudaGetLastError();
    cudaFree(c->mem);
    delete c;
    return MOE_ERR_CUDA;
  }
  *out = c;
  return MOE_OK;
}

int moe_attn_forward(moe_attn_ctx* ctx, void* stream, const moe_attn_args* a) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  const int st = attn_check(a);
  if (st != MOE_OK || a->N == 0 || a->B == 0) return st;
  DeviceGuard g(ctx->device);
  AttnParams p;
  p.a = *a;
  p.p_shift = __builtin_ctz((unsigned)a->page_size);
  p.scale_log2 = a->scale * 1.44269504088896340736f;
  p.err = ctx->err;
  p.tickets = ctx->tickets;
  p.parts = ctx->parts;
  p.G = a->Hq / a->Hkv;
  // A Q box is a whole number of 8-row swizzle atoms where that fits in a tile, so boxes can be
  // laid one behind the other; a tile is then a whole number of boxes.
  p.box_tok = 8 / std::gcd(p.G, 8);
  if (p.box_tok * p.G > kRows) p.box_tok = kRows / p.G;
  p.tpt = kRows / (p.box_tok * p.G) * p.box_tok;
  OpsPdl pdl;
  cudaStream_t s = (cudaStream_t)stream;
  if (a->dtype == MOE_DT_BF16)
    return a->D == 64 ? attn_by_rows<MOE_DT_BF16, 64>(ctx, p, s) : attn_by_rows<MOE_DT_BF16, 128>(ctx, p, s);
  return a->D == 64 ? attn_by_rows<MOE_DT_F16, 64>(ctx, p, s) : attn_by_rows<MOE_DT_F16, 128>(ctx, p, s);
}

int moe_attn_get_error(moe_attn_ctx* ctx, uint32_t* bits) {
  if (!ctx) return MOE_ERR_INVALID_ARG;
  DeviceGuard g(ctx->device);
  uint32_t v = 0;
  if (cudaDeviceSynchronize() != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaMemcpy(&v, ctx->err, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return MOE_ERR_CUDA;
  // a kernel that gave up leaves its tickets behind
  if (v && !clear_head(ctx)) return MOE_ERR_CUDA;
  if (bits) *bits = v;
  return v ? MOE_ERR_DEVICE_FLAG : MOE_OK;
}

int64_t moe_attn_device_bytes(const moe_attn_ctx* ctx) { return ctx ? (int64_t)ctx->bytes : 0; }

int moe_attn_destroy(moe_attn_ctx* ctx) {
  if (!ctx) return MOE_OK;
  DeviceGuard g(ctx->device);
  cudaFree(ctx->mem);
  delete ctx;
  return MOE_OK;
}

}  // extern "C"
