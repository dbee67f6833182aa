// Trees of drafted tokens: their plan and their acceptance. Interfaces and formulas: include/moe_ops_gb300.h.
// (Attention with a tree's masks: attn.cu.)
#include <algorithm>

#include "ops_internal.cuh"

namespace moe {

namespace {

constexpr int kTreeNodes = 32 * MOE_TREE_WORDS;

// ---- positions and masks -----------------------------------------------------------------------

// A node's mask is the union of its ancestors' bits and its depth their number less one. Pointers double: with
// mask[t] the bits of t and of the ancestors up to up[t] (exclusive), mask[t] |= mask[up[t]] and up[t] = up[up[t]] reach the
// root in log2(depth) rounds, where a walk would take depth steps (a chain of 256 nodes: 8 rounds).
// `per` threads (a power of two, 32 * words or more) take a request.
__global__ void __launch_bounds__(kTreeNodes) tree_plan_kernel(const moe_tree_plan_args a, int per_shift) {
  __shared__ uint32_t s_mask[MOE_TREE_WORDS][kTreeNodes];
  __shared__ int16_t s_up[kTreeNodes];
  __shared__ int s_chunk[kTreeNodes / 32][3];  // of each of the block's requests that is a chunk: tokens, first row, context
  pdl_entry();
  const int tid = threadIdx.x, per = 1 << per_shift, t = tid & (per - 1), g0 = tid - t, W = a.words;
  const int64_t request = (int64_t)blockIdx.x * (kTreeNodes >> per_shift) + (tid >> per_shift);
  uint32_t bad = 0;
  int n = 0, start = 0, ctx = 0;
  if (request < a.B) {
    start = a.q_start[request];
    const int end = a.q_start[request + 1];
    ctx = a.ctx_lens[request];
    if (start < 0 || end < start || end > a.N) bad = kErrIndex;
    else n = end - start;
    if (ctx < 0) {
      bad |= kErrPlan;
      ctx = 0;
    }
  }
  const bool tree = n <= 32 * W;
  int up = -1;
  uint32_t mask[MOE_TREE_WORDS];
#pragma unroll
  for (int w = 0; w < MOE_TREE_WORDS; ++w) mask[w] = t >> 5 == w ? 1u << (t & 31) : 0;
  if (t == 0) {
    int* c = s_chunk[tid >> per_shift];
    c[0] = tree ? 0 : n;
    c[1] = start;
    c[2] = ctx;
  }
  if (tree && t < n) {
    up = a.parents[start + t];
    if (up < -1 || up >= t) {
      up = -1;
      bad |= kErrPlan;
    }
  }
  s_up[tid] = (int16_t)up;
#pragma unroll
  for (int w = 0; w < MOE_TREE_WORDS; ++w)
    if (w < W) s_mask[w][tid] = mask[w];
  while (__syncthreads_or(up >= 0)) {
    const int at = g0 + up;
    int next = -1;
    if (up >= 0) {
      next = s_up[at];
#pragma unroll
      for (int w = 0; w < MOE_TREE_WORDS; ++w)
        if (w < W) mask[w] |= s_mask[w][at];
    }
    __syncthreads();
    if (up >= 0) {
      s_up[tid] = (int16_t)next;
#pragma unroll
      for (int w = 0; w < MOE_TREE_WORDS; ++w)
        if (w < W) s_mask[w][tid] = mask[w];
    }
    up = next;
  }
  // chunks by the whole block (the loop above has synchronised it): 16 trees take 2.3 us, beside a chunk of 2,048 tokens 2.3, of 8,192 4.3, of
  // 60,000 21
  for (int g = 0; g < kTreeNodes >> per_shift; ++g) {
    const int tokens = s_chunk[g][0], row = s_chunk[g][1], from = s_chunk[g][2];
#pragma unroll 4
    for (int i = tid; i < tokens; i += kTreeNodes) {
      if (a.parents[row + i] != i - 1) bad |= kErrPlan;
      a.positions[row + i] = from + i;
    }
  }
  if (tree && t < n) {
    int depth = -1;
#pragma unroll
    for (int w = 0; w < MOE_TREE_WORDS; ++w)
      if (w < W) {
        depth += __popc(mask[w]);
        a.mask[(int64_t)(start + t) * W + w] = (int32_t)mask[w];
      }
    a.positions[start + t] = ctx + depth;
  }
  if (bad && a.err) atomicOr(a.err, bad);
}

// ---- acceptance --------------------------------------------------------------------------------

constexpr int kAcceptThreads = 256;
constexpr int kMoves = 4;  // rows a thread has in flight
constexpr int kNodesHeld = 512;  // nodes of a request that are walked in shared memory

struct AcceptParams {
  moe_tree_accept_args a;
  int p_shift;
};

// Every block of a request walks down the tree for itself (its first warp, 32 nodes at a time; a step's three loads one after
// another are what bounds small calls, so the nodes are brought to shared memory at once), then moves its share of the
// pieces of PE elements. A thread moves a piece of all rows, in the order of the path and in batches that are
// read before they are written: a row's source is never before its destination, and sources grow, so no row is
// overwritten before it is read.
template <typename Piece, int PE>
__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(const __grid_constant__ AcceptParams p) {
  const moe_tree_accept_args& a = p.a;
  __shared__ int s_path[kTreeNodes];
  __shared__ int2 s_src[kTreeNodes], s_dst[kTreeNodes];  // page and row of the rows that move
  __shared__ int s_moves;
  __shared__ int s_parent[kNodesHeld], s_token[kNodesHeld], s_target[kNodesHeld];
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.y;
  const int start = a.q_start[b], end = a.q_start[b + 1], ctx = a.ctx_lens[b];
  const bool first_block = blockIdx.x == 0;
  const bool inside = start >= 0 && end >= start && end <= a.N;
  const int n = inside ? end - start : 0;
  const bool held = n <= kNodesHeld;
  if (held)
    for (int i = tid; i < n; i += kAcceptThreads) {
      s_parent[i] = a.parents[start + i];
      s_token[i] = a.tokens[start + i];
      s_target[i] = a.targets[start + i];
    }
  __syncthreads();
  if (tid < 32) {
    uint32_t bad = 0;
    const int* parents = held ? s_parent : a.parents + start;
    const int* tokens = held ? s_token : a.tokens + start;
    const int* targets = held ? s_target : a.targets + start;
    if (!inside) bad |= kErrIndex;
    int c = n ? 1 : 0;
    if (a.certain && n) {
      c = a.certain[b];
      if (c < 1 || c > n) {
        bad |= kErrPlan;
        c = max(1, min(c, n));
      }
    }
    int cur = c - 1, count = 0, target = -1;
    while (n) {
      target = targets[cur];
      if (count == a.depth) break;
      int child = -1;
      for (int j0 = cur + 1; j0 < n && child < 0; j0 += 32) {
        const int j = j0 + lane;
        const bool hit = j < n && parents[j] == cur && tokens[j] == target;
        const uint32_t hits = __ballot_sync(0xFFFFFFFFu, hit);
        if (hits) child = j0 + __ffs(hits) - 1;
      }
      if (child < 0) break;
      cur = child;
      if (lane == 0) s_path[count] = cur;
      ++count;
    }
    __syncwarp();
    if (first_block) {
      for (int i = lane; i < a.depth; i += 32) a.path[(int64_t)b * a.depth + i] = i < count ? s_path[i] : -1;
      if (lane == 0) {
        a.accepted[b] = c + count;
        a.ctx_out[b] = ctx + c + count;
        a.next_tokens[b] = n ? target : -1;
      }
    }
    // the rows that move: those behind the nodes that are where they belong already
    int moves = 0;
    for (int i0 = 0; i0 < count; i0 += 32) {
      const int i = i0 + lane;
      bool move = i < count && s_path[i] != c + i;
      int2 src = make_int2(0, 0), dst = src;
      if (move) {
        const auto place = [&](int64_t at, int2& to) {
          const int64_t col = at >> p.p_shift;
          if (at < 0 || col >= a.W) return false;
          to.x = a.block_table[b * a.table_stride + col];
          to.y = (int)(at & (a.page_size - 1));
          return to.x >= 0 && to.x < a.num_pages;
        };
        if (!place((int64_t)ctx + s_path[i], src) || !place((int64_t)ctx + c + i, dst)) {
          bad |= kErrIndex;
          move = false;
        }
      }
      const uint32_t some = __ballot_sync(0xFFFFFFFFu, move);
      if (move) {
        const int at = moves + __popc(some & ((1u << lane) - 1));
        s_src[at] = src;
        s_dst[at] = dst;
      }
      moves += __popc(some);
    }
    if (lane == 0) s_moves = moves;
    if (first_block && bad && a.err) atomicOr(a.err, bad);
  }
  __syncthreads();
  const int moves = s_moves;
  if (moves == 0) return;
  const int per_head = a.D / PE;
  const int64_t per_layer = (int64_t)a.Hkv * per_head, pieces = 2 * a.layers * per_layer;
  for (int64_t x = (int64_t)blockIdx.x * kAcceptThreads + tid; x < pieces; x += (int64_t)gridDim.x * kAcceptThreads) {
    const int64_t l2 = x / per_layer;
    const int rest = (int)(x - l2 * per_layer), h = rest / per_head, d = rest - h * per_head;
    const bool is_v = l2 >= a.layers;
    const int64_t layer = is_v ? l2 - a.layers : l2;
    uint16_t* base = is_v ? (uint16_t*)a.v_cache + layer * a.vc_layer + h * a.vc_head + d * PE
                          : (uint16_t*)a.k_cache + layer * a.kc_layer + h * a.kc_head + d * PE;
    const int64_t page = is_v ? a.vc_page : a.kc_page, row = is_v ? a.vc_row : a.kc_row;
    const auto at = [&](int2 to) { return reinterpret_cast<Piece*>(base + to.x * page + to.y * row); };
    for (int i = 0; i < moves; i += kMoves) {
      Piece v[kMoves];
#pragma unroll
      for (int u = 0; u < kMoves; ++u)
        if (i + u < moves) v[u] = *at(s_src[i + u]);
#pragma unroll
      for (int u = 0; u < kMoves; ++u)
        if (i + u < moves) *at(s_dst[i + u]) = v[u];
    }
  }
}

template <typename Piece, int PE>
cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s) {
  const int64_t pieces = (int64_t)2 * p.a.layers * p.a.Hkv * (p.a.D / PE);
  const int64_t most = std::max<int64_t>(1, (int64_t)8 * sm_count() / p.a.B);
  const int64_t blocks = std::min((pieces + kAcceptThreads - 1) / kAcceptThreads, most);
  return launch_pdl(tree_accept_kernel<Piece, PE>, dim3((unsigned)blocks, (unsigned)p.a.B), dim3(kAcceptThreads), 0, s, p);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_tree_plan(void* stream, const moe_tree_plan_args* a) {
  if (!a || a->N < 0 || a->B < 0 || a->words < 1) return MOE_ERR_INVALID_ARG;
  if (a->words > MOE_TREE_WORDS) return MOE_ERR_UNSUPPORTED;
  if (a->N == 0 || a->B == 0) return MOE_OK;
  const void* ptrs[] = {a->parents, a->q_start, a->ctx_lens, a->positions, a->mask};
  for (const void* q : ptrs)
    if (!q || !is_aligned(q, 4)) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(a->err, 4)) return MOE_ERR_INVALID_ARG;
  const Words t[] = {{a->positions, a->N},  {a->mask, (int64_t)a->N * a->words}, {a->err, a->err ? 1 : 0},  // outputs up to here
                     {a->parents, a->N},    {a->q_start, (int64_t)a->B + 1},     {a->ctx_lens, a->B}};
  if (shares_words(t, 3, 6)) return MOE_ERR_INVALID_ARG;
  const int per_shift = shift_of(32 * a->words), requests = kTreeNodes >> per_shift;
  OpsPdl pdl;
  return launch_pdl(tree_plan_kernel, dim3((unsigned)(((int64_t)a->B + requests - 1) / requests)), dim3(kTreeNodes), 0,
                    (cudaStream_t)stream, *a, per_shift) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int moe_tree_accept(void* stream, const moe_tree_accept_args* a) {
  if (!a || a->N < 0 || a->B < 0 || a->W < 1 || a->depth < 1 || a->layers < 1 || a->Hkv < 1 || a->D < 1 || a->num_pages < 1 ||
      !is_pow2(a->page_size) || a->table_stride < a->W)
    return MOE_ERR_INVALID_ARG;
  if (a->depth > kTreeNodes || a->B > 65535 || (int64_t)a->W * a->page_size >= ((int64_t)1 << 31) ||
      (int64_t)a->Hkv * a->D >= ((int64_t)1 << 30))
    return MOE_ERR_UNSUPPORTED;
  if (a->B == 0) return MOE_OK;
  const void* per_node[] = {a->parents, a->tokens, a->targets};
  for (const void* q : per_node)
    if ((!q && a->N > 0) || !is_aligned(q, 4)) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {a->q_start, a->ctx_lens, a->block_table, a->path, a->accepted, a->ctx_out, a->next_tokens};
  for (const void* q : ptrs)
    if (!q || !is_aligned(q, 4)) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(a->certain, 4) || !is_aligned(a->err, 4) || !a->k_cache || !a->v_cache || !is_aligned(a->k_cache, 2) ||
      !is_aligned(a->v_cache, 2))
    return MOE_ERR_INVALID_ARG;
  // a row goes in pieces of 16 bytes where all strides and addresses allow it
  bool wide = a->D % 8 == 0 && is_aligned(a->k_cache, 16) && is_aligned(a->v_cache, 16);
  const int64_t strides[] = {a->kc_layer, a->kc_page, a->kc_row, a->kc_head, a->vc_layer, a->vc_page, a->vc_row, a->vc_head};
  const int64_t extents[] = {a->layers, a->num_pages, a->page_size, a->Hkv};
  for (int i = 0; i < 8; ++i) {
    if (strides[i] < 0) return MOE_ERR_INVALID_ARG;
    if (extents[i & 3] > 1 && strides[i] % 8) wide = false;
  }
  const Words t[] = {{a->path, (int64_t)a->B * a->depth},
                     {a->accepted, a->B},
                     {a->ctx_out, a->B},
                     {a->next_tokens, a->B},
                     {a->err, a->err ? 1 : 0},  // outputs up to here
                     {a->parents, a->N},
                     {a->tokens, a->N},
                     {a->targets, a->N},
                     {a->q_start, (int64_t)a->B + 1},
                     {a->ctx_lens, a->B},
                     {a->certain, a->certain ? a->B : 0},
                     {a->block_table, (a->B - 1) * a->table_stride + a->W}};
  if (shares_words(t, 5, 12)) return MOE_ERR_INVALID_ARG;
  AcceptParams p;
  p.a = *a;
  p.p_shift = shift_of(a->page_size);
  OpsPdl pdl;
  const cudaError_t e = wide ? launch_accept<uint4, 8>(p, (cudaStream_t)stream) : launch_accept<uint16_t, 1>(p, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
