/*
 * moe_ops_gb300.h -- C ABI of the operators that stand beside the routed expert layer in a
 * decoder layer: the residual norm before attention and before the router, a serving step's
 * plan (positions, page tables, cache slots), rotary positions with the append to a paged
 * key/value cache, attention of each request's new tokens over its pages, drafted trees of
 * tokens (plan, attention, acceptance), and 8-bit projections (quantisation, product).
 *
 * Conventions are those of moe_gb300.h: MOE_OK or a negative moe_status, argument errors
 * detected on the host before anything is enqueued, streams as void* of the current device
 * (moe_attn_forward: of the handle's device), nothing allocated by a call, nothing
 * synchronised, every call may be captured in a CUDA graph, kernels never trap. Every kernel
 * here is launched with programmatic stream serialisation, waits for the kernel before it
 * before it touches memory (moe_matmul8_forward asks for its first weights to be brought into L2 before
 * that, and reads them after), and lets the next kernel launch early: a following kernel that
 * is itself launched with that attribute must wait on its grid dependency
 * (griddepcontrol.wait) before it reads these outputs, as for moe_forward.
 * 16-bit types: `dtype` is MOE_DT_BF16 or MOE_DT_F16 for every 16-bit tensor of a call.
 * Strides are in elements; the innermost dimension of every tensor is contiguous.
 * `err` (device uint32 or NULL): kernels OR the bits below into it; the caller clears it.
 */
#ifndef MOE_OPS_GB300_H
#define MOE_OPS_GB300_H

#include "moe_gb300.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_DT_BF16 0
#define MOE_DT_F16 1

/* Device error bits of the operators (same word layout as moe_get_error). */
#define MOE_OPS_ERR_PLAN 32u  /* a step did not fit: pages, table width, token capacity, or a negative length */
#define MOE_OPS_ERR_INDEX 64u /* a slot, page or request range outside its tensor (skipped, never accessed) */

/* Residual addition, root-mean-square norm and 8-bit output of T rows of width H:
 *   t = x + residual (fp32; residual NULL: t = x)      residual_out = round(t)
 *   y = t / sqrt(mean(t^2) + eps) * weight (fp32)      out = round(y)
 *   out8 = e4m3(y / s) rounded to nearest even, s = max|y| / 448 over the row (group 0) or
 *   over each `group` = 128 consecutive elements (the last block may be shorter); s in
 *   scales[row][block]. A block of zeros has s = 0 and zeros in out8, and so has one whose values are
 *   at most 448 * 2^-150, for which s rounds to 0.
 * The mean is of fp32 squares: it is that of the formula for |t| of 2^-60 to 2^56 (and below, where eps
 * is 2^-60 or more); a row whose squares overflow is divided by infinity, as by fp32 arithmetic throughout.
 * x, residual, out, residual_out [T][H] with row strides; weight [H] in dtype, or fp32 with
 * weight_f32 = 1. residual_out may be residual itself (in place) and out may be x itself;
 * no other overlap. out or out8 may be NULL (not both); scales goes with out8.
 * residual_out needs residual. 1 <= H <= 32768, T >= 0. err: bit 4 = a bounded wait gave up. */
typedef struct {
  const void* x;
  const void* residual;
  const void* weight;
  void* out;
  void* residual_out;
  uint8_t* out8;
  float* scales;
  uint32_t* err;
  int64_t x_stride, residual_stride, out_stride, residual_out_stride, out8_stride;
  int32_t T, H, dtype, weight_f32, group;
  float eps;
} moe_rmsnorm_args;
MOE_API int moe_add_rmsnorm(void* stream, const moe_rmsnorm_args* a);

/* One serving step of B requests over a paged cache, planned on the device from lengths.
 * Request b has ctx_lens[b] tokens in the cache and brings new_lens[b]; its row of
 * block_table holds the page of every `page_size` tokens. With have_b = ceil(ctx/P) and
 * end_b = ceil((ctx + new)/P), the missing pages are taken in request order from
 * free_pages, starting at *free_head, and entered into block_table[b][have_b .. end_b):
 * no other entry is written. Written for every b and every new token n of request b at
 * t = n - q_start[b]:
 *   q_start[B+1] exclusive sums of new_lens     kv_lens[b] = ctx + new
 *   positions[n] = ctx + t                      slots[n] = block_table[b][pos / P] * P + pos % P
 *   *free_head_out = free_head + pages taken
 * Entries of positions / slots past the last new token (up to N) are 0 / -1.
 * All or nothing: where the free pages, the table's width W or the capacity N do not
 * suffice, or a length is negative, MOE_OPS_ERR_PLAN is raised, the table is left as it
 * is, q_start and kv_lens are zeros, slots are -1, positions 0 and *free_head_out =
 * *free_head. No output (block_table, q_start, kv_lens, positions, slots, free_head_out, err) may
 * share a word with an input or with another output: other blocks may still read it. Such a call is
 * refused (MOE_ERR_INVALID_ARG); lengths and the head of the free list are kept in two copies.
 * 1 <= B <= MOE_PLAN_MAX_REQUESTS, F >= 0 (0: free_pages may be NULL), N >= 0 (0: positions and
 * slots may be NULL), page_size a power of two, W * page_size < 2^31. */
#define MOE_PLAN_MAX_REQUESTS 4096
typedef struct {
  const int32_t* ctx_lens;
  const int32_t* new_lens;
  int32_t* block_table;
  const int32_t* free_pages;
  const int32_t* free_head;
  int32_t* q_start;
  int32_t* kv_lens;
  int32_t* positions;
  int32_t* slots;
  int32_t* free_head_out;
  uint32_t* err;
  int64_t table_stride;
  int32_t B, W, F, N, page_size;
} moe_paged_plan_args;
MOE_API int moe_paged_plan(void* stream, const moe_paged_plan_args* a);

/* Rotary positions on q and k of N tokens; k and v appended to the paged cache.
 * Pair i (i < rot/2) of a head is elements (i, i + rot/2), or (2i, 2i+1) when interleaved;
 * elements rot .. D-1 pass unchanged. With angle = positions[n] * inv_freq[i]:
 *   (a, b) -> mscale * (a cos - b sin, a sin + b cos), rounded once.
 * inv_freq is fp64 (radians per position): scaling for long contexts is a choice of
 * inv_freq and mscale. The angle is reduced exactly, so large positions lose nothing.
 * Token n's k and v heads go to the cache at page slots[n] / P, row slots[n] % P; slot -1
 * skips the append (q is still rotated); a slot outside [-1, num_pages * P) raises
 * MOE_OPS_ERR_INDEX and is skipped. Two tokens must not share a slot.
 * q, q_out [N][Hq][D], k, v [N][Hkv][D] with token and head strides (q_out may be q, with its
 * strides; no other output shares an element with an input or another output);
 * caches with page, row and head strides (either order of rows and heads).
 * 2 <= rot <= D, rot even, D even, D <= 1024, P a power of two, num_pages * P < 2^31. */
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_cache;
  void* v_cache;
  const int32_t* positions;
  const int32_t* slots;
  const double* inv_freq;
  uint32_t* err;
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, qo_tok, qo_head;
  int64_t kc_page, kc_row, kc_head, vc_page, vc_row, vc_head;
  int32_t N, Hq, Hkv, D, rot, page_size, num_pages, interleaved, dtype;
  float mscale;
} moe_rotary_args;
MOE_API int moe_rotary_append(void* stream, const moe_rotary_args* a);

/* Attention of new tokens over a paged cache. Request b's new tokens are rows
 * q_start[b] .. q_start[b+1]-1 of q; its cache holds kv_lens[b] tokens, the new ones
 * (already appended) last. With c = kv_lens[b] - new, new token t sees keys j <= c + t:
 *   out[n][h] = sum_j softmax_j(scale * q[n][h] . k_j[g]) v_j[g],  g = h / (Hq / Hkv)
 *   lse[n][h] = ln sum_j exp(scale * q . k_j)   (fp32 [N][Hq], or NULL)
 * A row that sees no key (kv_lens < new) gets zeros and lse = -inf. Keys a row does not
 * see never reach it, whatever they hold. fp32 scores and sums; the weights are rounded to
 * dtype for the second product. Rows of q outside every request are not written; without rows
 * or without requests (N or B = 0) nothing is.
 * A page outside [0, num_pages) raises MOE_OPS_ERR_INDEX and counts as zeros; kv_lens beyond the
 * table's W * P raises it and counts as W * P (below 0: as 0); a request whose rows lie outside
 * [0, N] raises it and is skipped.
 * D is 64 or 128, Hq % Hkv == 0, Hq / Hkv <= 128, P a power of two of 16 to 1024, W * P < 2^30,
 * pointers 16-byte aligned and strides multiples of 8 elements (lse, tables: 4 bytes),
 * scale > 0, out shares no element with q. max_new: the most new tokens a request of this call
 * has, if known, else 0; it chooses a variant and never changes what is computed. */
typedef struct {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  void* out;
  float* lse;
  const int32_t* block_table;
  const int32_t* q_start;
  const int32_t* kv_lens;
  int64_t q_tok, q_head, out_tok, out_head;
  int64_t kc_page, kc_row, kc_head, vc_page, vc_row, vc_head;
  int64_t table_stride;
  int32_t N, B, Hq, Hkv, D, page_size, num_pages, W, max_new, dtype;
  float scale;
} moe_attn_args;

typedef struct moe_attn_ctx moe_attn_ctx; /* opaque: device workspace and error word */

/* Create a handle on `device` (sm_103). As with moe_ctx, one host thread and one stream
 * use it at a time. It is ready for any stream when the call returns (which waits for the
 * device's default stream). */
MOE_API int moe_attn_create(int device, moe_attn_ctx** out);
MOE_API int moe_attn_forward(moe_attn_ctx* ctx, void* stream, const moe_attn_args* a);
/* Read and clear the handle's device error word (synchronises the device): MOE_OK or
 * MOE_ERR_DEVICE_FLAG, *bits (may be NULL) the raw word (bit 4: a bounded wait gave up; what a
 * handle computes after that is not valid until this call has cleared it). */
MOE_API int moe_attn_get_error(moe_attn_ctx* ctx, uint32_t* bits);
/* Device bytes of the handle's workspace. */
MOE_API int64_t moe_attn_device_bytes(const moe_attn_ctx* ctx);
MOE_API int moe_attn_destroy(moe_attn_ctx* ctx);

/* ---- drafted tokens ------------------------------------------------------------------------
 * A step may bring a tree of drafted tokens for a request: its new tokens are the tree's nodes,
 * every node behind its parent, appended to the cache in that order. Node t's parent is
 * parents[q_start[b] + t], the parent's place in the request, or -1 where it follows the
 * cached tokens. A node sees the cached tokens, its ancestors and itself. */

/* Positions and masks of the nodes, once per step for all layers:
 *   depth[t] = parent < 0 ? 0 : depth[parent] + 1        positions[n] = ctx_lens[b] + depth
 *   mask[n]: bit j (bit j % 32 of word j / 32) is set where node t sees node j
 * parents [N], mask [N][words], positions [N]. A request with more than 32 * words new tokens
 * is a chunk without a tree: its parents have to be a chain (node t's is t - 1), its positions are
 * ctx + t, and its mask is neither written here nor read by moe_attn_forward_tree, which lets its
 * tokens see what is before them. A parent outside [-1, t), a longer request that is no chain, or a
 * negative context raises MOE_OPS_ERR_PLAN and counts as -1, as a chain, as 0; a request whose
 * rows lie outside [0, N] raises MOE_OPS_ERR_INDEX and is skipped. Rows of no request are not
 * written. No output shares a word with an input or another output. 1 <= words <= MOE_TREE_WORDS. */
#define MOE_TREE_WORDS 8
typedef struct {
  const int32_t* parents;
  const int32_t* q_start;
  const int32_t* ctx_lens;
  int32_t* positions;
  int32_t* mask;
  uint32_t* err;
  int32_t N, B, words;
} moe_tree_plan_args;
MOE_API int moe_tree_plan(void* stream, const moe_tree_plan_args* a);

/* moe_attn_forward for requests with trees: of a request with at most 32 * words new tokens,
 * row t sees the c = kv_lens - new cached keys and new key j where bit j of mask[n] is set (any
 * bits: a row need not see itself, bits from the number of new tokens on are ignored); of a longer one
 * it sees keys j <= c + t. A row that sees nothing gets zeros and lse = -inf. mask int32
 * [N][words], which shares no element with out or lse; everything else as in moe_attn_forward. */
MOE_API int moe_attn_forward_tree(moe_attn_ctx* ctx, void* stream, const moe_attn_args* a, const int32_t* mask,
                                  int32_t words);

/* The drafted tokens that the model's own tokens confirm, and their keys and values moved to the
 * places that the next step expects. tokens[n] is a node's token, targets[n] the token that the
 * model gives after it. The first c = certain[b] nodes of a request (1 where certain is NULL: the
 * root, decided by the step before) are a chain that stays in any case; then from cur = c - 1
 *   child = the lowest j > cur, j >= c, with parents[j] == cur and tokens[j] == targets[cur]
 * is taken while there is one, at most `depth` times:
 *   path[b][i] = the i-th node taken (-1 behind the last)      accepted[b] = c + nodes taken
 *   ctx_out[b] = ctx_lens[b] + accepted[b]                     next_tokens[b] = targets[cur]
 * and row ctx + path[b][i] of the caches goes to row ctx + c + i, in all layers. Other rows stay.
 * A request without new tokens has accepted 0 and next_tokens -1. tokens, targets [N], path
 * [B][depth]; a cache is [layers][pages][page_size][Hkv][D] of 16-bit elements with strides.
 * certain outside [1, new] raises MOE_OPS_ERR_PLAN and is clamped; a row whose page is outside
 * [0, num_pages) or whose place is outside the table raises MOE_OPS_ERR_INDEX and is not moved; a
 * request whose rows lie outside [0, N] raises it and counts as without new tokens. No output
 * shares a word with an input or another output; k_cache and v_cache share no element; a page
 * belongs to one request. 1 <= depth <= 32 * MOE_TREE_WORDS, layers >= 1, B <= 65535,
 * P a power of two, W * P < 2^31. */
typedef struct {
  const int32_t* parents;
  const int32_t* tokens;
  const int32_t* targets;
  const int32_t* q_start;
  const int32_t* ctx_lens;
  const int32_t* certain;
  const int32_t* block_table;
  void* k_cache;
  void* v_cache;
  int32_t* path;
  int32_t* accepted;
  int32_t* ctx_out;
  int32_t* next_tokens;
  uint32_t* err;
  int64_t table_stride;
  int64_t kc_layer, kc_page, kc_row, kc_head, vc_layer, vc_page, vc_row, vc_head;
  int32_t N, B, W, depth, layers, Hkv, D, page_size, num_pages;
} moe_tree_accept_args;
MOE_API int moe_tree_accept(void* stream, const moe_tree_accept_args* a);

/* ---- 8-bit projections ----------------------------------------------------------------------
 * Values in e4m3 with fp32 scales, s = max|x| / 448 over each block:
 *   out8 = e4m3(x / s), the quotient in fp32, rounded to nearest even
 * rows 1: blocks of `group` = 128 consecutive elements of a row, or the row (group 0); rows 128
 * (with group 128): blocks of 128 x 128, as moe_matmul8_forward takes weights. Blocks at the ends may be
 * smaller. scales [ceil(T / rows)][ceil(H / group)], contiguous. A block of zeros has s = 0 and zeros; a NaN
 * makes its block's scale and values NaN; an infinity its scale infinite, itself NaN and the
 * others 0. x [T][H] of dtype, out8 [T][H], rows strided; the memory that x, out8 and scales span, from first
 * to last element, does not overlap. 1 <= H <= 2^30. */
typedef struct {
  const void* x;
  uint8_t* out8;
  float* scales;
  int64_t x_stride, out8_stride;
  int32_t T, H, dtype, group, rows;
} moe_quantize8_args;
MOE_API int moe_quantize8(void* stream, const moe_quantize8_args* a);

/* Product of e4m3 activations and weights with scales per block of 128 along K:
 *   out[t][n] = sum_b a_scales[t][b] * w_scales[n / 128][b] * sum_{k in block b} a8[t][k] w8[n][k]
 * from left to right in fp32: the product of the two scales is formed first, the products of a block are summed by
 * the tensor cores, and the blocks are added up; out is rounded once to dtype. So a product of scales below 2^-126 is
 * rounded to a multiple of 2^-149, by which a block's term is off by 2^-125 at most, and one of 2^128 or more is infinite and
 * makes the term infinite, or NaN where the block's sum is 0.
 * a8 [T][K], w8 [N][K] (a library layer's [out][in]), out [T][N]; w_scales [ceil(N / 128)][ceil(K / 128)];
 * a_scales [T][a_blocks], a_blocks = ceil(K / 128), or 1 for a scale per row. The scales are as moe_add_rmsnorm (group 0, 128) and moe_quantize8 write them;
 * rows of every tensor may be strided. K a multiple of 16, a8 and w8 16-byte aligned with row strides that
 * are multiples of 16; out is aligned to its elements. The memory from out's first to its last element
 * overlaps no input's.
 * 0 <= T, N <= 2^30 (T or N 0: nothing is done), 16 <= K <= 2^20, ceil(T / 128) * ceil(N / 128) <= 2^30. */
typedef struct {
  const uint8_t* a8;
  const float* a_scales;
  const uint8_t* w8;
  const float* w_scales;
  void* out;
  int64_t a8_stride, a_scales_stride, w8_stride, w_scales_stride, out_stride;
  int32_t T, N, K, a_blocks, dtype;
} moe_matmul8_args;

typedef struct moe_matmul8_ctx moe_matmul8_ctx; /* opaque: device workspace and error word */

/* Handle, error word and workspace: as moe_attn_create and the calls behind it. */
MOE_API int moe_matmul8_create(int device, moe_matmul8_ctx** out);
MOE_API int moe_matmul8_forward(moe_matmul8_ctx* ctx, void* stream, const moe_matmul8_args* a);
MOE_API int moe_matmul8_get_error(moe_matmul8_ctx* ctx, uint32_t* bits);
MOE_API int64_t moe_matmul8_device_bytes(const moe_matmul8_ctx* ctx);
MOE_API int moe_matmul8_destroy(moe_matmul8_ctx* ctx);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_GB300_H */
