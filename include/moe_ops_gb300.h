/*
 * moe_ops_gb300.h -- C ABI of the operators that stand beside the routed expert layer in a
 * decoder layer: the residual norm before attention and before the router, a serving step's
 * plan (positions, page tables, cache slots), rotary positions with the append to a paged
 * key/value cache, and attention of each request's new tokens over its pages.
 *
 * Conventions are those of moe_gb300.h: MOE_OK or a negative moe_status, argument errors
 * detected on the host before anything is enqueued, streams as void* of the current device
 * (moe_attn_forward: of the handle's device), nothing allocated by a call, nothing
 * synchronised, every call may be captured in a CUDA graph, kernels never trap. Every kernel
 * here is launched with programmatic stream serialisation, waits for the kernel before it
 * before it touches memory, and lets the next kernel launch early: a following kernel that
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

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_GB300_H */
