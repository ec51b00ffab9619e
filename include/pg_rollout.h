/*
 * Building blocks of the rollout: generating the G responses of a shared-prefix group token by
 * token.  The prefix's keys and values are kept once, in pages of its own; every response has pages
 * for its own keys and values; one step appends one token per response, attends with its query to
 * the shared prefix and the response's own pages, and samples the next token.  (The skill page
 * "prefix-grouper-grpo" takes the responses of a group as given; this produces them from the same
 * sharing pattern: Pith review of Prefix Grouper, "Core claim".)
 * Same conventions as pg_grouped_attn.h: caller-owned device buffers, asynchronous on `stream`,
 * host-side argument checks, no allocation.
 *
 * The paged cache.  k_cache and v_cache are [num_pages, page_size, Hkv, d], contiguous, 16-byte
 * aligned, bf16 or fp32; page_size is 16, 32, 64, 128 or 256.  A page table row lists the pages of
 * one sequence of keys: key i lies in slot i % page_size of page pages[row][i / page_size].  Slots
 * that hold no key yet may hold anything, NaN included.
 */
#ifndef PG_ROLLOUT_H
#define PG_ROLLOUT_H

#include "pg_grouped_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Append n_tokens tokens to the cache, rotating on the way:
 *   K[slot(n), h] = rotate(k[n, h], p_n),  V[slot(n), h] = v[n, h],  q_out[n, h] = rotate(q[n, h], p_n)
 * with rotate the rotate-half RoPE of the attention calls (pairs (j, j + d/2), angle p_n *
 * rope_theta^(-2j/d); rope_theta 0: no rotation), p_n = positions[n] (NULL: cache_pos[n]) and
 * slot(n) given by index cache_pos[n] of page table row page_rows[n] (NULL: row n).
 *   q [n_tokens, Hq, d] rows ldq elements apart, or NULL with heads_q = 0; q_out [n_tokens, Hq, d]
 *   contiguous (may be q itself when ldq = Hq * d); k, v [n_tokens, Hkv, d] rows ldk, ldv apart
 *   pages int32 [num_page_rows] rows of pages_per_row, pages_stride elements apart (device);
 *   page_rows, cache_pos, positions int32 [n_tokens] (device)
 * All of dtype `dtype`, pointers 16-byte aligned, ldq, ldk, ldv multiples of 16 bytes covering a row.
 * A token whose cache_pos is negative (a padding row) is not stored; its q row is still rotated.
 * A token whose page table row, index or page is out of range is not stored either, and
 * PG_ERR_DEVICE is recorded in the status word.  No two stored tokens may share a slot: the slot
 * then holds parts of either.
 * Errors: PG_ERR_INVALID_ARG (host check, nothing launched); PG_ERR_CUDA on a launch failure.
 */
pg_status pg_cache_append(pg_dtype dtype, int64_t n_tokens, int32_t heads_q, int32_t heads_kv,
                          int32_t head_dim, const void* q, int64_t ldq, void* q_out, const void* k,
                          int64_t ldk, const void* v, int64_t ldv, const int32_t* positions,
                          float rope_theta, void* k_cache, void* v_cache, int64_t num_pages,
                          int32_t page_size, const int32_t* pages, int32_t num_page_rows,
                          int32_t pages_per_row, int64_t pages_stride, const int32_t* page_rows,
                          const int32_t* cache_pos, pg_stream_t stream);

/*
 * The paged cache in 8 bits: half the bytes to keep and to read.  k_codes and v_codes are
 * [num_pages, page_size, Hkv, d] e4m3 numbers (4 exponent bits, bias 7; 3 fraction bits; no infinity,
 * largest 448), k_scales and v_scales fp32 [num_pages, page_size / 16, Hkv], all contiguous and 16-byte
 * aligned: a slot's value is its code times the scale of its block, the 16 slots of a page from a multiple of
 * 16 on.  A scale is a power of two 2^e, -126 <= e <= 120, or 0 for a block without tokens.
 *
 * pg_cache_append_e4m3 appends as pg_cache_append does, and writes to the blocks of the appended tokens
 *   e = max(e_before, the least e >= -126 with |x| <= 448 * 2^e for all finite appended values x)
 * (e_before: the block's scale so far, if its first slot is not among the appended), the codes
 * round(x 2^-e), ties to even, of the appended values, and where e > e_before the earlier codes
 * again as round(code 2^(e_before - e)); that is exact but for codes that become smaller than 2^-6, whose
 * steps are 2^-9.  Rotated keys are rounded once, from fp32.  Values that are not finite are stored as NaN.
 * So tokens of a block have to be appended in order, from its first slot on, and in one call the tokens of a
 * block have to follow one another directly (a prompt's tokens in order, one token per response, or
 * rows of a padded batch); a block whose tokens are apart in one call, or that two calls at once append to,
 * holds parts of either.  Appending to an index again (a step that is taken back) keeps the scale it had.
 * Padding rows and bad tokens as in pg_cache_append; q and q_out as there.  n_tokens below 2^27.
 */
pg_status pg_cache_append_e4m3(pg_dtype dtype, int64_t n_tokens, int32_t heads_q, int32_t heads_kv,
                               int32_t head_dim, const void* q, int64_t ldq, void* q_out,
                               const void* k, int64_t ldk, const void* v, int64_t ldv,
                               const int32_t* positions, float rope_theta, void* k_codes,
                               void* v_codes, float* k_scales, float* v_scales, int64_t num_pages,
                               int32_t page_size, const int32_t* pages, int32_t num_page_rows,
                               int32_t pages_per_row, int64_t pages_stride,
                               const int32_t* page_rows, const int32_t* cache_pos,
                               pg_stream_t stream);

/*
 * The values of n_tokens tokens of the cache, k and v [n_tokens, Hkv, d] of dtype `dtype`, contiguous and
 * 16-byte aligned: token n is index cache_pos[n] of page table row page_rows[n] (NULL: row n), as in
 * the append (a cached prefix's keys and values, to prefill what follows it).  A negative cache_pos gives zeros;
 * so does a row, index or page out of range, recorded as PG_ERR_DEVICE.  n_tokens below 2^27.
 */
pg_status pg_cache_read_e4m3(pg_dtype dtype, int64_t n_tokens, int32_t heads_kv, int32_t head_dim,
                             const void* k_codes, const void* v_codes, const float* k_scales,
                             const float* v_scales, int64_t num_pages, int32_t page_size,
                             const int32_t* pages, int32_t num_page_rows, int32_t pages_per_row,
                             int64_t pages_stride, const int32_t* page_rows,
                             const int32_t* cache_pos, void* k, void* v, pg_stream_t stream);

/*
 * Host-side summary of a rollout's attention step, filled by pg_plan_decode / pg_plan_decode_host.
 * It holds for the whole rollout: the number of keys each response has so far is read on the device.
 */
typedef struct pg_decode_plan {
  int32_t num_groups;      /* B */
  int32_t num_seqs;        /* S: responses over all groups, group by group */
  int32_t heads_q, heads_kv, head_dim;
  int32_t dtype;           /* pg_dtype */
  int32_t page_size;
  int32_t own_pages;       /* page table width of a response: at most own_pages * page_size own keys */
  int64_t max_prefix;      /* the longest prefix */
  int32_t n_items;         /* work items per key/value head: a part of a prefix for seqs_per_item */
  int32_t seqs_per_item;   /* responses (up to 128 query rows) at most */
  int32_t prefix_slots;    /* partial results per query row: parts of its prefix ... */
  int32_t own_slots;       /* ... and of its own keys */
  int32_t simt_splits;     /* partial results per query row of the SIMT kernel */
  int32_t own_slots_e4m3;  /* own_slots of the call over a cache in 8 bits: at most, as far as responses are long */
  int64_t off_seqs;        /* byte offsets in the tables: per-response records, */
  int64_t off_items;       /* work items */
  int64_t table_bytes;
  size_t workspace_bytes;  /* workspace of pg_decode_attn, and the least of pg_decode_attn_e4m3 */
  size_t workspace_bytes_e4m3; /* workspace that has room for all own_slots_e4m3 */
  const void* tables;
} pg_decode_plan;

/*
 * Bytes of the tables of a plan.  prefix_lens[num_groups] and group_sizes[num_groups] are host
 * arrays: group b's responses share a prefix of prefix_lens[b] keys.
 * Errors: PG_ERR_INVALID_ARG if num_groups < 1, a length or group size is negative or a prefix is
 * 2^30 or longer, there is no response or there are 2^20 or more, own_pages * page_size >= 2^30, or
 * for a dtype, head count, head_dim (64 or 128) or page size that is not supported.
 */
pg_status pg_plan_decode_size(int32_t num_groups, const int32_t* prefix_lens,
                              const int32_t* group_sizes, pg_dtype dtype, int32_t heads_q,
                              int32_t heads_kv, int32_t head_dim, int32_t page_size,
                              int32_t own_pages, int64_t* table_bytes);

/* Build the plan's tables in a caller host buffer (no CUDA call) and fill *plan. */
pg_status pg_plan_decode_host(int32_t num_groups, const int32_t* prefix_lens,
                              const int32_t* group_sizes, pg_dtype dtype, int32_t heads_q,
                              int32_t heads_kv, int32_t head_dim, int32_t page_size,
                              int32_t own_pages, void* tables, int64_t table_bytes,
                              pg_decode_plan* plan);

/* pg_plan_decode_host into a temporary buffer, then a copy to the caller's device buffer on `stream`
 * (as pg_pack).  PG_ERR_INVALID_ARG while `stream` is being captured into a graph: the temporary buffer
 * is gone when the graph is replayed. */
pg_status pg_plan_decode(int32_t num_groups, const int32_t* prefix_lens,
                         const int32_t* group_sizes, pg_dtype dtype, int32_t heads_q,
                         int32_t heads_kv, int32_t head_dim, int32_t page_size, int32_t own_pages,
                         void* tables_dev, int64_t table_bytes, pg_decode_plan* plan,
                         pg_stream_t stream);

/*
 * Attention of one query token per response over its group's prefix and its own keys:
 *   o[s, h] = sum_j p_j v_j,  p = softmax_j(scale q[s, h] . k_j),  lse[h, s] = ln sum_j exp(scale q . k_j)
 * where j runs over the prefix_lens[b] prefix keys of s's group b (row b of prefix_pages) and the
 * first own_lens[s] own keys (row s of own_pages).  q [S, Hq, d] and the cached keys are already
 * rotated.  A response without any key gets o = 0 and lse = -inf.  The group's prefix keys and
 * values are read once per key/value head for (128 Hkv / Hq) responses at a time.
 *   q, o [S, Hq, d], lse [Hq, S] fp32; prefix_pages int32, rows prefix_stride elements apart (may be
 *   NULL when every prefix is empty); own_pages int32, rows own_stride apart, own_lens int32 [S]
 *   (both may be NULL when the plan's own_pages is 0); all on the device, q, o, the caches, lse and
 *   the workspace 16-byte aligned
 * own_lens[s] <= 0 means no own keys; a length above own_pages * page_size is cut to it and a page
 * outside [0, num_pages) reads as zero keys and values, both with PG_ERR_DEVICE in the status word.
 * With bf16 caches the softmax weights are rounded to bf16 for the product with the values (their sum
 * is of the fp32 weights), as in the attention calls; with PG_FLAG_SIMT they are not.
 * num_pages * page_size must be below 2^31.  opts: softmax_scale (0: d^-1/2) and flags (0, or
 * PG_FLAG_SIMT for the fp32-arithmetic kernel); rope_theta and debug must be 0.  Every element of o
 * and lse is written; results do not depend on the order in which CTAs run.  The workspace
 * (plan->workspace_bytes) carries nothing from call to call; calls that may overlap need one each.
 * Errors: PG_ERR_INVALID_ARG (host check, nothing launched); PG_ERR_CUDA on a launch failure.
 */
pg_status pg_decode_attn(const pg_decode_plan* plan, const void* q, const void* k_cache,
                         const void* v_cache, int64_t num_pages, const int32_t* prefix_pages,
                         int64_t prefix_stride, const int32_t* own_pages, int64_t own_stride,
                         const int32_t* own_lens, void* o, float* lse, const pg_opts* opts,
                         void* workspace, size_t workspace_bytes, pg_stream_t stream);

/*
 * pg_decode_attn over a cache in 8 bits (its layout at pg_cache_append_e4m3): keys and values are the codes
 * times their block's scale.  The same plan (its dtype is that of q and o), options and rules.  The workspace
 * has plan->workspace_bytes at least; with plan->workspace_bytes_e4m3 long responses are shared by as many CTAs
 * as pay off, with less by as many as it has room for.  A block's scale is a power of two; scales of blocks
 * without a key that is attended to are not used, whatever they hold.
 * Tensor-core kernels (bf16): the codes enter the products as they are, the rest is rounded so.  Over the
 * prefix the query is the sum of two e4m3 numbers, exact to 2^-17 of its row's largest element, and a weight
 * (times the scale of its value, relative to the row's largest such product) the sum of an e5m2 and an e4m3
 * number, off by 2^-7 of itself at most or by 2^-17 of the largest.  Over the own keys both are fp16 numbers: the query
 * exact to 2^-31 of its row's largest element, a weight off by 2^-11 of itself or by 2^-31 of the largest.  The weights'
 * sum is of the fp32 ones.  A scale of values below 2^-118 of the largest that a row has met counts as that.  PG_FLAG_SIMT
 * computes with fp32 queries and weights instead.
 */
pg_status pg_decode_attn_e4m3(const pg_decode_plan* plan, const void* q, const void* k_codes,
                              const void* v_codes, const float* k_scales, const float* v_scales,
                              int64_t num_pages, const int32_t* prefix_pages,
                              int64_t prefix_stride, const int32_t* own_pages, int64_t own_stride,
                              const int32_t* own_lens, void* o, float* lse, const pg_opts* opts,
                              void* workspace, size_t workspace_bytes, pg_stream_t stream);

/*
 * Sample one token per row of logits [rows, vocab] (dtype `dtype`, rows ld elements apart) from a
 * given random number u[r] in [0, 1).  With T = temperature[r], m = max_i x_i and w_i = exp((x_i - m) / T):
 *   the tokens are ordered by logit, equal logits by index, and of them are kept
 *   - the first top_k[r] (all if top_k[r] <= 0),
 *   - of those, each whose predecessors hold less than the share top_p[r] of the weight of all those
 *     (all if top_p[r] >= 1),
 *   - each with w_i >= min_p[r] (all if min_p[r] <= 0);
 *   the first token of the order is always kept, and is the only one with a min_p[r] above 1 (equal
 *   logits included) or a NaN top_p[r] or min_p[r];
 *   token[r] = the first kept i, in index order, with sum_{kept j <= i} w_j > u[r] * sum_{kept j} w_j;
 *   logprob[r] = ln(w_token / sum_i w_i) over the whole vocabulary, at the row's temperature.
 * T = 0 is greedy: the first token of the order, its logprob at T = 1 (a negative or NaN T is
 * taken as 0); with T = +inf every logit above -inf has weight 1.  Each of temperature, top_k, top_p,
 * min_p may be NULL: 1, all, all, all.  logprobs may be NULL.  A NaN logit counts as -inf; if the
 * largest is +inf, all tokens with +inf have weight 1 and the others 0, at any T.  A row of -inf
 * throughout gives token -1 and logprob -inf.
 * A u[r] below 0 or NaN is taken as 0, one of 1 or above gives the last kept token.
 * The weights are fixed-point numbers with b = min(45, 62 - ceil(log2 vocab)) fraction bits: each is
 * within 2^-31 of its value and half a step of 2^-b of w_i (so those below about 2^-(b+1) count as
 * 0, and borders of top_p and min_p are settled in steps of 2^-b), and they are summed exactly: the
 * result does not depend on any order of summation.
 * rows >= 1, 1 <= vocab <= 2^20, ld >= vocab; device pointers aligned to their element type.
 * Errors: PG_ERR_INVALID_ARG (host check, nothing launched); PG_ERR_CUDA on a launch failure.
 */
pg_status pg_sample(pg_dtype dtype, int64_t rows, int32_t vocab, const void* logits, int64_t ld,
                    const float* u, const float* temperature, const int32_t* top_k,
                    const float* top_p, const float* min_p, int32_t* tokens, float* logprobs,
                    pg_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* PG_ROLLOUT_H */
