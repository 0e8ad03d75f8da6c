/*
 * pmg_long.h — C ABI of the operators for long contexts over the paged latent
 * cache (libpmg.so, next to the gather of pmg.h and the operators of
 * pmg_mla.h).
 *
 * Sparse attention: every new token attends to a few pages of its request.
 *   pmg_block_bounds    largest and smallest value of each column of a page,
 *                       kept up to date as entries join
 *   pmg_block_scores    an upper bound of a page's scores for each new token
 *   pmg_select_blocks   the pages with the best scores, as a block table that
 *                       pmg_latent_decode takes with one request a token
 * Shared prefixes: requests behind one prompt read it once for all.
 *   pmg_latent_decode_shared
 *
 * The conventions are those of pmg_mla.h: device arrays and host scalars,
 * strides in elements with a last dimension of stride 1, asynchronous calls on
 * `stream`, host-detected errors returned as a pmg_status with nothing
 * launched, data errors OR-ed into *error_flag. No call allocates memory or
 * synchronises. Every index read from the device is checked before it is used.
 */
#ifndef PMG_LONG_H_
#define PMG_LONG_H_

#include <stdint.h>

#include "pmg_mla.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * pmg_block_bounds — bounds of the entries that joined pages of the cache.
 *
 * For every page b that holds places [ctx_lens[r], seq_lens[r]) of a request r,
 * over those of its entries e_j:
 *   bounds[b, 0, d] = max_j e_j[d],   bounds[b, 1, d] = min_j e_j[d]
 * and, where the page holds places before ctx_lens[r] too, over the bounds that
 * it has as well. Exact: values as they are in the cache, an e4m3 one's
 * without its scale. A NaN makes NaN of its column. Other pages are not
 * touched. Entries that joined and were taken back (drafted tokens that were
 * refused) stay in the bounds of a begun page, which bound those that take their
 * places all the same, until a call has the page from its first place on.
 *
 *  cache      [num_blocks, block_size, entry_dim] of cache_dtype (bf16, fp16,
 *             fp32 or e4m3)
 *  bounds     [num_blocks, 2, entry_dim] of bounds_dtype: cache_dtype, or for an
 *             e4m3 cache bf16, fp16 or fp32 (as the queries that will meet it).
 *             It must not overlap the cache. Its rows must not overlap: pages lie
 *             behind each other (block stride >= row stride + entry_dim), or all
 *             largest values before all smallest ones (row stride >=
 *             (num_blocks - 1) * block stride + entry_dim).
 *  block_table int32 [num_reqs, block_table_stride]. A page outside [0,
 *             num_blocks) is skipped (PMG_FLAG_PHYS_BLOCK), places past the row
 *             too (PMG_FLAG_LOGICAL_BLOCK). The bounds of a page that two places
 *             in the table name, and both change, are undefined.
 *  ctx_lens   int32 [num_reqs]: places of which the bounds know, or NULL (none).
 *             Negative counts as 0 (PMG_FLAG_LENGTH).
 *  seq_lens   int32 [num_reqs]; negative counts as 0 (PMG_FLAG_LENGTH).
 * entry_dim <= PMG_MAX_ENTRY, num_reqs <= PMG_MAX_REQS.
 */
int pmg_block_bounds(const void* cache, int64_t cache_block_stride, int64_t cache_token_stride, int64_t num_blocks,
                     int32_t block_size, int32_t entry_dim, int32_t cache_dtype, void* bounds,
                     int64_t bounds_block_stride, int64_t bounds_row_stride, int32_t bounds_dtype,
                     const int32_t* block_table, int64_t block_table_stride, const int32_t* ctx_lens,
                     const int32_t* seq_lens, int32_t num_reqs, int32_t* error_flag, void* stream);

/*
 * pmg_block_scores — what a page's entries can score at most.
 *
 * For token i of the q_len new tokens of request r and column c of its block
 * table, with the bounds hi, lo of page block_table[r, c]:
 *   scores[r, i, c] = max_h (sm_scale * scale * s_h - lse[r, i, h]),
 *   s_h = sum_d max(q[r, i, h, d] hi[d], q[r, i, h, d] lo[d])
 * which no score of an entry of the page passes by more than the rounding of the
 * sum (2 entry_dim products in 32 bits: at most (2 entry_dim + 72) 2^-24 of
 * sm_scale * scale * sum_d max(|q hi|, |q lo|) + |lse|); with the log sums of an
 * earlier step, no logarithm of a weight. -INFINITY for a page of which token i
 * sees no entry (it sees the first seq_lens[r] - q_len + 1 + i entries, as in
 * pmg_latent_decode) and for a page outside the cache. NaN where a term is NaN
 * (0 times an infinite bound is). Every column of the table is written.
 *
 *  q          [num_reqs, q_len, heads, entry_dim] of dtype (bf16, fp16, fp32)
 *  bounds     [num_blocks, 2, entry_dim] of dtype
 *  block_table int32 [num_reqs, block_table_stride] (flags as in
 *             pmg_latent_decode)
 *  seq_lens   int32 [num_reqs]; negative counts as 0 (PMG_FLAG_LENGTH)
 *  scale      fp32 device scalar >= 0 or NULL (1.0): the e4m3 cache's
 *  lse        fp32 [num_reqs, q_len, heads], contiguous, or NULL (0). A value
 *             that is not finite counts as 0.
 *  scores     fp32 [num_reqs, q_len, block_table_stride]: rows score_stride
 *             apart
 *
 * The tensor-core kernel runs for entry_dim 576, bf16 or fp16 with 16-byte
 * aligned rows of q and bounds; the general kernel, also taken with
 * PMG_OPT_FORCE_GENERAL, for everything else. Products are exact and summed in
 * 32 bits in both.
 */
int pmg_block_scores(const void* q, int64_t q_req_stride, int64_t q_token_stride, int64_t q_head_stride,
                     const void* bounds, int64_t bounds_block_stride, int64_t bounds_row_stride, int64_t num_blocks,
                     const int32_t* block_table, int64_t block_table_stride, const int32_t* seq_lens, int32_t num_reqs,
                     int32_t q_len, int32_t heads, int32_t entry_dim, int32_t block_size, int32_t dtype,
                     const float* scale, float sm_scale, const float* lse, float* scores, int64_t score_stride,
                     int32_t* error_flag, void* stream, uint32_t options);

/*
 * pmg_select_blocks — the pages that each new token attends to.
 *
 * Token i of request r sees n = seq_lens[r] - q_len + 1 + i entries (0 where
 * that is negative) on ceil(n / block_size) pages. Of more than `keep` it keeps
 * its first `first`, its last `last` and those with the largest scores between
 * (equal ones: the lower column; NaN above all), in the order of their columns:
 *   selected[r * q_len + i, :]  = their ids in block_table[r], -1 behind the last
 *   selected_lens[r * q_len + i] = entries on them that the token sees
 * The last page is always kept, so these are the first selected_lens entries of
 * the row's pages: pmg_latent_decode takes them as the block table and lengths
 * of num_reqs * q_len requests of one token.
 *
 *  scores     fp32 [num_reqs, q_len, block_table_stride]: rows score_stride apart
 *  block_table int32 [num_reqs, block_table_stride]. Ids are passed on as they
 *             are. Entries past the row count as not there
 *             (PMG_FLAG_LOGICAL_BLOCK).
 *  seq_lens   int32 [num_reqs]; negative counts as 0 (PMG_FLAG_LENGTH)
 *  selected   int32 [num_reqs * q_len, keep]: rows selected_stride apart
 *  columns    the columns of the kept pages, like selected, or NULL
 * 0 <= first, 1 <= last, first + last <= keep <= INT32_MAX. Results must not
 * overlap the inputs.
 */
int pmg_select_blocks(const float* scores, int64_t score_stride, const int32_t* block_table, int64_t block_table_stride,
                      const int32_t* seq_lens, int32_t num_reqs, int32_t q_len, int32_t block_size, int32_t* selected,
                      int64_t selected_stride, int32_t* columns, int32_t* selected_lens, int64_t keep, int32_t first,
                      int32_t last, int32_t* error_flag, void* stream);

/*
 * pmg_latent_decode_shared — absorbed latent attention of requests that share
 * prefixes.
 *
 * Requests [cu_groups[g], cu_groups[g + 1]) see all prefix_lens[g] entries of
 * prefix g, whose pages are row g of prefix_table, and then entries of their
 * own as in pmg_latent_decode: row (r, i, h) the first seq_lens[r] - q_len + 1 +
 * i. Requests of no group have no prefix. Scores, result and log sum are those
 * of pmg_latent_decode over both together; a row that sees nothing gives out =
 * 0, lse = -inf. A prefix is read once for a tile of rows of all its requests.
 *
 *  prefix_table int32 [num_groups, prefix_table_stride], prefix_lens int32
 *             [num_groups]: as block_table and seq_lens, flags too
 *  cu_groups  int32 [num_groups + 1], cut to [0, num_reqs]. A decrease gives that
 *             group no requests (PMG_FLAG_CU_ORDER, for a negative value too);
 *             requests before cu_groups[0] have no prefix, and the rows of one
 *             that such an order puts in two groups are undefined.
 *  workspace  pmg_shared_workspace() bytes, 256-byte aligned; its content does
 *             not matter. Calls that may overlap need one each.
 * The rest as in pmg_latent_decode, its kernels' limits, choice and rounding
 * too. num_groups <= PMG_MAX_REQS, num_reqs * q_len * heads <= INT32_MAX.
 */
int pmg_latent_decode_shared(const void* q, int64_t q_req_stride, int64_t q_token_stride, int64_t q_head_stride,
                             const void* cache, int64_t cache_block_stride, int64_t cache_token_stride,
                             int64_t num_blocks, const int32_t* prefix_table, int64_t prefix_table_stride,
                             const int32_t* prefix_lens, const int32_t* cu_groups, int32_t num_groups,
                             const int32_t* block_table, int64_t block_table_stride, const int32_t* seq_lens,
                             int32_t num_reqs, int32_t q_len, int32_t heads, int32_t latent_dim, int32_t rope_dim,
                             int32_t block_size, int32_t q_dtype, int32_t cache_dtype, const float* scale,
                             float sm_scale, void* out, int64_t out_req_stride, int64_t out_token_stride,
                             int64_t out_head_stride, float* lse, void* workspace, int64_t workspace_bytes,
                             int32_t* error_flag, void* stream, uint32_t options);

/* Bytes of the workspace of pmg_latent_decode_shared for so many rows (num_reqs
 * * q_len * heads) of latent_dim values on the current device, or a negative
 * number where there is no device or a size is out of range. It suffices for
 * the attention calls of pmg_mla.h too. */
int64_t pmg_shared_workspace(int64_t rows, int32_t latent_dim);

/* These calls through pmg_call_packed, next to those of enum pmg_packed. */
#define PMG_CALL_BLOCK_BOUNDS 4
#define PMG_CALL_BLOCK_SCORES 5
#define PMG_CALL_SELECT_BLOCKS 6
#define PMG_CALL_LATENT_DECODE_SHARED 7

#ifdef __cplusplus
}
#endif

#endif /* PMG_LONG_H_ */
