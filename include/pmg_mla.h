/*
 * pmg_mla.h — C ABI of the latent-attention operators around the paged cache
 * (libpmg.so, next to the gather of pmg.h).
 *
 * One serving step over a paged latent (MLA) cache:
 *   pmg_plan_step       lengths -> block table, slots, positions, prefix sums
 *   pmg_append          norm, rotation and the write of new entries
 *   pmg_latent_decode   absorbed attention of one or a few new tokens a
 *                       request, straight over the paged cache
 *   pmg_latent_prefill  expanded attention of a chunk of new tokens over keys
 *                       and values expanded from gathered entries, joined with
 *                       the state of keys seen before
 *
 * The conventions are those of pmg.h: device arrays and host scalars, strides
 * in elements with a last dimension of stride 1, asynchronous calls on
 * `stream`, host-detected errors returned as a pmg_status with nothing
 * launched, data errors OR-ed into *error_flag with the affected rows skipped.
 * No call allocates memory or synchronises. Every index read from the device
 * is checked before it is used. Waits on the device are bounded: where one of
 * the attention calls' runs out (two seconds; PMG_FLAG_TIMEOUT), the rows that
 * it was for become NaN, result and log sum, whether or not a flag was given.
 */
#ifndef PMG_MLA_H_
#define PMG_MLA_H_

#include <stdint.h>

#include "pmg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits OR-ed into *error_flag by these calls, next to those of pmg.h. */
#define PMG_FLAG_LENGTH 64      /* a length is negative, or a context passes INT32_MAX: taken as 0, or cut */
#define PMG_FLAG_CAPACITY 128   /* more new tokens than max_tokens: the rest is dropped */
#define PMG_FLAG_NO_BLOCKS 256  /* free_blocks ran out: table entry and slots are -1 */
#define PMG_FLAG_POSITION 512   /* a position outside the rotation table: token skipped */

/*
 * pmg_plan_step — block table, slots and positions of one step.
 *
 * Request r has ctx_lens[r] tokens in the cache and new_lens[r] joining it in
 * this step. Its pages [0, ceil(ctx/B)) are in its block-table row already;
 * pages up to ceil((ctx + new)/B) are taken from free_blocks, in the order of
 * the requests and of their pages.
 *
 *  ctx_lens, new_lens  int32 [num_reqs]. A negative length counts as 0
 *                      (PMG_FLAG_LENGTH).
 *  block_table         int32 [num_reqs, block_table_stride]: only the columns
 *                      of fresh pages are written. A page past the row is not
 *                      written (PMG_FLAG_LOGICAL_BLOCK) and its tokens get
 *                      slot -1.
 *  free_blocks         int32 [num_free]: ids in [0, num_blocks). An id outside
 *                      is not used (PMG_FLAG_PHYS_BLOCK: -1 in its place).
 *  slots               int64 [max_tokens]: block id * block_size + offset of
 *                      every new token, requests back to back; -1 for a token
 *                      without a page and for the rows past the last token.
 *  positions           int32 [max_tokens]: position in the request (-1 past
 *                      the last token).
 *  token_to_seq        int32 [max_tokens]: request (-1 past the last token).
 *  cu_new, cu_seq      int32 [num_reqs + 1]: exclusive prefix sums of the new
 *                      and of the total lengths (cut at INT32_MAX,
 *                      PMG_FLAG_CAPACITY).
 *  seq_lens            int32 [num_reqs]: ctx + new.
 *  blocks_taken        int32 [1]: ids taken from free_blocks.
 * num_reqs <= PMG_MAX_REQS, max_tokens <= INT32_MAX. slots, positions,
 * token_to_seq, cu_seq and blocks_taken may be NULL (not wanted). Results must
 * not overlap ctx_lens, new_lens or free_blocks, which are read throughout the
 * call (PMG_ERR_ARG): lengths are not updated in place. Ids are taken from the
 * list's beginning each time: before the next call, a replayed graph's too, the
 * caller moves the list on by *blocks_taken.
 */
int pmg_plan_step(const int32_t* ctx_lens, const int32_t* new_lens, int32_t num_reqs, int32_t* block_table,
                  int64_t block_table_stride, const int32_t* free_blocks, int64_t num_free, int64_t num_blocks,
                  int32_t block_size, int64_t* slots, int32_t* positions, int32_t* token_to_seq, int64_t max_tokens,
                  int32_t* cu_new, int32_t* seq_lens, int32_t* cu_seq, int32_t* blocks_taken, int32_t* error_flag,
                  void* stream);

/* Options of pmg_append. */
#define PMG_OPT_ROPE_PAIRS 1u  /* rotate elements (2i, 2i + 1); default: (i, i + rope_dim / 2) */

/*
 * pmg_append — write the entries of new tokens into the paged cache.
 *
 * For every token t with slots[t] >= 0:
 *   latent = c_kv[t] * rsqrt(mean(c_kv[t]^2) + eps) * norm_weight   (or c_kv[t] where norm_weight is NULL)
 *   pe     = rotate(k_pe[t], cos_sin[positions[t]])
 *   cache[slot / block_size, slot % block_size] = (latent, pe)      (divided by *scale for an fp8 cache, at most +-448)
 * and for every token with positions[t] >= 0, with q_pe given:
 *   q_out[t, h] = rotate(q_pe[t, h], cos_sin[positions[t]])
 * in 32 bits, rounded once to the type of the output. rotate takes pairs
 * (a, b) to (a cos - b sin, b cos + a sin).
 *
 *  c_kv       [num_tokens, latent_dim], k_pe [num_tokens, rope_dim], q_pe
 *             [num_tokens, heads, rope_dim]: src_dtype (bf16, fp16 or fp32)
 *  norm_weight fp32 [latent_dim] or NULL
 *  cos_sin    fp32 [num_positions, rope_dim]: rope_dim / 2 cosines, then sines
 *  slots      int64, positions int32 [num_tokens]. A negative slot writes no
 *             entry, a slot past the cache neither (PMG_FLAG_PHYS_BLOCK). A
 *             position past num_positions, or a negative one beside a slot,
 *             skips the token (PMG_FLAG_POSITION). Two tokens with one slot
 *             race.
 *  cache      [num_blocks, block_size, latent_dim + rope_dim] of cache_dtype
 *             (bf16, fp16, fp32 or e4m3)
 *  scale      fp32 device scalar or NULL (1.0); used for an fp8 cache.
 *  q_pe, q_out NULL with heads 0. q_out has src_dtype; it may be q_pe itself.
 */
int pmg_append(const void* c_kv, int64_t c_kv_stride, const void* k_pe, int64_t k_pe_stride, const float* norm_weight,
               float eps, const float* cos_sin, int64_t num_positions, const int64_t* slots, const int32_t* positions,
               int64_t num_tokens, int32_t latent_dim, int32_t rope_dim, int32_t src_dtype, void* cache,
               int64_t cache_block_stride, int64_t cache_token_stride, int64_t num_blocks, int32_t block_size,
               int32_t cache_dtype, const float* scale, const void* q_pe, int64_t q_pe_token_stride,
               int64_t q_pe_head_stride, void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
               int32_t heads, int32_t* error_flag, void* stream, uint32_t options);

/* Options of the attention calls. */
#define PMG_OPT_CAUSAL 1u        /* pmg_latent_prefill: query i of q sees the first k - q + i + 1 of k keys */
#define PMG_OPT_FORCE_GENERAL 2u /* the kernel for any sizes, even where the tensor-core kernel applies */

/* Largest latent_dim + rope_dim of the attention calls. */
#define PMG_MAX_ENTRY 1024

/*
 * pmg_latent_decode — absorbed latent attention over the paged cache.
 *
 * Query row (r, i, h) sees the first seq_lens[r] - q_len + 1 + i entries e_j
 * of request r (causal among the q_len new tokens, which are in the cache):
 *   s_j = sm_scale * sum_d q[r, i, h, d] e_j[d]          over all of an entry
 *   out = sum_j softmax(s)_j e_j[0 : latent_dim],   lse = log sum_j exp(s_j)
 * A row that sees nothing gives out = 0, lse = -inf.
 *
 *  q          [num_reqs, q_len, heads, latent_dim + rope_dim] of q_dtype
 *             (bf16, fp16 or fp32)
 *  cache      [num_blocks, block_size, latent_dim + rope_dim] of cache_dtype:
 *             q_dtype, or e4m3 with `scale` (fp32 device scalar, NULL: 1.0)
 *  block_table int32 [num_reqs, block_table_stride]. Entries on a page outside
 *             [0, num_blocks) or past the row are left out of the sums
 *             (PMG_FLAG_PHYS_BLOCK, PMG_FLAG_LOGICAL_BLOCK).
 *  seq_lens   int32 [num_reqs]; negative counts as 0 (PMG_FLAG_LENGTH).
 *  out        [num_reqs, q_len, heads, latent_dim] of q_dtype
 *  lse        fp32 [num_reqs, q_len, heads], contiguous, or NULL
 *  workspace  pmg_attention_workspace() bytes, 16-byte aligned; its content
 *             does not matter. Calls that may overlap need one each.
 * Slots of the cache at or past seq_lens[r] may hold anything, NaN too, and a
 * row is not touched by infinities or NaN in entries that it does not see.
 *
 * The tensor-core kernel runs for latent_dim 512, rope_dim 64, q_dtype bf16 or
 * fp16, a block_size that is a multiple of 8, 16-byte aligned rows of cache and
 * q, strides below 2^38 elements; the general kernel, many times slower on long
 * requests, for everything else. Scores, sums and accumulators are 32-bit in
 * both. For the second product the tensor-core kernel rounds weights to the
 * type of a 16-bit cache (2^-8 of each, fp16 2^-11); over an e4m3 cache to 2^-9
 * of each, or to 2^-28 of the row's largest where that is more. Over an e4m3
 * cache it takes query values to within 2^-17 of the row's largest.
 */
int pmg_latent_decode(const void* q, int64_t q_req_stride, int64_t q_token_stride, int64_t q_head_stride,
                      const void* cache, int64_t cache_block_stride, int64_t cache_token_stride, int64_t num_blocks,
                      const int32_t* block_table, int64_t block_table_stride, const int32_t* seq_lens,
                      int32_t num_reqs, int32_t q_len, int32_t heads, int32_t latent_dim, int32_t rope_dim,
                      int32_t block_size, int32_t q_dtype, int32_t cache_dtype, const float* scale, float sm_scale,
                      void* out, int64_t out_req_stride, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                      void* workspace, int64_t workspace_bytes, int32_t* error_flag, void* stream, uint32_t options);

/*
 * pmg_latent_prefill — expanded latent attention of a chunk of new tokens.
 *
 * Request r owns query rows [cu_q[r], cu_q[r+1]) and key rows [cu_k[r],
 * cu_k[r+1]). For query row i of head h and the keys j that it sees (all, or
 * with PMG_OPT_CAUSAL those with j - i <= k_len - q_len, counted inside the
 * request):
 *   s_j = sm_scale * (q[i, h, :nope] . k_nope[j, h] + q[i, h, nope:] . k_pe[j])
 *   out = sum_j softmax(s)_j v[j, h],   lse = log sum_j exp(s_j)
 * The rotated key part is one row a token, shared by the heads. With prev_out
 * and prev_lse (the result over other keys) the two are joined:
 *   lse' = log(exp(lse) + exp(prev_lse)),
 *   out' = exp(lse - lse') out + exp(prev_lse - lse') prev_out.
 * A row that sees nothing gives out = 0, lse = -inf (or the previous state).
 * A row is not touched by infinities or NaN in keys and values that it does not
 * see, nor by a previous result whose prev_lse is -inf.
 *
 *  q       [total_q, heads, nope_dim + rope_dim], k_nope [total_k, heads,
 *          nope_dim], k_pe [total_k, rope_dim], v [total_k, heads, v_dim], out
 *          and prev_out [total_q, heads, v_dim]: dtype (bf16, fp16 or fp32)
 *  lse     fp32 [total_q, heads] contiguous or NULL; prev_lse likewise.
 *          prev_out may be out and prev_lse may be lse.
 *  cu_q, cu_k int32 [num_reqs + 1], row ranges cut to [0, total). A negative
 *          value or a decrease gives that request no rows
 *          (PMG_FLAG_CU_ORDER). Requests whose query rows overlap race.
 *  workspace as in pmg_latent_decode.
 *
 * The tensor-core kernel runs for nope_dim 128, rope_dim 64, v_dim 128, bf16
 * or fp16 with 16-byte aligned rows, no stride of 0 and sm_scale > 0; the
 * general kernel for everything else (nope_dim + rope_dim and v_dim up to
 * PMG_MAX_ENTRY). Scores, sums and accumulators are 32-bit in both; the
 * tensor-core kernel rounds weights to the type of v for the second product.
 */
int pmg_latent_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_nope,
                       int64_t k_token_stride, int64_t k_head_stride, const void* k_pe, int64_t k_pe_stride,
                       const void* v, int64_t v_token_stride, int64_t v_head_stride, const int32_t* cu_q,
                       const int32_t* cu_k, int32_t num_reqs, int64_t total_q, int64_t total_k, int32_t heads,
                       int32_t nope_dim, int32_t rope_dim, int32_t v_dim, int32_t dtype, float sm_scale, void* out,
                       int64_t out_token_stride, int64_t out_head_stride, float* lse, const void* prev_out,
                       int64_t prev_token_stride, int64_t prev_head_stride, const float* prev_lse, void* workspace,
                       int64_t workspace_bytes, int32_t* error_flag, void* stream, uint32_t options);

/* Bytes of the workspace of the attention calls on the current device (any
 * sizes), or a negative number where there is no device. */
int64_t pmg_attention_workspace(void);

/*
 * pmg_call_packed — one of the calls above with its arguments in an array of
 * 8-byte words, in the order of its parameter list: pointers and whole numbers
 * as int64_t, floats as double, the stream among them. For callers whose
 * foreign-function layer takes longer to pass thirty arguments than the call
 * itself takes. An unknown call returns PMG_ERR_ARG, NULL words PMG_ERR_NULL.
 */
typedef enum pmg_packed {
  PMG_CALL_PLAN_STEP = 0,
  PMG_CALL_APPEND = 1,
  PMG_CALL_LATENT_DECODE = 2,
  PMG_CALL_LATENT_PREFILL = 3
} pmg_packed;
int pmg_call_packed(int call, const void* words);

#ifdef __cplusplus
}
#endif

#endif /* PMG_MLA_H_ */
