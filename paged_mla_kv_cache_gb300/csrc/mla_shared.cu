// Absorbed latent attention of requests behind shared prefixes
// (pmg_latent_decode_shared): the C entry.
//
// Mathematics: a row's weights over its prefix and over its own entries have
// sums (o1, m1, l1) and (o2, m2, l2), unnormalised under references m; with m =
// max(m1, m2) and w_i = 2^(m_i - m), out = (w1 o1 + w2 o2) / (w1 l1 + w2 l2).
//
// The prefix is a product of few entries with the rows of many requests, which
// is bound by the tensor core from a few hundred rows on; the own entries are a
// decode as before. Two passes: the first leaves (o1, m1, l1) of every row in the
// workspace, in 32 bits (2 KB a row, written and read once, mostly in L2), the
// second joins them as it finishes its rows.
#include <algorithm>

#include "mla_decode.cuh"
#include "pmg_long.h"

namespace pmg_mla {
namespace {

// What lies behind the attention workspace: sums of all rows, references and
// sums of weights, covered requests.
struct StateBytes {
  int64_t sums, ml, covered, end;
  StateBytes(int sms, int64_t rows, int32_t dv) {
    sums = (workspace_bytes(sms) + 255) / 256 * 256;
    ml = sums + (rows * dv * 4 + 255) / 256 * 256;
    covered = ml + (rows * 8 + 255) / 256 * 256;
    end = covered + 256;
  }
};

}  // namespace
}  // namespace pmg_mla

extern "C" int64_t pmg_shared_workspace(int64_t rows, int32_t latent_dim) {
  using namespace pmg_mla;
  int sms = 0;
  if (rows < 0 || rows > INT32_MAX || latent_dim < 1 || latent_dim > PMG_MAX_ENTRY || sm_count(&sms) != PMG_OK) return -1;
  return StateBytes(sms, rows, latent_dim).end;
}

extern "C" int pmg_latent_decode_shared(
    const void* q, int64_t q_req_stride, int64_t q_token_stride, int64_t q_head_stride, const void* cache,
    int64_t cache_block_stride, int64_t cache_token_stride, int64_t num_blocks, const int32_t* prefix_table,
    int64_t prefix_table_stride, const int32_t* prefix_lens, const int32_t* cu_groups, int32_t num_groups,
    const int32_t* block_table, int64_t block_table_stride, const int32_t* seq_lens, int32_t num_reqs, int32_t q_len,
    int32_t heads, int32_t latent_dim, int32_t rope_dim, int32_t block_size, int32_t q_dtype, int32_t cache_dtype,
    const float* scale, float sm_scale, void* out, int64_t out_req_stride, int64_t out_token_stride,
    int64_t out_head_stride, float* lse, void* workspace, int64_t workspace_bytes_given, int32_t* error_flag,
    void* stream, uint32_t options) {
  using namespace pmg_mla;
  DecodeParams p;
  int st = decode_params(p, q, q_req_stride, q_token_stride, q_head_stride, cache, cache_block_stride, cache_token_stride,
                         num_blocks, block_table, block_table_stride, seq_lens, num_reqs, q_len, heads, latent_dim,
                         rope_dim, block_size, q_dtype, cache_dtype, scale, sm_scale, out, out_req_stride,
                         out_token_stride, out_head_stride, lse, workspace, error_flag, options);
  if (st != PMG_OK) return st;
  if (num_groups < 0 || prefix_table_stride < 0) return PMG_ERR_ARG;
  if (num_groups > PMG_MAX_REQS || prefix_table_stride > INT32_MAX) return PMG_ERR_UNSUPPORTED;
  if (p.R == 0) return PMG_OK;
  const int64_t rows = static_cast<int64_t>(num_reqs) * q_len * heads;
  if (rows > INT32_MAX) return PMG_ERR_UNSUPPORTED;
  if (num_groups > 0 && (prefix_lens == nullptr || cu_groups == nullptr || (prefix_table == nullptr && prefix_table_stride > 0)))
    return PMG_ERR_NULL;
  if (!aligned(prefix_table, 4) || !aligned(prefix_lens, 4) || !aligned(cu_groups, 4)) return PMG_ERR_ALIGN;
  int sms = 0;
  st = sm_count(&sms);
  if (st != PMG_OK) return st;
  const StateBytes at(sms, rows, latent_dim);
  if (workspace_bytes_given < at.end) return PMG_ERR_ARG;
  p.ws = workspace_at(workspace, sms);
  if (num_groups > 0) {
    uint8_t* base = static_cast<uint8_t*>(workspace);
    p.state = reinterpret_cast<float*>(base + at.sums);
    p.state_ml = reinterpret_cast<float*>(base + at.ml);
    p.covered = reinterpret_cast<int32_t*>(base + at.covered);
    DecodeParams prefix = p;
    prefix.cu = cu_groups;
    prefix.reqs = num_reqs;
    prefix.R = num_groups;
    prefix.bt = prefix_table;
    prefix.bt_stride = prefix_table_stride;
    prefix.seq_lens = prefix_lens;
    st = run_prefix(prefix, q_dtype, cache_dtype, sms, stream, options);
    if (st != PMG_OK) return st;
  }
  return run_decode(p, q_dtype, cache_dtype, sms, stream, options);
}
