// Upper bounds of the scores of the cache's pages (pmg_block_scores): the kernel
// for any sizes and the C entry.
//
// Mathematics: over the entries e of a page, lo <= e <= hi column by column, so
// q . e = sum_d q_d e_d <= sum_d max(q_d hi_d, q_d lo_d) = sum_d (max(q_d, 0) hi_d
// + min(q_d, 0) lo_d) for finite bounds, and the largest of these over the heads
// bounds every score that the page can have. An infinite bound's product with 0
// would be NaN: where a sum is, it is taken again as the first form.
#include <algorithm>

#include "mla_scores.cuh"

namespace pmg_mla {
namespace {

// Any sizes and types. A warp takes a page of a request, keeps its bounds in
// registers (a lane every 32nd column) and meets every row of queries with
// them; the sum over the lanes costs more than the products. It exists for what
// the tensor-core kernel does not take: 938 pages and 16 heads in fp32 take 95 us
// (in 16 bits 107, on the tensor core 6.8), 64 requests of 64 pages and 128 heads
// 1.3 ms (11 us).
constexpr int kGeneralThreads = 256;
constexpr int kLaneColumns = PMG_MAX_ENTRY / 32;

template <class T>
__global__ void __launch_bounds__(kGeneralThreads) scores_general_kernel(const __grid_constant__ ScoreParams p) {
  __shared__ int64_t scratch[33], found[2];
  pdl_entry();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Share share = find_share([&](int r) { return score_pieces(p, r); }, p.R, blockIdx.x, p.units, scratch, found);
  const float factor = p.sm_scale * (p.scale != nullptr ? *p.scale : 1.0f);
  int bad = 0;
  int64_t at = share.begin, skip = share.offset;
  for (int r = share.item; at < share.end; ++r, skip = 0) {
    const SparseLen len = sparse_len(p.seq, r, p.bt_stride, p.B);
    const int64_t pages = score_pages(p, len), pieces = score_pieces(p, r);
    const int64_t n = min(pieces - skip, share.end - at);
    at += n;
    bad |= len.bad;
    const int32_t* table = p.bt + static_cast<int64_t>(r) * p.bt_stride;
    for (int64_t c = skip * kScoreTile + warp; c < min(pages, (skip + n) * kScoreTile); c += kGeneralThreads / 32) {
      const int32_t id = table[c];
      const bool good = id >= 0 && id < p.num_blocks;
      if (!good) bad |= PMG_FLAG_PHYS_BLOCK;
      float hi[kLaneColumns], lo[kLaneColumns];
      const T* row = reinterpret_cast<const T*>(p.bounds) + (good ? id : 0) * p.bb_stride;
#pragma unroll
      for (int k = 0; k < kLaneColumns; ++k) {
        const bool in = good && lane + 32 * k < p.E;
        hi[k] = in ? to_f(row[lane + 32 * k]) : 0.0f;
        lo[k] = in ? to_f(row[p.br_stride + lane + 32 * k]) : 0.0f;
      }
      for (int i = 0; i < p.q_len; ++i) {
        float best = -INFINITY;
        if (good && c * p.B < sparse_seen(len, i, p.q_len)) {
          for (int h = 0; h < p.H; ++h) {
            const T* q = reinterpret_cast<const T*>(p.q) + r * p.qr_stride + i * p.qt_stride + h * p.qh_stride;
            float x = 0.0f;
#pragma unroll
            for (int k = 0; k < kLaneColumns; ++k)
              if (lane + 32 * k < p.E) {
                const float y = to_f(q[lane + 32 * k]);
                const bool below = signbit(y);
                x += (below ? 0.0f : y) * hi[k];
                x += (below ? y : 0.0f) * lo[k];
              }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (isnan(x)) x = score_sum_odd<T, 1>(q, row, row + p.br_stride, p.E);
            const int64_t rr = (static_cast<int64_t>(r) * p.q_len + i) * p.H + h;
            best = max_nan(best, x * factor - score_shift(p, rr));
          }
        }
        if (lane == 0) p.scores[(static_cast<int64_t>(r) * p.q_len + i) * p.s_stride + c] = best;
      }
    }
    if (skip + n == pieces) score_rest(p, r, pages, tid, kGeneralThreads);
  }
  set_flag(p.err, bad);
}

}  // namespace
}  // namespace pmg_mla

extern "C" int pmg_block_scores(const void* q, int64_t q_req_stride, int64_t q_token_stride, int64_t q_head_stride,
                                const void* bounds, int64_t bounds_block_stride, int64_t bounds_row_stride,
                                int64_t num_blocks, const int32_t* block_table, int64_t block_table_stride,
                                const int32_t* seq_lens, int32_t num_reqs, int32_t q_len, int32_t heads,
                                int32_t entry_dim, int32_t block_size, int32_t dtype, const float* scale,
                                float sm_scale, const float* lse, float* scores, int64_t score_stride,
                                int32_t* error_flag, void* stream, uint32_t options) {
  using namespace pmg_mla;
  const int es = elem_bytes(dtype);
  if (es < 2) return PMG_ERR_DTYPE;
  if (num_reqs < 0 || q_len < 0 || heads < 0 || entry_dim < 1 || block_size < 1 || num_blocks < 0 ||
      block_table_stride < 0 || !(sm_scale >= 0.0f) || (options & ~PMG_OPT_FORCE_GENERAL))
    return PMG_ERR_ARG;
  for (const int64_t s : {q_req_stride, q_token_stride, q_head_stride, bounds_block_stride, bounds_row_stride, score_stride})
    if (!stride_ok(s)) return PMG_ERR_ARG;
  if (score_stride < block_table_stride) return PMG_ERR_ARG;  // rows of scores do not overlap
  if (entry_dim > PMG_MAX_ENTRY || num_blocks > INT32_MAX || block_table_stride > INT32_MAX || num_reqs > PMG_MAX_REQS ||
      static_cast<int64_t>(q_len) * heads > (1 << 20) || static_cast<int64_t>(num_reqs) * q_len > INT32_MAX)
    return PMG_ERR_UNSUPPORTED;
  if (num_reqs == 0 || q_len == 0 || block_table_stride == 0) return PMG_OK;
  if ((q == nullptr && heads > 0) || scores == nullptr || seq_lens == nullptr || block_table == nullptr ||
      (bounds == nullptr && num_blocks > 0))
    return PMG_ERR_NULL;
  if (!aligned(q, es) || !aligned(bounds, es) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(scale, 4) || !aligned(lse, 4) || !aligned(scores, 4) || !aligned(error_flag, 4))
    return PMG_ERR_ALIGN;
  int sms = 0;
  const int st = sm_count(&sms);
  if (st != PMG_OK) return st;
  ScoreParams p{};
  p.q = static_cast<const uint8_t*>(q);
  p.qr_stride = q_req_stride;
  p.qt_stride = q_token_stride;
  p.qh_stride = q_head_stride;
  p.bounds = static_cast<const uint8_t*>(bounds);
  p.bb_stride = bounds_block_stride;
  p.br_stride = bounds_row_stride;
  p.num_blocks = num_blocks;
  p.bt = block_table;
  p.bt_stride = block_table_stride;
  p.seq = seq_lens;
  p.R = num_reqs;
  p.q_len = q_len;
  p.H = heads;
  p.E = entry_dim;
  p.B = block_size;
  p.scale = scale;
  p.sm_scale = sm_scale;
  p.lse = lse;
  p.scores = scores;
  p.s_stride = score_stride;
  p.err = error_flag;
  if (!(options & PMG_OPT_FORCE_GENERAL) && scores_tc_takes(p, dtype)) {
    p.units = sms;
    return scores_tc(p, dtype, stream);
  }
  p.units = 2 * sms;
  const auto k = dtype == PMG_BF16 ? scores_general_kernel<bf16> : dtype == PMG_FP16 ? scores_general_kernel<f16>
                                                                                     : scores_general_kernel<float>;
  return launch(k, dim3(static_cast<unsigned>(p.units)), kGeneralThreads, 0, stream, p);
}
