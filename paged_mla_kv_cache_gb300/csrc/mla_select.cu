// The pages that each new token attends to (pmg_select_blocks).
//
// Mathematics: the k-th largest of a row's competing scores is found digit by
// digit: scores are mapped to whole numbers of the same order (all bits of a
// negative one flipped, the sign bit of the others; NaN above all, -0 as 0),
// eight bits are counted in shared memory, and the digit that holds the k-th is
// kept. Pages above that value stay, and of those equal to it the first ones. A
// thread owns a run of neighbouring columns, so that one prefix sum over the
// threads gives every kept page its place, in order.
//
// Bound by latency: a row is a few thousand scores, read once. A CTA takes a
// row and holds it in shared memory (what does not fit there is read again in
// each pass, from L2); one warp finds the digit, and the search ends as soon as
// all of a digit's scores stay, after two passes as a rule. Measured: 2 rows of 938
// pages 4.3 us, 256 of them 8.2, one of 8000 10.1 (a launch that copies a short row
// 1.3).
#include <algorithm>

#include "mla_long.cuh"
#include "pmg_long.h"

namespace pmg_mla {
namespace {

constexpr int kHeld = 8192;  // scores in shared memory

struct SelectParams {
  const float* scores;
  int64_t s_stride;
  const int32_t* bt;
  int64_t bt_stride;
  const int32_t* seq;
  int32_t q_len, B;
  int32_t* selected;
  int64_t sel_stride;
  int32_t* columns;
  int32_t* lens;
  int64_t keep;
  int32_t first, last;
  int32_t* err;
};

// Whole numbers in the order of the scores.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (isnan(x)) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ uint32_t held[kHeld];
  __shared__ uint32_t counts[256];
  __shared__ int64_t scratch[33];
  __shared__ uint32_t found[3];  // digit; how many are wanted of its scores, and how many there are
  pdl_entry();
  const int tid = threadIdx.x;
  const int64_t token = blockIdx.x;
  const int r = static_cast<int>(token / p.q_len), i = static_cast<int>(token - static_cast<int64_t>(r) * p.q_len);
  const SparseLen len = sparse_len(p.seq, r, p.bt_stride, p.B);
  const int64_t seen = sparse_seen(len, i, p.q_len);
  const uint32_t B = static_cast<uint32_t>(p.B);
  const uint32_t pages = (static_cast<uint32_t>(seen) + B - 1) / B;
  const int32_t* table = p.bt + static_cast<int64_t>(r) * p.bt_stride;
  int32_t* selected = p.selected + token * p.sel_stride;
  int32_t* columns = p.columns != nullptr ? p.columns + token * p.sel_stride : nullptr;
  if (tid == 0 && i == 0) set_flag(p.err, len.bad);
  if (pages <= p.keep) {
    for (int64_t c = tid; c < p.keep; c += kThreads) {
      selected[c] = c < pages ? table[c] : -1;
      if (columns != nullptr) columns[c] = c < pages ? static_cast<int32_t>(c) : -1;
    }
    if (tid == 0) p.lens[token] = static_cast<int32_t>(seen);
    return;
  }
  // pages [lo, hi) compete for `need` places
  const uint32_t lo = static_cast<uint32_t>(p.first), hi = pages - static_cast<uint32_t>(p.last);
  const uint32_t need = static_cast<uint32_t>(p.keep) - p.first - p.last;
  const float* scores = p.scores + token * p.s_stride;
  const uint32_t kept = min(hi, static_cast<uint32_t>(kHeld));
#pragma unroll 4
  for (uint32_t c = lo + tid; c < kept; c += kThreads) held[c] = score_key(scores[c]);
  auto key = [&](uint32_t c) { return c < kHeld ? held[c] : score_key(scores[c]); };
  uint32_t prefix = 0, rest = need;  // digits so far of the need-th largest; how many of its like are wanted
  if (need > 0) {
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) counts[tid] = 0;
      __syncthreads();
      const uint32_t above = shift == 24 ? 0 : 0xffffffffu << (shift + 8);
      for (uint32_t c = lo + tid; c < hi; c += kThreads) {
        const uint32_t k = key(c);  // (its own: each thread has put it there)
        if ((k & above) == prefix) atomicAdd(&counts[k >> shift & 255], 1u);
      }
      __syncthreads();
      if (tid < 32) {  // the largest digit at or above which there are `rest`: a lane has eight, from the top
        uint32_t n[8], sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += n[k] = counts[255 - 8 * tid - k];
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (tid >= o) inc += y;
        }
        uint32_t before = inc - sum;
        if (before < rest && rest <= inc) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (before < rest && rest <= before + n[k]) {
              found[0] = 255 - 8 * tid - k;
              found[1] = rest - before;
              found[2] = n[k];
            }
            before += n[k];
          }
        }
      }
      __syncthreads();
      prefix |= found[0] << shift;
      rest = found[1];
      if (rest == found[2]) break;  // all that begin like this stay: those above the prefix, and those that are it
    }
  }
  __syncthreads();
  // a run of columns a thread: those that stay for sure, and those equal to the border of which `rest` stay
  const uint32_t run = (pages + kThreads - 1) / kThreads, c0 = min(pages, tid * run), c1 = min(pages, c0 + run);
  uint32_t sure = 0, equal = 0;
  auto competes = [&](uint32_t c) { return c >= lo && c < hi; };
  for (uint32_t c = c0; c < c1; ++c) {
    if (!competes(c)) ++sure;
    else if (need > 0) {
      const uint32_t k = key(c);
      sure += k > prefix;
      equal += k == prefix;
    }
  }
  int64_t total;
  const int64_t before = block_scan<int64_t>(static_cast<int64_t>(equal) << 32 | sure, scratch, total);
  uint32_t equals = static_cast<uint32_t>(before >> 32);
  int64_t at = static_cast<int64_t>(before & 0xffffffff) + min(equals, rest);
  for (uint32_t c = c0; c < c1; ++c) {
    bool stays = !competes(c);
    if (!stays && need > 0) {
      const uint32_t k = key(c);
      stays = k > prefix || (k == prefix && equals++ < rest);
    }
    if (stays) {
      selected[at] = table[c];
      if (columns != nullptr) columns[at] = static_cast<int32_t>(c);
      ++at;
    }
  }
  if (tid == 0) p.lens[token] = static_cast<int32_t>(seen - static_cast<int64_t>(pages - static_cast<uint32_t>(p.keep)) * B);
}

}  // namespace
}  // namespace pmg_mla

extern "C" int pmg_select_blocks(const float* scores, int64_t score_stride, const int32_t* block_table,
                                 int64_t block_table_stride, const int32_t* seq_lens, int32_t num_reqs, int32_t q_len,
                                 int32_t block_size, int32_t* selected, int64_t selected_stride, int32_t* columns,
                                 int32_t* selected_lens, int64_t keep, int32_t first, int32_t last, int32_t* error_flag,
                                 void* stream) {
  using namespace pmg_mla;
  if (num_reqs < 0 || q_len < 0 || block_size < 1 || block_table_stride < 0 || first < 0 || last < 1 ||
      static_cast<int64_t>(first) + last > keep || selected_stride < keep || score_stride < block_table_stride ||
      !stride_ok(score_stride) || !stride_ok(selected_stride))
    return PMG_ERR_ARG;
  if (block_table_stride > INT32_MAX || num_reqs > PMG_MAX_REQS || static_cast<int64_t>(num_reqs) * q_len > INT32_MAX ||
      keep > INT32_MAX)
    return PMG_ERR_UNSUPPORTED;
  if (num_reqs == 0 || q_len == 0) return PMG_OK;
  if (seq_lens == nullptr || selected == nullptr || selected_lens == nullptr ||
      ((scores == nullptr || block_table == nullptr) && block_table_stride > 0))
    return PMG_ERR_NULL;
  if (!aligned(scores, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(selected, 4) ||
      !aligned(columns, 4) || !aligned(selected_lens, 4) || !aligned(error_flag, 4))
    return PMG_ERR_ALIGN;
  SelectParams p{};
  p.scores = scores;
  p.s_stride = score_stride;
  p.bt = block_table;
  p.bt_stride = block_table_stride;
  p.seq = seq_lens;
  p.q_len = q_len;
  p.B = block_size;
  p.selected = selected;
  p.sel_stride = selected_stride;
  p.columns = columns;
  p.lens = selected_lens;
  p.keep = keep;
  p.first = first;
  p.last = last;
  p.err = error_flag;
  int sms = 0;
  const int st = sm_count(&sms);
  if (st != PMG_OK) return st;
  // Long rows in a larger CTA, and shorter ones while each has an SM for itself: 2 rows of 938 pages 4.3 us instead of 6.3,
  // one of 8000 10.1 instead of 23; but 256 rows of 938 pages 9.4 instead of 8.2, 1000 of 512 27 instead of 9. The host does
  // not know the lengths: a row is as long as the table is wide, and many short rows in a table of more than 2048 columns
  // take those 27.
  const int64_t rows = static_cast<int64_t>(num_reqs) * q_len;
  const dim3 grid(static_cast<unsigned>(rows));
  return block_table_stride > 2048 || (block_table_stride > 512 && rows <= sms) ? launch(select_kernel<1024>, grid, 1024, 0, stream, p)
                                                                                : launch(select_kernel<256>, grid, 256, 0, stream, p);
}
