// Parameters of the page scores' kernels.
#pragma once

#include "mla_attn.cuh"
#include "mla_long.cuh"
#include "pmg_long.h"

namespace pmg_mla {

struct ScoreParams {
  const uint8_t* q;
  int64_t qr_stride, qt_stride, qh_stride;
  const uint8_t* bounds;
  int64_t bb_stride, br_stride;
  int64_t num_blocks;
  const int32_t* bt;
  int64_t bt_stride;
  const int32_t* seq;
  int32_t R, q_len, H, E, B;
  const float* scale;
  float sm_scale;
  const float* lse;
  float* scores;
  int64_t s_stride;
  int32_t units;
  int32_t* err;
};

// Columns of a request of which some token sees an entry, and pieces of work of
// kScoreTile columns. Whoever has the last piece writes the columns behind them;
// a request without any has a piece for that.
constexpr int kScoreTile = 64;
__device__ __forceinline__ int64_t score_pages(const ScoreParams& p, const SparseLen& l) {
  const uint32_t n = static_cast<uint32_t>(sparse_seen(l, p.q_len - 1, p.q_len)), b = static_cast<uint32_t>(p.B);
  return (n + b - 1) / b;
}
__device__ __forceinline__ int64_t score_tiles(int64_t pages) { return (pages + kScoreTile - 1) / kScoreTile; }
__device__ __forceinline__ int64_t score_pieces(const ScoreParams& p, int r) {
  return max(score_tiles(score_pages(p, sparse_len(p.seq, r, p.bt_stride, p.B))), static_cast<int64_t>(1));
}

__device__ __forceinline__ float score_shift(const ScoreParams& p, int64_t row) {
  const float x = p.lse != nullptr ? p.lse[row] : 0.0f;
  return isfinite(x) ? x : 0.0f;
}

// One row's sum as it is defined, by a warp; a lane takes N values at a time. The
// kernels add max(q, 0) hi and min(q, 0) lo, of which one is a product with 0: NaN
// where that bound is infinite, although the other one bounds the page. They come
// here only with a sum of NaN.
template <class T, int N>
__device__ __forceinline__ float score_sum_odd(const T* q, const T* hi, const T* lo, int E) {
  float x = 0.0f;
  for (int d = (threadIdx.x & 31) * N; d < E; d += 32 * N) {
    Values<T, N> y, a, b;
    y.load(q + d);
    a.load(hi + d);
    b.load(lo + d);
#pragma unroll
    for (int k = 0; k < N; ++k) x += max_nan(to_f(y.v[k]) * to_f(a.v[k]), to_f(y.v[k]) * to_f(b.v[k]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Columns [from, width) of a request that no token sees anything of.
__device__ __forceinline__ void score_rest(const ScoreParams& p, int r, int64_t from, int tid, int threads) {
  for (int i = 0; i < p.q_len; ++i) {
    float* row = p.scores + (static_cast<int64_t>(r) * p.q_len + i) * p.s_stride;
    for (int64_t c = from + tid; c < p.bt_stride; c += threads) row[c] = -INFINITY;
  }
}

// The tensor-core kernel: entries of 576 16-bit values, rows of 16 bytes.
bool scores_tc_takes(const ScoreParams& p, int dtype);
int scores_tc(const ScoreParams& p, int dtype, void* stream);

}  // namespace pmg_mla
