// What the operators for long contexts share: values that keep NaN, and how
// much of a request each of its new tokens sees.
#pragma once

#include <type_traits>

#include "mla_common.cuh"

namespace pmg_mla {

// Maximum and minimum that a NaN does not drop out of.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// N values moved in pieces of 16 bytes (one element alone as it is).
template <class T, int N>
struct Values {
  static constexpr int kBytes = N * static_cast<int>(sizeof(T));
  alignas(kBytes < 16 ? sizeof(T) : 16) T v[N];
  __device__ __forceinline__ void load(const T* src) {
    if constexpr (kBytes < 16) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = src[i];
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(src)[i];
    }
  }
  __device__ __forceinline__ void store(T* dst) const {
    if constexpr (kBytes < 16) {
#pragma unroll
      for (int i = 0; i < N; ++i) dst[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(v)[i];
    }
  }
};

// Lengths of the sparse calls: what a request has, as far as its table reaches.
struct SparseLen {
  int32_t full;  // its length
  int64_t room;  // places of its row of the table
  int bad;
};
__device__ __forceinline__ SparseLen sparse_len(const int32_t* seq_lens, int r, int64_t width, int block_size) {
  SparseLen l{seq_lens[r], width * block_size, 0};
  if (l.full < 0) {
    l.full = 0;
    l.bad = PMG_FLAG_LENGTH;
  }
  if (l.full > l.room) l.bad |= PMG_FLAG_LOGICAL_BLOCK;
  return l;
}
// entries that token i of q_len sees
__device__ __forceinline__ int64_t sparse_seen(const SparseLen& l, int i, int q_len) {
  const int64_t n = static_cast<int64_t>(l.full) - q_len + 1 + i;
  return n < 0 ? 0 : n < l.room ? n : l.room;
}

}  // namespace pmg_mla
