// Queries of the tensor-core decode kernels, from global into shared memory.
#pragma once

#include "mla_sm103.cuh"

namespace pmg_mla {

constexpr int kEntry = 576;  // values of an entry

__device__ __forceinline__ float half_of(uint32_t two, int i, bf16) { return __uint_as_float(i ? two & 0xffff0000u : two << 16); }
__device__ __forceinline__ float half_of(uint32_t two, int i, f16) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(i ? two >> 16 : two & 0xffff)));
}

// One row group's queries into shared memory, K-major. A warp takes every
// fourth row, several rows' loads in flight; the rows are then converted one at
// a time by one copy of the code.
//   row_at(r): where row r of the group begins
template <class TQ, int kParts, int N, class Misc, class RowAt>
__device__ __forceinline__ void load_queries(RowAt row_at, int n_rows, uint8_t* q_smem, Misc& mi, float factor) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kUnits = kEntry / 8;  // 16 bytes each
  constexpr int kBatch = N < 32 ? N / 4 : 8;  // rows of a warp in flight
#pragma unroll 1
  for (int r0 = warp; r0 < N; r0 += 4 * kBatch) {
    uint4 x[kBatch][3];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + 4 * i;
      const uint4* src = reinterpret_cast<const uint4*>(row_at(min(r, n_rows - 1)));
#pragma unroll
      for (int k = 0; k < 3; ++k)
        x[i][k] = r < n_rows && lane + 32 * k < kUnits ? src[lane + 32 * k] : make_uint4(0, 0, 0, 0);
    }
    // (two rows a turn: their chains of instructions overlap)
#pragma unroll 1
    for (int i0 = 0; i0 < kBatch; i0 += 2) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = r0 + 4 * (i0 + half);
        uint4 y[3] = {x[half][0], x[half][1], x[half][2]};
#pragma unroll
        for (int j = 2; j < kBatch; j += 2)
          if (i0 == j) {
            y[0] = x[j + half][0];
            y[1] = x[j + half][1];
            y[2] = x[j + half][2];
          }
        if constexpr (kParts == 1) {
          if (lane == 0) mi.factor[r] = factor;
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int u = lane + 32 * k;
            if (u < kUnits) *reinterpret_cast<uint4*>(q_smem + (u >> 3) * (N * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = y[k];
          }
        } else {
          // largest magnitude: 16-bit floats without their signs are ordered as whole numbers
          uint32_t top2 = 0;
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint32_t w[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top2 = __vmaxu2(top2, w[j] & 0x7fff7fffu);
          }
          const uint32_t top16 = __reduce_max_sync(0xffffffffu, max(top2 & 0xffff, top2 >> 16));
          const uint32_t top = __float_as_uint(half_of(top16, 0, TQ()));
          // 2^e * top in [224, 448), 224 = 1.75 * 2^7, with 2^e and its inverse normal numbers
          int e = 135 - static_cast<int>(top >> 23) - ((top & 0x7fffff) >= 0x600000 ? 1 : 0);
          e = top == 0 ? 0 : max(-126, min(126, e));
          const float scale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
          // (an infinite or NaN query makes NaN of its row, which e4m3 values that saturate would not)
          if (lane == 0)
            mi.factor[r] = top < 0x7f800000u ? factor * __uint_as_float(static_cast<uint32_t>(127 - e) << 23)
                                             : __uint_as_float(0x7fffffffu);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int u = lane + 32 * k;  // 8 values: 8 bytes of each part
            if (u < kUnits) {
              uint32_t v[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = pack2<f16>(half_of(v[j], 0, TQ()) * scale, half_of(v[j], 1, TQ()) * scale);
              uint8_t* dst = q_smem + (u >> 4) * (N * 128) + r * 128 + ((((u & 15) >> 1) ^ (r & 7)) << 4) + (u & 1) * 8;
#pragma unroll
              for (int c = 0; c < kParts; ++c) {
                uint32_t q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = e4m3_part(v[j]);
                *reinterpret_cast<uint2*>(dst + c * (5 * N * 128)) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
              }
            }
          }
        }
      }
    }
  }
}

}  // namespace pmg_mla
