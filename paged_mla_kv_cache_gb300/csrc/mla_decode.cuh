// Parameters and length arithmetic of the decode kernels.
#pragma once

#include "mla_attn.cuh"

namespace pmg_mla {

constexpr int kDecodeTile = 64;  // keys of one piece of work

struct DecodeParams {
  const void* q;
  int64_t qr_stride, qt_stride, qh_stride;
  const void* cache;
  int64_t blk_stride, tok_stride;
  int64_t num_blocks;
  const int32_t* bt;
  int64_t bt_stride;
  const int32_t* seq_lens;
  int32_t R, q_len, H;
  int32_t dv, dr, B;
  const float* scale;
  float sm_scale;
  void* out;
  int64_t or_stride, ot_stride, oh_stride;
  float* lse;
  Workspace ws;
  int32_t* err;
  int32_t rows_per_group, groups, units;
  int64_t slot_floats;
  int32_t out_pairs;  // rows of out begin at 4 bytes
  int32_t q_tma;      // heads of a query box (0: queries are loaded and converted by the softmax warps)
};

struct DecodeLen {
  int32_t full;  // the request's length
  int32_t use;   // keys with a table entry
  int bad;
};

__device__ __forceinline__ DecodeLen decode_len(const DecodeParams& p, int b) {
  DecodeLen l;
  l.full = p.seq_lens[b];
  l.bad = 0;
  if (l.full < 0) {
    l.full = 0;
    l.bad = PMG_FLAG_LENGTH;
  }
  const int64_t room = p.bt_stride * p.B;
  l.use = l.full;
  if (l.full > room) {
    l.use = static_cast<int32_t>(room);
    l.bad |= PMG_FLAG_LOGICAL_BLOCK;
  }
  return l;
}

// Tiles of a request; an empty one has a piece too, which writes its rows.
__device__ __forceinline__ int64_t decode_tiles(const DecodeParams& p, int b) {
  const int64_t n = decode_len(p, b).use;
  return n > 0 ? (n + kDecodeTile - 1) / kDecodeTile : 1;
}

}  // namespace pmg_mla
