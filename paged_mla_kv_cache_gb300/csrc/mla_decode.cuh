// Parameters, length arithmetic and work lists of the decode kernels.
//
// A call over shared prefixes (pmg_latent_decode_shared) is two passes of these
// kernels, whose rows a join of its own finishes (mla_shared.cu). The first, a
// prefix pass, takes groups of requests in place of requests: `cu` says which, bt
// and seq_lens are the prefixes', R is their number, and all rows of a group see
// all of its prefix. The second is a decode over the requests' own entries. Both
// leave every row's unnormalised sums, reference (in base 2) and sum of weights:
// of rows whose keys one share held in `state`, of others in the shares' slots.
// Neither reads what the other writes, so the second starts where the first
// leaves SMs free, and ends after it.
#pragma once

#include "mla_attn.cuh"

namespace pmg_mla {

constexpr int kDecodeTile = 64;  // keys of one piece of work

// Where a pass left a row.
struct RowNote {
  uint16_t cta, parts;  // in the slots of so many shares from this CTA's on; 0: in the state
  int32_t row;          // which row of a slot
};

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
  const int32_t* cu;  // a prefix pass: the groups' first requests
  int32_t reqs;       // and how many requests there are
  float* state;       // [rows][dv] of a pass of a call over shared prefixes, or NULL
  float* state_ml;    // [rows][2]: reference and sum
  RowNote* row_notes; // [rows]
  int32_t* covered;   // [2]: requests whose rows have a prefix, noted by the prefix pass
};

// The beginning and end of a kernel of a pass: the second pass does not wait for
// the first, whose launch of it comes when the kernels before are done, but ends
// after it.
template <bool kPrefix>
__device__ __forceinline__ void pass_entry(const DecodeParams& p) {
  if constexpr (kPrefix) {
    pdl_wait();
    pdl_launch();
  } else {
    if (p.state != nullptr) pdl_launch();
    else pdl_entry();
  }
}
template <bool kPrefix>
__device__ __forceinline__ void pass_exit(const DecodeParams& p) {
  if (!kPrefix && p.state != nullptr) pdl_wait();
}

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

// (lengths go up to INT32_MAX: no sum passes it before it is divided)
__device__ __forceinline__ int tiles_of(int len) {
  return static_cast<int>((static_cast<uint32_t>(len) + kDecodeTile - 1) / kDecodeTile);
}
// Pieces of a request of `len` keys: its tiles and kCost idle ones for its
// beginning and end (queries, first reference, epilogue). An empty request has
// one, which writes its rows.
template <int kCost>
__device__ __forceinline__ int pieces_of(int len) { return len > 0 ? kCost + tiles_of(len) : 1; }
// The tensor-core kernel's: without them the CTAs that got many short requests ended last.
constexpr int kItemCost = 4;

// ---- prefix passes -----------------------------------------------------------------

// Requests [from, to) of a group: boundaries are cut to the requests that there
// are, a decrease gives none. Every request from the first boundary on and below
// the largest one is then in some group: a path of whole numbers from the one to
// the other steps over it.
struct Group {
  int32_t from, to;
  int bad;
};
__device__ __forceinline__ Group group_of(const DecodeParams& p, int g) {
  const int32_t first = p.cu[0], a = p.cu[g], b = p.cu[g + 1];
  Group x;
  x.from = min(max(max(a, first), 0), p.reqs);
  x.to = max(x.from, min(max(b, 0), p.reqs));
  x.bad = a < 0 || b < a ? PMG_FLAG_CU_ORDER : 0;
  return x;
}

// By a whole CTA of the prefix pass, which reports what is wrong with the groups too; `to` is shared.
__device__ __forceinline__ void note_covered(const DecodeParams& p, int tid, int threads, int32_t& to) {
  if (tid == 0) to = 0;
  __syncthreads();
  int32_t mine = 0;
  int bad = 0;
  for (int g = tid; g < p.R; g += threads) {
    const Group x = group_of(p, g);
    if (x.to > x.from) mine = max(mine, x.to);
    bad |= x.bad | decode_len(p, g).bad;
  }
  atomicMax(&to, mine);
  set_flag(p.err, bad);
  __syncthreads();
  if (tid == 0) {
    p.covered[0] = min(max(p.cu[0], 0), p.reqs);
    p.covered[1] = to;
  }
}

// (rows of a call go up to INT32_MAX: 32-bit divisions, which cost a tenth of those of 64 bits)
__device__ __forceinline__ uint32_t group_tiles(const DecodeParams& p, const Group& x) {
  const uint32_t rows = static_cast<uint32_t>((x.to - x.from) * p.q_len * p.H), n = static_cast<uint32_t>(p.rows_per_group);
  return (rows + n - 1) / n;
}
template <int kCost>
__device__ __forceinline__ int64_t prefix_pieces(const DecodeParams& p, int g) {
  const int64_t tiles = group_tiles(p, group_of(p, g));
  return tiles > 0 ? tiles * pieces_of<kCost>(decode_len(p, g).use) : 0;
}

// Walks the row tiles of a share of a prefix pass: pieces of a group, row tile
// after row tile.
template <int kCost>
struct PrefixItems {
  const DecodeParams* p;
  int64_t at, end;
  int64_t off, total;   // pieces of the group before `at`, and all
  int64_t skip;         // pieces of the first group before the share
  int64_t first;        // the row tile's first piece
  int b;                // group
  int row_tile;
  int row0;             // the row tile's first row, of all rows of the call
  int group_row0, group_rows;
  int n_rows;           // its rows
  int tile, tiles;      // first tile of keys of this share, tiles of the prefix
  int n;                // tiles of this share
  int len, full_len;
  __device__ PrefixItems(const DecodeParams& p_, const Share& s) : p(&p_), at(s.begin), end(s.end), b(s.item - 1) {
    off = total = first = 0;
    row0 = group_row0 = group_rows = 0;
    row_tile = n_rows = tile = tiles = n = len = full_len = 0;
    skip = s.offset;
  }
  // the next row tile of which this share has tiles, or whose prefix is empty
  __device__ bool next() {
    do {
      if (at >= end) return false;
      while (off >= total) {
        ++b;
        const Group x = group_of(*p, b);
        const DecodeLen l = decode_len(*p, b);
        len = full_len = l.use;
        group_row0 = x.from * p->q_len * p->H;
        group_rows = (x.to - x.from) * p->q_len * p->H;
        total = static_cast<int64_t>(group_tiles(*p, x)) * pieces_of<kCost>(len);
        off = skip;
        skip = 0;
      }
      const int per = pieces_of<kCost>(len);
      row_tile = static_cast<int>(off <= UINT32_MAX ? static_cast<uint32_t>(off) / static_cast<uint32_t>(per) : off / per);
      const int in = static_cast<int>(off - static_cast<int64_t>(row_tile) * per);
      const int take = static_cast<int>(min(static_cast<int64_t>(per - in), end - at));
      tiles = tiles_of(len);
      tile = max(0, in - kCost);
      n = max(0, in + take - kCost) - tile;
      first = at - in;
      row0 = group_row0 + row_tile * p->rows_per_group;
      n_rows = min(p->rows_per_group, group_row0 + group_rows - row0);
      at += take;
      off += take;
    } while (n == 0 && len > 0);
    return true;
  }
  // the piece of the row tile's last tile
  __device__ int64_t last_piece() const { return first + kCost + tiles - 1; }
};

// ---- host: what the entries share --------------------------------------------------

// Checks the arguments of a decode and fills p (workspace and state apart). PMG_OK
// with p.R == 0: there is nothing to do.
int decode_params(DecodeParams& p, const void* q, int64_t q_req_stride, int64_t q_token_stride, int64_t q_head_stride,
                  const void* cache, int64_t cache_block_stride, int64_t cache_token_stride, int64_t num_blocks,
                  const int32_t* block_table, int64_t block_table_stride, const int32_t* seq_lens, int32_t num_reqs,
                  int32_t q_len, int32_t heads, int32_t latent_dim, int32_t rope_dim, int32_t block_size,
                  int32_t q_dtype, int32_t cache_dtype, const float* scale, float sm_scale, void* out,
                  int64_t out_req_stride, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                  void* workspace, int32_t* error_flag, uint32_t options);

// Launch a decode over the requests' entries, or a prefix pass, without a join.
int run_decode(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream, uint32_t options);
int run_prefix(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream, uint32_t options);
// A decode over the requests' entries with its join.
int decode_alone(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream, uint32_t options);

// Tiles of a request; an empty one has a piece too, which writes its rows.
__device__ __forceinline__ int64_t decode_tiles(const DecodeParams& p, int b) {
  const int64_t n = decode_len(p, b).use;
  return n > 0 ? (n + kDecodeTile - 1) / kDecodeTile : 1;
}

}  // namespace pmg_mla
