// Absorbed latent attention on the fifth-generation tensor core: entries of
// 512 latent and 64 rotated values, 16-bit queries, a 16-bit or e4m3 cache.
//
// Mathematics. For a group of N query rows (heads, or heads of a few tokens) a
// tile of 64 entries E gives S^T = E Q^T (64 x N) and, with P = 2^(S - ref)
// for a reference `ref` of each row, O^T += E[:, :512]^T P (512 x N). The
// entries are the M side of both products, so the number of rows is the free
// N side (16, 32 or 64) and is not padded to 128, the tile is read from HBM
// once, staged once in shared memory, and used K-major for S and MN-major for
// O. O^T (four accumulators of 128 x N) and two S^T stay in tensor memory.
//
// Bound: the cache's bytes, up to about 64 rows a request (a CTA reads 1152
// bytes for 64 * 1088 multiply-adds); with 128 rows two CTAs read the same
// entries side by side, the second from L2, and the tensor core's products come
// to about the same time as the stream. Measured: 64 ragged requests of 1 to
// 32768 entries, 128 heads, 83 us (1.83 TB/s, 390 TFLOP/s; memory at 29%, the
// tensor pipe at 32% of the kernel's 70 us): neither bounds it. A tile's way
// from its scores over its weights to its freed slots is one chain of about
// 2 us, with one buffer of weights and one group of softmax warps. 8 skewed
// requests over an e4m3 cache, 64 heads of 2 tokens, 55 us (memory at 7%, the
// tensor pipe at 23% of 47 us), with three tiles in flight where the 16-bit
// layout has two. One request of 60000 entries, 16 heads, 31 us (floor 10):
// the first loads, seven tiles a CTA and the join.
//
// Roles: warp 4 loads (a copy a tile where a page holds whole tiles, else one
// for each page: pages of any multiple of 8 tokens), warp 5 issues products,
// warps 0-3 do the softmax and the epilogue. An entry tile travels as four
// slots of 128 latent values and one of the rotated part. One barrier tells of
// a tile's arrival (a barrier a slot, with scores issued slot by slot, measured
// 99 us instead of 82 on the ragged case above), each slot is freed by itself
// when its product is done, so loads run up to two tiles ahead of the softmax.
//
// The reference of a row follows its maximum only when a score passes it by
// 2^kCap: weights then stay inside the range of their type (fp16 ones are kept
// from 2^8 to 2^15 where the largest are, so that those beside a strong key do
// not fall below 2^-24). They are rounded to the type of the entries for the
// second product (2^-8 or 2^-11 of each; wider ones would need the entries
// widened too), their sum is of the unrounded ones. Sums are 32-bit, and the accumulators are rescaled (read, multiplied, written back)
// only in the first tiles of a request. All threads learn whether a tile needs
// that from one barrier with a vote, so the usual tile has no maximum over
// the lanes at all.
//
// An e4m3 cache is not widened. The 8-bit tensor core multiplies it as it is
// with queries and weights split in parts (x = x0 + x1 + ...).
// Queries: e4m3 parts of 4 significant bits, two for a bf16 query's 8 bits,
// three for an fp16 query's 11, after a scaling by a power of two for each row
// that puts its largest value in [224, 448); what is lost is below a step of
// 2^-9, 2^-16.8 of the largest.
// Weights: rounded to fp16, then three e5m2 parts of 3 significant bits, which
// holds them to 2^-9 of their value, as bf16 would, down to half a step of
// 2^-17. They are kept below 2^15.5 (fp16 ends at 2^16): a request's first
// tile sets its largest weights to 2^11, which leaves room for the maximum to
// grow as more entries come, later corrections to 2^13. So one strong key
// among n weak ones costs them at most n 2^-28 of its weight. (Two e4m3 parts,
// one product less, end at 2^-10 with the largest at 2^4: of a tail of 16384
// keys that together weigh as much as a strong first one a quarter was lost.)
#include <algorithm>
#include <type_traits>

#include "mla_decode.cuh"
#include "mla_decode_tc.cuh"
#include "mla_sm103.cuh"

namespace pmg_mla {
namespace {

constexpr int kThreads = 192;
constexpr int kSoft = 128;          // threads of the softmax warps
constexpr int kLatent = 512, kRope = 64, kEntry = kLatent + kRope;
constexpr int kSmemMax = 232448;    // shared memory a CTA can have

// Shared memory of one variant. Slots hold 64 rows of 128-byte pieces.
template <int kParts, int N>
struct Lay {
  static constexpr bool kFp8 = kParts > 1;
  static constexpr int kPiece = 64 * 128;                // 64 rows of one 128-byte piece
  static constexpr int kPieces = kFp8 ? 1 : 2;           // pieces of a slot: 128 latent values
  static constexpr int kSlot = kPiece * kPieces;
  static constexpr int kQPieces = kFp8 ? 5 : 9;
  static constexpr int kQ = kQPieces * N * 128 * kParts;
  static constexpr int kWeights = kFp8 ? 3 : 1;          // parts of a weight
  static constexpr int kP = kPiece * kWeights;
  static constexpr int kMisc = 2048;
  static constexpr int kRoom = kSmemMax - 1024 - kMisc - kQ - kP;
  // a rope slot for each tile in flight
  static constexpr int kTiles = kRoom / (4 * kSlot + kPiece);
  static constexpr int kRopeSlots = kTiles + (kRoom - kTiles * (4 * kSlot + kPiece) >= kPiece + kSlot ? 1 : 0);
  static constexpr int kSlotsFit = (kRoom - kRopeSlots * kPiece) / kSlot;
  static constexpr int kSlots = kSlotsFit < 24 ? kSlotsFit : 24;
  static constexpr int kQAt = 0;
  static constexpr int kPAt = kQAt + kQ;
  static constexpr int kSlotAt = kPAt + kP;
  static constexpr int kRopeAt = kSlotAt + kSlots * kSlot;
  static constexpr int kMiscAt = kRopeAt + kRopeSlots * kPiece;
  static constexpr int kBytes = kMiscAt + kMisc + 1024;
  static_assert(kTiles >= 2 && kRopeSlots <= 8 && kBytes <= kSmemMax, "two tiles in flight, notes for all");
};

template <int kSlots, int kRopeSlots, int N>
struct MiscOf {
  uint64_t full[kRopeSlots], rope_empty[kRopeSlots], empty[kSlots];  // a tile is full as a whole, by its rope slot
  uint64_t s_full[2], s_free[2], p_full, pv_done, q_full, q_empty, end;
  uint64_t mask[8];      // entries of a tile that exist, by tile & 7
  union {
    struct {
      int64_t scratch[33], found[2];  // while the share is looked up
    };
    float warp_sums[4 * N];
  };
  float factor[N];       // of each row: what a raw score is multiplied by
  union {
    float alpha[N];      // what its sums are multiplied by as its reference moves
    float inv[N];        // what its result is multiplied by
  };
  uint8_t step[N];       // which of the group's new tokens it belongs to
  uint32_t tmem;
  int32_t stop, never;
};

// Pieces of a request of `len` keys: its tiles and kItemCost idle ones for its
// beginning and end (queries, first reference, epilogue). An empty request has
// one, which writes its rows. (Four: without them the CTAs that got many short
// requests ended last.)
constexpr int kItemCost = 4;
// (lengths go up to INT32_MAX: no sum passes it before it is divided)
__device__ __forceinline__ int tiles_of(int len) {
  return static_cast<int>((static_cast<uint32_t>(len) + kDecodeTile - 1) / kDecodeTile);
}
__device__ __forceinline__ int pieces_of(int len) { return len > 0 ? kItemCost + tiles_of(len) : 1; }

// Walks the requests of a share. The next request's length is loaded one step
// early.
struct Items {
  const DecodeParams* p;
  int64_t at, end;
  int64_t first;    // the request's first piece
  int b;
  int tile, tiles;  // first tile of this share, tiles of the request
  int n;            // tiles of this share
  int len;          // keys of the request
  int full_len;
  int skip;         // pieces of the request before this share
  DecodeLen ahead;
  __device__ Items(const DecodeParams& p_, const Share& s) : p(&p_), at(s.begin), end(s.end), b(s.item - 1) {
    tile = tiles = n = len = full_len = 0;
    first = 0;
    skip = static_cast<int>(s.offset);
    if (at < end) ahead = decode_len(*p, s.item);
  }
  // the next request of which this share has tiles, or that is empty
  __device__ bool next() {
    do {
      if (at >= end) return false;
      ++b;
      len = ahead.use;
      full_len = ahead.full;
      if (b + 1 < p->R) ahead = decode_len(*p, b + 1);
      tiles = tiles_of(len);
      first = at - skip;
      const int take = static_cast<int>(min(static_cast<int64_t>(pieces_of(len) - skip), end - at));
      tile = max(0, skip - kItemCost);
      n = max(0, skip + take - kItemCost) - tile;
      at += take;
      skip = 0;
    } while (n == 0 && len > 0);
    return true;
  }
  // the piece of the request's last tile
  __device__ int64_t last_piece() const { return first + kItemCost + tiles - 1; }
};

__device__ __forceinline__ float half_of(uint32_t two, int i, bf16) { return __uint_as_float(i ? two & 0xffff0000u : two << 16); }
__device__ __forceinline__ float half_of(uint32_t two, int i, f16) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(i ? two >> 16 : two & 0xffff)));
}

// One row group's queries into shared memory, K-major. A warp takes every
// fourth row, several rows' loads in flight; the rows are then converted one at
// a time by one copy of the code.
template <class TQ, int kParts, int N, class Misc>
__device__ __forceinline__ void load_queries(const DecodeParams& p, int b, int g0, int n_rows, uint8_t* q_smem,
                                             Misc& mi, float factor) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kUnits = kEntry / 8;  // 16 bytes each
  constexpr int kBatch = N < 32 ? N / 4 : 8;  // rows of a warp in flight
#pragma unroll 1
  for (int r0 = warp; r0 < N; r0 += 4 * kBatch) {
    uint4 x[kBatch][3];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + 4 * i, rr = g0 + min(r, n_rows - 1);
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const TQ*>(p.q) + b * p.qr_stride +
                                                        (rr / p.H) * p.qt_stride + (rr % p.H) * p.qh_stride);
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

template <class TQ, int kParts, int N>
__global__ void __launch_bounds__(kThreads, 1)
    decode_tc_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap map,
                     const __grid_constant__ CUtensorMap rope_map, const __grid_constant__ CUtensorMap q_map,
                     int box_rows) {
  using L = Lay<kParts, N>;
  constexpr bool kFp8 = kParts > 1;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  using Misc = MiscOf<L::kSlots, L::kRopeSlots, N>;
  static_assert(sizeof(Misc) <= L::kMisc, "fits");
  Misc& mi = *reinterpret_cast<Misc*>(smem + L::kMiscAt);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  constexpr int kColumns = N == 16 ? 128 : N == 32 ? 256 : 512;  // 2 S and 4 O accumulators of N columns

  // before the previous kernel's results are needed
  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) mbar_init(smem_u32(&mi.empty[i]), 1);
    for (int i = 0; i < L::kRopeSlots; ++i) {
      mbar_init(smem_u32(&mi.full[i]), 1);
      mbar_init(smem_u32(&mi.rope_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&mi.s_full[i]), 1);
      mbar_init(smem_u32(&mi.s_free[i]), 4);
    }
    mbar_init(smem_u32(&mi.p_full), 4);
    mbar_init(smem_u32(&mi.pv_done), 1);
    mbar_init(smem_u32(&mi.q_full), p.q_tma ? 1 : 4);
    mbar_init(smem_u32(&mi.q_empty), 1);
    mi.stop = mi.never = 0;
    mbar_init(smem_u32(&mi.end), 1);
    mbar_fence_init();
    tma_prefetch(&map);
    tma_prefetch(&rope_map);
    if (p.q_tma) tma_prefetch(&q_map);
  }
  if (warp == 5) tmem_alloc(smem_u32(&mi.tmem), kColumns);
  if (p.q_tma) {
    // rows of queries that no copy fills: 0, before the CTA's barrier below, after which they are multiplied
    const int fill = N - p.rows_per_group;
    for (int i = tid; i < 9 * fill * 8; i += kThreads) {
      const int c = i / (fill * 8), y = i % (fill * 8);
      *reinterpret_cast<uint4*>(smem + L::kQAt + c * (N * 128) + p.rows_per_group * 128 + y * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
  }
  pdl_entry();

  const int unit = blockIdx.x / p.groups, group = blockIdx.x % p.groups;
  const Share share = find_share([&](int b) -> int64_t { return pieces_of(decode_len(p, b).use); }, p.R, unit, p.units,
                                 mi.scratch, mi.found);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = mi.tmem;
  const uint32_t stop = smem_u32(&mi.stop);
  constexpr int kFmt = kFp8 ? 0 : (sizeof(TQ) == 2 && std::is_same<TQ, bf16>::value ? 1 : 0);
  constexpr uint32_t kIdescS = umma_idesc(kFmt, kFmt, 0, 0, 64, N);
  constexpr uint32_t kIdescO = umma_idesc(kFmt, kFp8 ? 1 : kFmt, 1, 1, 128, N);  // e5m2 weights of e4m3 values

  if (warp == 4) {
    // ---- loads ----
    Items it(p, share);
    int slot = 0, phase = 0, rslot = 0, rphase = 0;
    uint32_t t = 0;
    int bad = 0;
    bool alive = true;
    const uint32_t full = smem_u32(&mi.full[0]), empty = smem_u32(&mi.empty[0]), rope_empty = smem_u32(&mi.rope_empty[0]);
    uint32_t items = 0;
    const int segs = kDecodeTile / box_rows;  // boxes of a tile along its rows: 1, 2, 4 or 8
    while (alive && it.next()) {
      if (lane == 0) bad |= decode_len(p, it.b).bad;
      if (it.len == 0) continue;
      const int32_t* table = p.bt + static_cast<int64_t>(it.b) * p.bt_stride;
      // lane s < segs looks up the page of box s, one tile ahead of its use (places have no sign: boxes past the end of a
      // request may lie past INT32_MAX)
      const uint32_t len = static_cast<uint32_t>(it.len);
      auto page_of = [&](uint32_t j) { return lane < segs && j < len ? table[j / static_cast<uint32_t>(p.B)] : -1; };
      uint32_t j = static_cast<uint32_t>(it.tile * kDecodeTile) + lane * box_rows;
      int next_id = page_of(j);
#pragma unroll 1
      for (int i = 0; i < it.n; ++i, ++t, j += kDecodeTile) {
        const int j0 = (it.tile + i) * kDecodeTile;
        const bool in = lane < segs && j < len;
        int id = next_id;
        const int row = static_cast<int>(j % static_cast<uint32_t>(p.B));
        next_id = i + 1 < it.n ? page_of(j + kDecodeTile) : -1;
        const bool good = id >= 0 && id < p.num_blocks;
        if (in && !good) {
          bad |= PMG_FLAG_PHYS_BLOCK;
          id = static_cast<int>(p.num_blocks);  // outside: the box is filled with zeros
        }
        const uint32_t boxes = __ballot_sync(0xffffffffu, in), goods = __ballot_sync(0xffffffffu, in && good);
        const int n_boxes = __popc(boxes);
        // which entries of the tile exist
        uint64_t mask = 0;
        for (int s = 0; s < segs; ++s)
          if (goods >> s & 1) mask |= (box_rows == 64 ? ~0ull : ((1ull << box_rows) - 1) << (s * box_rows));
        const int left = it.len - j0;
        if (left < 64) mask &= (1ull << left) - 1;
        const uint32_t bytes = static_cast<uint32_t>(n_boxes * box_rows * 128);
        const int id0 = __shfl_sync(0xffffffffu, id, 0), row0 = __shfl_sync(0xffffffffu, row, 0);
        if (box_rows == kDecodeTile && group == 0 && i + 1 < it.n) {
          // the next tile on its way into L2 while this one waits for slots
          const int next0 = __shfl_sync(0xffffffffu, next_id, 0);
          const int next_row = static_cast<int>(static_cast<uint32_t>(j0 + kDecodeTile) % static_cast<uint32_t>(p.B));
          if (next0 >= 0 && next0 < p.num_blocks && elect_one()) {
#pragma unroll 1
            for (int m = 0; m < 4; ++m) tma_prefetch_4d(&map, 0, next_row, m * L::kPieces, next0);
            tma_prefetch_3d(&rope_map, kLatent, next_row, next0);
          }
          __syncwarp();
        }
        if (stopped(stop)) {
          alive = false;
          break;
        }
        // the rotated part's slot, free since the tile's scores two tiles ago, brings the tile's barrier
        const uint32_t bar = full + 8 * rslot;
        mbar_wait(rope_empty + 8 * rslot, rphase ^ 1, stop);
        if (elect_one()) {
          mi.mask[t & 7] = mask;  // by the lane that arrives: the barrier orders it for its readers
          mbar_expect(bar, bytes * (4 * L::kPieces + 1));
        }
        __syncwarp();
        const bool one_box = n_boxes == 1 && box_rows == kDecodeTile;
        if (one_box) {
          if (elect_one()) tma_load_3d(base + L::kRopeAt + rslot * L::kPiece, &rope_map, bar, kLatent, row0, id0);
          __syncwarp();
        } else {
#pragma unroll 1
          for (int s = 0; s < n_boxes; ++s) {
            const int sid = __shfl_sync(0xffffffffu, id, s), srow = __shfl_sync(0xffffffffu, row, s);
            if (elect_one())
              tma_load_3d(base + L::kRopeAt + rslot * L::kPiece + s * box_rows * 128, &rope_map, bar, kLatent, srow, sid);
            __syncwarp();
          }
        }
#pragma unroll 1
        for (int m = 0; m < 4; ++m) {
          mbar_wait(empty + 8 * slot, phase ^ 1, stop);
          const uint32_t dst = base + L::kSlotAt + slot * L::kSlot;
          if (one_box) {
            if (elect_one()) tma_load_4d(dst, &map, bar, 0, row0, m * L::kPieces, id0);
          } else {
            // boxes of fewer rows than a slot has leave gaps between their pieces: a copy a piece
#pragma unroll 1
            for (int s = 0; s < n_boxes; ++s) {
              const int sid = __shfl_sync(0xffffffffu, id, s), srow = __shfl_sync(0xffffffffu, row, s);
              if (elect_one()) {
#pragma unroll
                for (int c = 0; c < L::kPieces; ++c)
                  tma_load_4d(dst + c * L::kPiece + s * box_rows * 128, &map, bar, 0, srow, m * L::kPieces + c, sid);
              }
            }
          }
          __syncwarp();
          if (++slot == L::kSlots) { slot = 0; phase ^= 1; }
        }
        if (++rslot == L::kRopeSlots) { rslot = 0; rphase ^= 1; }
        if (i == 0 && p.q_tma) {
          // the request's queries, once the products with the ones before are done
          if (items > 0) mbar_wait(smem_u32(&mi.q_empty), (items - 1) & 1, stop);
          ++items;
          if (elect_one()) {
            const int g0 = group * p.rows_per_group;
            const uint32_t bar = smem_u32(&mi.q_full);
            mbar_expect(bar, static_cast<uint32_t>(p.rows_per_group) * kEntry * 2);
#pragma unroll 1
            for (int c = 0; c < 9; ++c)
              tma_load_4d(base + L::kQAt + c * (N * 128), &q_map, bar, 64 * c, g0 % p.H, g0 / p.H, it.b);
          }
          __syncwarp();
        }
      }
    }
    set_flag(p.err, bad);
    if (!alive && items > 0) mbar_wait(smem_u32(&mi.q_full), (items - 1) & 1, smem_u32(&mi.never));
    // after a timeout, copies in flight land before the CTA ends (`never` is not set: these waits run on)
    if (!alive) {
      const uint32_t never = smem_u32(&mi.never);
      for (int i = 0; i < L::kRopeSlots; ++i) mbar_wait(full + 8 * i, i < rslot ? rphase : rphase ^ 1, never);
    }
  } else if (warp == 5) {
    // ---- products ----
    Items qi(p, share), vi(p, share);
    auto advance = [](Items& it) {
      bool more = it.next();
      while (more && it.len == 0) more = it.next();
      return more;
    };
    const uint32_t full = smem_u32(&mi.full[0]), empty = smem_u32(&mi.empty[0]), rope_empty = smem_u32(&mi.rope_empty[0]);
    const uint32_t s_full = smem_u32(&mi.s_full[0]), s_free = smem_u32(&mi.s_free[0]);
    bool q_more = advance(qi), v_more = advance(vi);
    int q_tile = 0, v_tile = 0;                 // within the items
    uint32_t q_item = 0;                        // items begun, for the queries' barrier
    uint32_t qt = 0, vt = 0;                    // tiles issued
    int qslot = 0, rslot = 0, rphase = 0, vslot = 0;
    const uint32_t p_full = smem_u32(&mi.p_full);
    // O of the oldest tile
    auto values = [&]() {
      tmem_fence_after();
      const bool first = v_tile == 0;
      if (elect_one()) {
        const uint64_t pa = umma_desc(base + L::kPAt, L::kPiece, 1024);
        int at = vslot;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint64_t va = umma_desc(base + L::kSlotAt + at * L::kSlot, L::kPiece, 1024);
          const uint32_t d = tmem + (2 + m) * N;
#pragma unroll
          for (int k = 0; k < (kFp8 ? 2 : 4); ++k) {
            const uint32_t step = k * (kFp8 ? 32 : 16) * 8;  // rows of 128 bytes, in units of 16
#pragma unroll
            for (int x = 0; x < L::kWeights; ++x)
              umma_ss<kFp8>(d, va + step, pa + step + x * (L::kPiece / 16), kIdescO, !first || k > 0 || x > 0);
          }
          umma_commit(empty + 8 * at);
          if (++at == L::kSlots) at = 0;
        }
        umma_commit(smem_u32(&mi.pv_done));
      }
      __syncwarp();
      vslot = vslot + 4 < L::kSlots ? vslot + 4 : vslot + 4 - L::kSlots;
      ++vt;
      if (++v_tile == vi.n) {
        v_tile = 0;
        v_more = advance(vi);
      }
    };
    // S of a tile when it has arrived; O of the tile before it once its weights are there: while the next tile is still
    // on its way, or at the latest after its scores.
    auto wait_for = [&](uint32_t bar, uint32_t parity) {
      while (vt != qt && mbar_wait_either(p_full, vt & 1, bar, parity, stop)) values();
      mbar_wait(bar, parity, stop);
    };
    while (q_more) {
      const uint32_t buf = qt & 1, d = tmem + buf * N;
      if (qt >= 2) mbar_wait(s_free + 8 * buf, ((qt >> 1) + 1) & 1, stop);
      if (q_tile == 0) {
        // the queries of a new request come after the last scores with the ones before
        wait_for(smem_u32(&mi.q_full), q_item & 1);
        ++q_item;
      }
      wait_for(full + 8 * rslot, rphase);
      tmem_fence_after();
      if (elect_one()) {
        int at = qslot;
#pragma unroll
        for (int part = 0; part < 4; ++part) {
#pragma unroll
          for (int c = 0; c < L::kPieces; ++c) {
            const uint64_t ka = umma_desc(base + L::kSlotAt + at * L::kSlot + c * L::kPiece, 16, 1024);
            const uint64_t qa = umma_desc(base + L::kQAt + (part * L::kPieces + c) * (N * 128), 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 32 bytes of K each
#pragma unroll
              for (int x = 0; x < kParts; ++x)
                umma_ss<kFp8>(d, ka + 2 * k, qa + 2 * k + x * (5 * N * 8), kIdescS, part > 0 || c > 0 || k > 0 || x > 0);
          }
          if (++at == L::kSlots) at = 0;
        }
        const uint64_t ka = umma_desc(base + L::kRopeAt + rslot * L::kPiece, 16, 1024);
        const uint64_t qa = umma_desc(base + L::kQAt + 4 * L::kPieces * (N * 128), 16, 1024);
#pragma unroll
        for (int k = 0; k < (kFp8 ? 2 : 4); ++k)
#pragma unroll
          for (int x = 0; x < kParts; ++x)
            umma_ss<kFp8>(d, ka + 2 * k, qa + 2 * k + x * (5 * N * 8), kIdescS, true);
        umma_commit(rope_empty + 8 * rslot);
        umma_commit(s_full + 8 * buf);
        if (p.q_tma && q_tile + 1 == qi.n) umma_commit(smem_u32(&mi.q_empty));
      }
      __syncwarp();
      qslot = qslot + 4 < L::kSlots ? qslot + 4 : qslot + 4 - L::kSlots;
      if (++rslot == L::kRopeSlots) { rslot = 0; rphase ^= 1; }
      ++qt;
      if (++q_tile == qi.n) {
        q_tile = 0;
        q_more = advance(qi);
      }
      if (qt - vt == 2) {
        mbar_wait(p_full, vt & 1, stop);
        values();
      }
    }
    while (v_more) {
      mbar_wait(p_full, vt & 1, stop);
      values();
    }
    // everything issued ends before the tensor memory is given back
    if (elect_one()) umma_commit(smem_u32(&mi.end));
    __syncwarp();
    mbar_wait(smem_u32(&mi.end), 0, smem_u32(&mi.never));
  } else {
    // ---- softmax and epilogue ----
    Items it(p, share);
    const int rows = p.q_len * p.H;
    const int g0 = group * p.rows_per_group;
    const int n_rows = min(p.rows_per_group, rows - g0);
    const float kv_scale = kFp8 && p.scale != nullptr ? *p.scale : 1.0f;
    const float factor = p.sm_scale * kLog2e * kv_scale;
    constexpr bool kF16 = std::is_same<TQ, f16>::value;
    constexpr float kCap = kFp8 ? 15.5f : kF16 ? 15.0f : 8.0f;       // weights stay below 2^kCap
    constexpr float kFirst = kFp8 ? 11.0f : kF16 ? 8.0f : 0.0f;      // where a first reference puts the largest
    constexpr float kLater = kFp8 ? 13.0f : kF16 ? 8.0f : 0.0f;      // where a later one does
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    // Scores (M = 64: 16 rows in each quarter of the lanes) are read so that this thread has entries tok and tok + 8
    // of the tile, and of every 8 columns 2 c and 2 c + 1.
    constexpr int kG = N / 8;
    const int c = lane & 3, tok = warp * 16 + (lane >> 2);
    JoinNote note{-1, 0, 0, 0};
    uint32_t t = 0;                 // tiles of the share
    uint32_t slot0 = 0;             // slot of the tile's first part
    uint32_t tile_slot = 0, tile_phase = 0;
    const int step0 = g0 / p.H;  // the group's first new token
    if (tid < N) mi.step[tid] = static_cast<uint8_t>((g0 + tid) / p.H - step0);
    // where row h of the group is in a request's output
    auto out_at = [&](int h) {
      const int step = step0 + mi.step[h];
      return step * p.ot_stride + (g0 + h - step * p.H) * p.oh_stride;
    };
    // For each request: its queries, then the epilogue of the request before (whose last product runs meanwhile), then
    // its tiles.
    bool more = it.next();
    int prev_b = -1, prev_n = 0;
    bool prev_whole = false;
    float* prev_slot = nullptr;
    for (;;) {
      if (more && it.len > 0 && !p.q_tma) {
        load_queries<TQ, kParts, N>(p, it.b, g0, n_rows, smem + L::kQAt, mi, factor);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&mi.q_full));
      }
      if (prev_b >= 0) {
        if (prev_n > 0) mbar_wait(smem_u32(&mi.pv_done), (t - 1) & 1, stop);
        tmem_fence_after();
        if (stopped(stop)) {  // a wait ran out: the rows become NaN by their factors or sums (every warp sees to it for itself)
          const float nan = __uint_as_float(0x7fffffffu);
#pragma unroll 1
          for (int i = lane; i < n_rows; i += 32) {
            mi.inv[i] = nan;
            if (!prev_whole) prev_slot[p.rows_per_group * kLatent + 2 * i + 1] = nan;
            else if (p.lse != nullptr) p.lse[static_cast<int64_t>(prev_b) * rows + g0 + i] = nan;
          }
          __syncwarp();
        }
        TQ* out = static_cast<TQ*>(p.out) + prev_b * p.or_stride;
        const int d = warp * 32 + lane;  // and 128 further for each m
#pragma unroll 1
        for (int h0 = 0; h0 < n_rows; h0 += 16) {
          uint32_t o[4][16];
          __syncwarp();
          if (prev_n > 0) {
#pragma unroll
            for (int m = 0; m < 4; ++m) tmem_ld16(tmem + (2 + m) * N + h0 + lanes, o[m]);
            tmem_wait_ld();
#pragma unroll
            for (int m = 0; m < 4; ++m) tmem_pin<16>(o[m]);
          } else {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
              for (int k = 0; k < 16; ++k) o[m][k] = 0;
          }
          if (!prev_whole) {
            float* at = prev_slot + h0 * kLatent + d;
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (h0 + k < n_rows) {
#pragma unroll
                for (int m = 0; m < 4; ++m) at[k * kLatent + m * 128] = __uint_as_float(o[m][k]) * kv_scale;
              }
          } else {
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              // even lanes write row k, odd lanes row k + 1, two neighbours' values each
              const int h = h0 + k + (lane & 1);
              const float ia = mi.inv[h0 + k], ib = mi.inv[h0 + k + 1];
              TQ* at = out + out_at(min(h, n_rows - 1)) + (d & ~1);
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const float a = __uint_as_float(o[m][k]) * ia, b = __uint_as_float(o[m][k + 1]) * ib;
                const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
                const uint32_t two = lane & 1 ? pack2<TQ>(other, b) : pack2<TQ>(a, other);
                if (h < n_rows) {
                  if (p.out_pairs) {
                    *reinterpret_cast<uint32_t*>(at + m * 128) = two;
                  } else {
                    reinterpret_cast<uint16_t*>(at + m * 128)[0] = static_cast<uint16_t>(two);
                    reinterpret_cast<uint16_t*>(at + m * 128)[1] = static_cast<uint16_t>(two >> 16);
                  }
                }
              }
            }
          }
        }
        tmem_fence_before();
      }
      if (!more) break;
      const int n = it.n;
      named_sync<kSoft>(1);  // the queries' factors are there, and everybody is done with the last request's sums
      float ref[2 * kG], l[2 * kG], f[2 * kG];  // of columns 8 g + 2 c and the next
#pragma unroll
      for (int i = 0; i < 2 * kG; ++i) {
        ref[i] = -INFINITY;
        l[i] = 0.0f;
        f[i] = kFp8 ? mi.factor[(i >> 1) * 8 + 2 * c + (i & 1)] : factor;
      }
      for (int i = 0; i < n; ++i, ++t) {
        const uint32_t buf = t & 1;
        const int j0 = (it.tile + i) * kDecodeTile;
        // the loading warp's note of the tile is ordered by the tile's barrier
        mbar_wait(smem_u32(&mi.full[0]) + 8 * tile_slot, tile_phase, stop);
        if (++tile_slot == L::kRopeSlots) { tile_slot = 0; tile_phase ^= 1; }
        mbar_wait(smem_u32(&mi.s_full[0]) + 8 * buf, t >> 1 & 1, stop);
        __syncwarp();
        tmem_fence_after();
        uint32_t raw_s[4 * kG];
        tmem_ld_rows16(tmem + buf * N + lanes, raw_s);
        const uint64_t mask = mi.mask[t & 7] >> tok;
        const bool in0 = mask & 1, in1 = mask >> 8 & 1;
        tmem_wait_ld();
        tmem_pin<4 * kG>(raw_s);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&mi.s_free[0]) + 8 * buf);
        float* s = reinterpret_cast<float*>(raw_s);
        const bool all = __all_sync(0xffffffffu, in0 && in1);
        // some row does not see the whole tile for its place among the new tokens
        const int common = it.full_len - j0 - p.q_len + 1;  // entries from the tile's first on that all rows see
        const bool edge = p.q_len > 1 && common < kDecodeTile;
        if (!all || edge) {
          const int first = common + step0 - tok;  // of row 0's token: entries tok + k < first are seen
#pragma unroll
          for (int g = 0; g < kG; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int step = edge ? mi.step[8 * g + 2 * c + (k & 1)] : 0;
              const bool seen = (k < 2 ? in0 : in1) && (!edge || (k < 2 ? 0 : 8) < first + step);
              // an unseen score is -inf whatever its entry holds (factors are not negative; 0 makes a NaN, cleared below)
              if (!seen) s[4 * g + k] = -INFINITY;
            }
        }
        // scores less the references; -inf less -inf only where nothing was seen yet, which raises nothing
        float x[4 * kG];
        float over = -INFINITY;
#pragma unroll
        for (int g = 0; g < kG; ++g)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float y = s[4 * g + k] == -INFINITY ? -INFINITY : fmaf(s[4 * g + k], f[2 * g + (k & 1)], -ref[2 * g + (k & 1)]);
            x[4 * g + k] = y;
            over = fmaxf(over, y);
          }
        const bool raise = named_any<kSoft>(2, over > kCap);
        if (raise) {
          // maximum of every row over the tile's entries
          float* part = reinterpret_cast<float*>(smem + L::kPAt);  // free once the last tile's product is done
          if (t > 0) mbar_wait(smem_u32(&mi.pv_done), (t - 1) & 1, stop);
          __syncwarp();
          tmem_fence_after();
#pragma unroll
          for (int k = 0; k < 2 * kG; ++k) {
            const float a = s[4 * (k >> 1) + (k & 1)], b = s[4 * (k >> 1) + (k & 1) + 2];
            float top = fmaxf(a == -INFINITY ? a : a * f[k], b == -INFINITY ? b : b * f[k]);
#pragma unroll
            for (int o = 16; o >= 4; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (lane < 4) part[warp * N + (k >> 1) * 8 + 2 * c + (k & 1)] = top;
          }
          named_sync<kSoft>(1);
#pragma unroll
          for (int k = 0; k < 2 * kG; ++k) {
            const int col = (k >> 1) * 8 + 2 * c + (k & 1);
            const float top = fmaxf(fmaxf(part[col], part[N + col]), fmaxf(part[2 * N + col], part[3 * N + col])) -
                              (ref[k] == -INFINITY ? kFirst : kLater);
            float a = 1.0f;
            if (top > ref[k]) {  // where the tile raises it at all
              a = ref[k] == -INFINITY ? 0.0f : ex2(ref[k] - top);
              ref[k] = top;
              l[k] *= a;
            }
            if (tid < 4) mi.alpha[col] = a;
          }
          named_sync<kSoft>(1);  // (also: the maxima's place is where the weights go)
          if (i > 0) {
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
#pragma unroll
              for (int h = 0; h < N; h += 16) {
                uint32_t o[16];
                const uint32_t at = tmem + (2 + m) * N + h + lanes;
                tmem_ld16(at, o);
                tmem_wait_ld();
                tmem_pin<16>(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * mi.alpha[h + k]);
                tmem_st16(at, o);
              }
            }
            tmem_wait_st();
            tmem_fence_before();
          }
#pragma unroll
          for (int g = 0; g < kG; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[4 * g + k] = s[4 * g + k] == -INFINITY ? -INFINITY : fmaf(s[4 * g + k], f[2 * g + (k & 1)], -ref[2 * g + (k & 1)]);
        }
        // weights
#pragma unroll
        for (int g = 0; g < kG; ++g)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[4 * g + k] = ex2(x[4 * g + k]);
            l[2 * g + (k & 1)] += x[4 * g + k];
          }
        // the last tile's product has read its weights
        if (t > 0) mbar_wait(smem_u32(&mi.pv_done), (t - 1) & 1, stop);
        // values past the end of the request may be anything: their weights are 0, so must they be
        const int first = it.len - j0;
        if (first < kDecodeTile) {
          for (uint32_t m = 0; m < 4; ++m) {
            const uint32_t sl = slot0 + m < L::kSlots ? slot0 + m : slot0 + m - L::kSlots;
            uint4* at = reinterpret_cast<uint4*>(smem + L::kSlotAt + sl * L::kSlot + first * 128);
            for (int y = tid; y < (kDecodeTile - first) * 8; y += kSoft) {
#pragma unroll
              for (int q = 0; q < L::kPieces; ++q) at[q * (L::kPiece / 16) + y] = make_uint4(0, 0, 0, 0);
            }
          }
        }
        if (edge) {
          // infinities and NaN of entries that some row does not see likewise; one that sees them has the NaN of its score
          using TC = std::conditional_t<kFp8, e4m3, TQ>;
#pragma unroll 1
          for (uint32_t m = 0; m < 4; ++m) {
            const uint32_t sl = slot0 + m < L::kSlots ? slot0 + m : slot0 + m - L::kSlots;
            uint4* at = reinterpret_cast<uint4*>(smem + L::kSlotAt + sl * L::kSlot);
#pragma unroll
            for (int y = tid; y < L::kSlot / 16; y += kSoft)
              if ((y >> 3) % kDecodeTile < first) at[y] = only_finite<TC>(at[y]);  // (the others are 0)
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint8_t* row = smem + L::kPAt + (tok + 8 * h) * 128;
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            const float a = x[4 * g + 2 * h], b = x[4 * g + 2 * h + 1];
            if constexpr (!kFp8) {
              *reinterpret_cast<uint32_t*>(row + ((g ^ (tok & 7)) << 4) + 4 * c) = pack2<TQ>(a, b);
            } else {
              uint8_t* at = row + (((g >> 1) ^ (tok & 7)) << 4) + (g & 1) * 8 + 2 * c;
              uint32_t two = pack2<f16>(a, b);
              const uint32_t part0 = e5m2_cut(two), part1 = e5m2_cut(two);
              reinterpret_cast<uint16_t*>(at)[0] = static_cast<uint16_t>(part0);
              reinterpret_cast<uint16_t*>(at + L::kPiece)[0] = static_cast<uint16_t>(part1);
              reinterpret_cast<uint16_t*>(at + 2 * L::kPiece)[0] = static_cast<uint16_t>(e5m2_last(two));
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&mi.p_full));
        slot0 += 4;
        if (slot0 >= L::kSlots) slot0 -= L::kSlots;
      }

      // sums of every row over the lanes, then over the warps in their order
      const bool whole = it.n == it.tiles;  // (an empty request too)
#pragma unroll
      for (int k = 0; k < 2 * kG; ++k) {
#pragma unroll
        for (int o = 16; o >= 4; o >>= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], o);
        if (lane < 4) mi.warp_sums[warp * N + (k >> 1) * 8 + 2 * c + (k & 1)] = l[k];
      }
      if (tid < 4) {  // these four have all references; the factors are in registers by now
#pragma unroll
        for (int k = 0; k < 2 * kG; ++k) mi.factor[(k >> 1) * 8 + 2 * c + (k & 1)] = ref[k];
      }
      named_sync<kSoft>(1);
      float* slot = p.ws.slots + (static_cast<int64_t>(blockIdx.x) * 2 + (it.tile == 0 ? 1 : 0)) * p.slot_floats;
      if (tid < N) {
        const float sum = (mi.warp_sums[tid] + mi.warp_sums[N + tid]) + (mi.warp_sums[2 * N + tid] + mi.warp_sums[3 * N + tid]);
        const float r = mi.factor[tid];
        mi.inv[tid] = sum != 0.0f ? kv_scale / sum : 0.0f;
        if (tid < n_rows) {
          if (!whole) *reinterpret_cast<float2*>(slot + p.rows_per_group * kLatent + 2 * tid) = make_float2(r, sum);
          else if (p.lse != nullptr)
            p.lse[static_cast<int64_t>(it.b) * rows + g0 + tid] = sum != 0.0f ? (r + log2f(sum)) * kLn2 : -INFINITY;
        }
      }
      if (!whole && it.tile == 0 && tid == 0) {
        note.item = it.b;
        note.parts = unit_of(it.last_piece(), share.total, share.units) - unit + 1;
      }
      named_sync<kSoft>(1);  // the rows' factors are there for the epilogue
      prev_b = it.b;
      prev_n = n;
      prev_whole = whole;
      prev_slot = slot;
      more = it.next();
    }
    if (tid == 0 && p.units > 1) p.ws.notes[blockIdx.x] = note;
    if (stopped(stop) && tid == 0) set_flag(p.err, PMG_FLAG_TIMEOUT);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 5) tmem_free(tmem, kColumns);
}

struct Maps {
  CUtensorMap latent, rope, q;
};

template <class TQ, int kParts, int N>
int run(const DecodeParams& p, const Maps& maps, int box_rows, void* stream) {
  auto k = decode_tc_kernel<TQ, kParts, N>;
  constexpr int kBytes = Lay<kParts, N>::kBytes;
  const int st = allow_smem(reinterpret_cast<const void*>(k), kBytes);
  if (st != PMG_OK) return st;
  return launch(k, dim3(static_cast<unsigned>(p.units) * p.groups), kThreads, kBytes, stream, p, maps.latent, maps.rope,
                maps.q, box_rows);
}

template <class TQ, int kParts>
int run(const DecodeParams& p, const Maps& maps, int box_rows, void* stream) {
  if (p.rows_per_group <= 16) return run<TQ, kParts, 16>(p, maps, box_rows, stream);
  if (p.rows_per_group <= 32) return run<TQ, kParts, 32>(p, maps, box_rows, stream);
  return run<TQ, kParts, 64>(p, maps, box_rows, stream);
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

}  // namespace

bool decode_tc_takes(const DecodeParams& p, int q_dtype, int cache_dtype) {
  const int ec = elem_bytes(cache_dtype);
  return p.dv == kLatent && p.dr == kRope && (q_dtype == PMG_BF16 || q_dtype == PMG_FP16) && p.B % 8 == 0 &&
         p.num_blocks > 0 && p.tok_stride > 0 && p.blk_stride > 0 && aligned(p.cache, 16) &&
         p.tok_stride * ec % 16 == 0 && p.blk_stride * ec % 16 == 0 && p.blk_stride * ec < (int64_t{1} << 40) &&
         p.tok_stride * ec < (int64_t{1} << 40) && aligned(p.q, 16) && p.qr_stride % 8 == 0 && p.qt_stride % 8 == 0 &&
         p.qh_stride % 8 == 0 && p.qr_stride < (int64_t{1} << 38) && p.qt_stride < (int64_t{1} << 38) &&
         p.qh_stride < (int64_t{1} << 38);
}

int decode_tc(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream) {
  const int rows = p.q_len * p.H;
  p.groups = (rows + 63) / 64;
  p.rows_per_group = (rows + p.groups - 1) / p.groups;
  p.groups = (rows + p.rows_per_group - 1) / p.rows_per_group;
  p.units = std::max(1, sms / p.groups);
  p.slot_floats = (static_cast<int64_t>(p.rows_per_group) * (p.dv + 2) + 3) / 4 * 4;
  p.out_pairs = aligned(p.out, 4) && p.or_stride % 2 == 0 && p.ot_stride % 2 == 0 && p.oh_stride % 2 == 0;
  const bool fp8 = cache_dtype == PMG_FP8_E4M3;
  const int ec = elem_bytes(cache_dtype);
  const int box_rows = gcd(p.B, kDecodeTile);
  const CUtensorMapDataType type = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : q_dtype == PMG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const uint64_t page = static_cast<uint64_t>(p.B), blocks = static_cast<uint64_t>(p.num_blocks);
  const uint64_t row_stride = static_cast<uint64_t>(p.tok_stride) * ec, blk_stride = static_cast<uint64_t>(p.blk_stride) * ec;
  const uint32_t piece = 128 / ec, box = static_cast<uint32_t>(box_rows);  // elements of 128 bytes
  Maps maps;
  // the latent part as pieces of 128 bytes; the rotated part from the whole row (an e4m3 one is half a piece, and what
  // lies past the row reads as 0)
  int st = tensor_map<4>(&maps.latent, type, p.cache, {piece, page, kLatent / piece, blocks},
                         {row_stride, 128, blk_stride}, {piece, box, box_rows == kDecodeTile && !fp8 ? 2u : 1u, 1});
  if (st == PMG_OK)
    st = tensor_map<3>(&maps.rope, type, p.cache, {kEntry, page, blocks}, {row_stride, blk_stride}, {piece, box, 1});
  if (st != PMG_OK) return st;
  // queries of a 16-bit cache: whole boxes of heads and tokens, where a group is one
  const int rpg = p.rows_per_group, heads = std::min(p.H, rpg);
  p.q_tma = 0;
  maps.q = maps.rope;
  if (!fp8 && p.H % heads == 0 && rpg % heads == 0 && (p.qh_stride > 0 || p.H == 1) && (p.qt_stride > 0 || p.q_len == 1) &&
      (p.qr_stride > 0 || p.R == 1)) {
    // the stride of a dimension of one is not used; it has to be a valid one all the same
    const uint64_t s1 = p.H > 1 ? p.qh_stride * 2 : kEntry * 2, s2 = p.q_len > 1 ? p.qt_stride * 2 : kEntry * 2,
                   s3 = p.R > 1 ? p.qr_stride * 2 : kEntry * 2;
    st = tensor_map<4>(&maps.q, type, p.q,
                       {kEntry, static_cast<uint64_t>(p.H), static_cast<uint64_t>(p.q_len), static_cast<uint64_t>(p.R)},
                       {s1, s2, s3}, {64, static_cast<uint32_t>(heads), static_cast<uint32_t>(rpg / heads), 1});
    if (st != PMG_OK) return st;
    p.q_tma = heads;
  }
  if (q_dtype == PMG_BF16) return fp8 ? run<bf16, 2>(p, maps, box_rows, stream) : run<bf16, 1>(p, maps, box_rows, stream);
  return fp8 ? run<f16, 3>(p, maps, box_rows, stream) : run<f16, 1>(p, maps, box_rows, stream);
}

}  // namespace pmg_mla
