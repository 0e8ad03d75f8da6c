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
// entries side by side, the second from L2, and shared-memory reads of the
// operands come to the same size as the stream.
//
// Roles: warp 4 loads (one lane a TMA box: pages of any multiple of 8 tokens),
// warp 5 issues products, warps 0-3 do the softmax and the epilogue. An entry
// tile travels as four slots of 128 latent values and one of the rotated
// part, each freed as soon as its product is done, so loads run up to two tiles
// ahead of the softmax.
//
// The reference of a row follows its maximum only when a score passes it by
// 2^kSlack: weights then stay far inside the range of their type, sums are
// 32-bit, and the accumulators are rescaled (read, multiplied, written back)
// only in the first tiles of a request. All threads learn whether a tile needs
// that from one barrier with a vote, so the usual tile has no maximum over
// the lanes at all.
//
// An e4m3 cache is not widened. The 8-bit tensor core multiplies it as it is
// with queries and weights split in e4m3 parts of 4 significant bits each
// (x = x0 + x1 + ...): two parts hold a bf16 query's 8 bits, three an fp16
// query's 11, and two a weight to 2^-8 of its value, as bf16 would. With two
// parts that is as many instructions as the 16-bit products at half the bytes.
// Queries are first scaled by a power of two for each row that puts its
// largest value in [224, 448); what is lost is below a step of 2^-9, 2^-16.8 of
// the largest. Weights are taken at 2^6, where that step is 2^-15 of the
// reference weight.
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
  static constexpr int kP = kPiece * (kFp8 ? 2 : 1);
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
  static_assert(kTiles >= 2 && kBytes <= kSmemMax, "two tiles in flight");
};

struct Misc {
  uint64_t full[24], empty[24], rope_full[8], rope_empty[8];
  uint64_t s_full[2], s_free[2], p_full, pv_done, q_full;
  uint64_t mask[8];        // entries of a tile that exist, by tile & 7
  int64_t scratch[33], found[2];
  float ref[64], factor[64], alpha[64];  // of each row: reference, what a raw score is multiplied by, rescaling
  int32_t step[64];                      // of each row: which of the new tokens it belongs to
  uint32_t tmem;
  int32_t stop;
};
static_assert(sizeof(Misc) <= 2048, "Misc fits");

// Walks the requests of a share.
struct Items {
  const DecodeParams* p;
  int64_t at, end;
  int b;
  int64_t tile, tiles;
  int n;      // tiles of this share
  int len;    // keys of the request
  int full_len;
  __device__ Items(const DecodeParams& p_, const Share& s) : p(&p_), at(s.begin), end(s.end), b(s.item - 1) {
    tile = s.offset;
    tiles = n = len = full_len = 0;
    first_ = true;
  }
  __device__ bool next() {
    if (at >= end) return false;
    ++b;
    if (!first_) tile = 0;
    first_ = false;
    const DecodeLen l = decode_len(*p, b);
    len = l.use;
    full_len = l.full;
    tiles = len > 0 ? (len + kDecodeTile - 1) / kDecodeTile : 1;
    n = static_cast<int>(min(tiles - tile, end - at));
    at += n;
    return true;
  }
  __device__ int64_t piece() const { return at - n; }
 private:
  bool first_;
};

// The next e4m3 part of two values, packed low first; what is left of them
// stays in a and b. Rounded to 4 significant bits by Dekker's multiplication
// with 2^20 + 1, each step rounded by itself (no fused multiply-add).
__device__ __forceinline__ uint32_t part2(float& a, float& b) {
  const float ca = __fmul_rn(a, 1048577.0f), cb = __fmul_rn(b, 1048577.0f);
  const float ha = __fsub_rn(ca, __fsub_rn(ca, a)), hb = __fsub_rn(cb, __fsub_rn(cb, b));
  a -= ha;
  b -= hb;
  return __nv_cvt_float2_to_fp8x2(make_float2(ha, hb), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float half_of(uint32_t two, int i, bf16) { return __uint_as_float(i ? two & 0xffff0000u : two << 16); }
__device__ __forceinline__ float half_of(uint32_t two, int i, f16) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(i ? two >> 16 : two & 0xffff)));
}

// One row group's queries into shared memory, K-major. A warp takes every
// fourth row.
template <class TQ, int kParts, int N>
__device__ __forceinline__ void load_queries(const DecodeParams& p, int b, int g0, int n_rows, uint8_t* q_smem,
                                             Misc& mi, float factor) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kUnits = kEntry / 8;  // 16 bytes each
  constexpr int kBatch = 4;
#pragma unroll 1
  for (int r0 = warp; r0 < N; r0 += 4 * kBatch) {
    uint4 x[kBatch][3];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + 4 * i;
      if (r < N) {
        const int rr = g0 + r;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const TQ*>(p.q) + b * p.qr_stride +
                                                          (rr / p.H) * p.qt_stride + (rr % p.H) * p.qh_stride);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          x[i][k] = r < n_rows && lane + 32 * k < kUnits ? src[lane + 32 * k] : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + 4 * i;
      if (r >= N) continue;
      if constexpr (kParts == 1) {
        if (lane == 0) mi.factor[r] = factor;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const int u = lane + 32 * k;
          if (u < kUnits)
            *reinterpret_cast<uint4*>(q_smem + (u >> 3) * (N * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = x[i][k];
        }
      } else {
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const uint32_t w[4] = {x[i][k].x, x[i][k].y, x[i][k].z, x[i][k].w};
#pragma unroll
          for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(half_of(w[j >> 1], j & 1, TQ())));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^e * top in [224, 448): 224 = 1.75 * 2^7
        float scale = 1.0f;
        if (top > 0.0f && top < INFINITY) {
          int e = 0;
          const float m = frexpf(top, &e);  // top = m 2^e, m in [0.5, 1)
          scale = ldexpf(1.0f, (m < 0.875f ? 9 : 8) - e);
        }
        if (lane == 0) mi.factor[r] = factor / scale;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const int u = lane + 32 * k;  // 8 values: 8 bytes of each part
          if (u < kUnits) {
            const uint32_t w[4] = {x[i][k].x, x[i][k].y, x[i][k].z, x[i][k].w};
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = half_of(w[j >> 1], j & 1, TQ()) * scale;
            uint8_t* dst = q_smem + (u >> 4) * (N * 128) + r * 128 + ((((u & 15) >> 1) ^ (r & 7)) << 4) + (u & 1) * 8;
#pragma unroll
            for (int c = 0; c < kParts; ++c) {
              uint32_t y[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) y[j] = part2(v[2 * j], v[2 * j + 1]);
              *reinterpret_cast<uint2*>(dst + c * (5 * N * 128)) = make_uint2(y[0] | y[1] << 16, y[2] | y[3] << 16);
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
                     const __grid_constant__ CUtensorMap rope_map, int box_rows) {
  using L = Lay<kParts, N>;
  constexpr bool kFp8 = kParts > 1;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Misc& mi = *reinterpret_cast<Misc*>(smem + L::kMiscAt);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  constexpr int kColumns = N == 16 ? 128 : N == 32 ? 256 : 512;  // 2 S and 4 O accumulators of N columns

  // before the previous kernel's results are needed
  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(smem_u32(&mi.full[i]), 1);
      mbar_init(smem_u32(&mi.empty[i]), 1);
    }
    for (int i = 0; i < L::kRopeSlots; ++i) {
      mbar_init(smem_u32(&mi.rope_full[i]), 1);
      mbar_init(smem_u32(&mi.rope_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&mi.s_full[i]), 1);
      mbar_init(smem_u32(&mi.s_free[i]), 4);
    }
    mbar_init(smem_u32(&mi.p_full), 4);
    mbar_init(smem_u32(&mi.pv_done), 1);
    mbar_init(smem_u32(&mi.q_full), 4);
    mi.stop = 0;
    mbar_fence_init();
    tma_prefetch(&map);
    tma_prefetch(&rope_map);
  }
  if (warp == 5) tmem_alloc(smem_u32(&mi.tmem), kColumns);
  pdl_entry();

  const int unit = blockIdx.x / p.groups, group = blockIdx.x % p.groups;
  const Share share = find_share([&](int b) { return decode_tiles(p, b); }, p.R, unit, p.units, mi.scratch, mi.found);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = mi.tmem;
  volatile int* stop = &mi.stop;
  constexpr int kFmt = kFp8 ? 0 : (sizeof(TQ) == 2 && std::is_same<TQ, bf16>::value ? 1 : 0);
  constexpr uint32_t kIdescS = umma_idesc(kFmt, 0, 0, 64, N);
  constexpr uint32_t kIdescO = umma_idesc(kFmt, 1, 1, 128, N);

  if (warp == 4) {
    // ---- loads ----
    Items it(p, share);
    int slot = 0, phase = 0, rslot = 0, rphase = 0;
    int64_t t = 0;
    int bad = 0;
    bool alive = true;
    const uint32_t full = smem_u32(&mi.full[0]), empty = smem_u32(&mi.empty[0]);
    const uint32_t rope_full = smem_u32(&mi.rope_full[0]), rope_empty = smem_u32(&mi.rope_empty[0]);
    const int segs = kDecodeTile / box_rows;  // boxes of a tile along its rows: 1, 2, 4 or 8
    while (alive && it.next()) {
      if (lane == 0) bad |= decode_len(p, it.b).bad;
      if (it.len == 0) continue;
      const int32_t* table = p.bt + static_cast<int64_t>(it.b) * p.bt_stride;
      for (int i = 0; i < it.n && alive; ++i, ++t) {
        const int j0 = static_cast<int>(it.tile + i) * kDecodeTile;
        // lane s < segs looks up the page of box s
        const int j = j0 + lane * box_rows;
        const bool in = lane < segs && j < it.len;
        int id = -1, row = 0;
        if (in) {
          const uint32_t page = static_cast<uint32_t>(j) / static_cast<uint32_t>(p.B);
          id = table[page];
          row = j - static_cast<int>(page) * p.B;
        }
        const bool good = id >= 0 && id < p.num_blocks;
        if (in && !good) {
          bad |= PMG_FLAG_PHYS_BLOCK;
          id = static_cast<int>(p.num_blocks);  // outside: the box is filled with zeros
        }
        const uint32_t boxes = __ballot_sync(0xffffffffu, in), goods = __ballot_sync(0xffffffffu, in && good);
        const int n_boxes = __popc(boxes);
        if (lane == 0) {
          uint64_t m = 0;
          for (int s = 0; s < segs; ++s)
            if (goods >> s & 1) m |= (box_rows == 64 ? ~0ull : ((1ull << box_rows) - 1) << (s * box_rows));
          const int left = it.len - j0;
          if (left < 64) m &= (1ull << left) - 1;
          mi.mask[t & 7] = m;
        }
        const uint32_t bytes = static_cast<uint32_t>(n_boxes * box_rows * 128);
#pragma unroll 1
        for (int m = 0; m < 4; ++m) {
          alive = mbar_wait_warp(empty + 8 * slot, phase ^ 1, stop);
          if (!alive) break;
          const uint32_t dst = base + L::kSlotAt + slot * L::kSlot;
          if (elect_one()) mbar_expect(full + 8 * slot, bytes * L::kPieces);
          for (int s = 0; s < n_boxes; ++s) {
            const int sid = __shfl_sync(0xffffffffu, id, s), srow = __shfl_sync(0xffffffffu, row, s);
            // boxes of fewer rows than a slot has leave gaps between their pieces: a copy a piece
            if (box_rows == kDecodeTile) {
              if (elect_one()) tma_load_4d(dst, &map, full + 8 * slot, 0, srow, m * L::kPieces, sid);
            } else if (elect_one()) {
#pragma unroll
              for (int c = 0; c < L::kPieces; ++c)
                tma_load_4d(dst + c * L::kPiece + s * box_rows * 128, &map, full + 8 * slot, 0, srow, m * L::kPieces + c, sid);
            }
          }
          if (++slot == L::kSlots) { slot = 0; phase ^= 1; }
        }
        if (!alive) break;
        alive = mbar_wait_warp(rope_empty + 8 * rslot, rphase ^ 1, stop);
        if (!alive) break;
        if (elect_one()) mbar_expect(rope_full + 8 * rslot, bytes);
        for (int s = 0; s < n_boxes; ++s) {
          const int sid = __shfl_sync(0xffffffffu, id, s), srow = __shfl_sync(0xffffffffu, row, s);
          if (elect_one())
            tma_load_3d(base + L::kRopeAt + rslot * L::kPiece + s * box_rows * 128, &rope_map, rope_full + 8 * rslot, kLatent,
                        srow, sid);
        }
        if (++rslot == L::kRopeSlots) { rslot = 0; rphase ^= 1; }
      }
    }
    set_flag(p.err, bad);
    // copies that nobody will use any more still have to land before the CTA ends
    if (!alive && lane == 0) {
      int never = 0;
      for (int i = 0; i < L::kSlots; ++i) mbar_wait(smem_u32(&mi.full[i]), (i < slot ? phase : phase ^ 1), &never);
      for (int i = 0; i < L::kRopeSlots; ++i)
        mbar_wait(smem_u32(&mi.rope_full[i]), (i < rslot ? rphase : rphase ^ 1), &never);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ---- products ----
    Items qi(p, share), vi(p, share);
    auto advance = [](Items& it) {
      bool more = it.next();
      while (more && it.len == 0) more = it.next();
      return more;
    };
    const uint32_t full = smem_u32(&mi.full[0]), empty = smem_u32(&mi.empty[0]);
    const uint32_t rope_full = smem_u32(&mi.rope_full[0]), rope_empty = smem_u32(&mi.rope_empty[0]);
    const uint32_t s_full = smem_u32(&mi.s_full[0]), s_free = smem_u32(&mi.s_free[0]);
    bool q_more = advance(qi), v_more = advance(vi);
    int q_tile = 0, q_part = 0, v_tile = 0;     // within the items
    int q_item = 0;                             // items begun, for the queries' barrier
    uint32_t qt = 0, vt = 0;                    // tiles issued
    int qslot = 0, qphase = 0, rslot = 0, rphase = 0, vslot = 0;
    uint64_t t0 = 0;
    int idle = 0;
    bool alive = true;
    // whichever product has its operands: O of a tile once its weights are there, parts of S up to two tiles ahead
    while (alive && (q_more || v_more)) {
      bool progress = false;
      if (v_more && vt != qt && mbar_test_warp(smem_u32(&mi.p_full), vt & 1)) {
        tmem_fence_after();
        const bool first = v_tile == 0;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (elect_one()) {
            const uint64_t va = umma_desc(base + L::kSlotAt + vslot * L::kSlot, L::kPiece, 1024);
            const uint64_t pa = umma_desc(base + L::kPAt, L::kPiece, 1024);
            const uint32_t d = tmem + (2 + m) * N;
#pragma unroll
            for (int k = 0; k < (kFp8 ? 2 : 4); ++k) {
              const uint32_t step = k * (kFp8 ? 32 : 16) * 8;  // rows of 128 bytes, in units of 16
              umma_ss<kFp8>(d, va + step, pa + step, kIdescO, !first || k > 0);
              if constexpr (kFp8) umma_ss<kFp8>(d, va + step, pa + step + L::kPiece / 16, kIdescO, true);
            }
            umma_commit(empty + 8 * vslot);
            if (m == 3) umma_commit(smem_u32(&mi.pv_done));
          }
          __syncwarp();
          if (++vslot == L::kSlots) vslot = 0;
        }
        ++vt;
        if (++v_tile == vi.n) {
          v_tile = 0;
          v_more = advance(vi);
        }
        progress = true;
      }
      if (q_more && qt - vt < 2) {
        const uint32_t buf = qt & 1;
        bool ready = true;
        if (q_part == 0) {
          if (qt >= 2) ready = mbar_test_warp(s_free + 8 * buf, ((qt >> 1) + 1) & 1);
          if (ready && q_tile == 0) ready = mbar_test_warp(smem_u32(&mi.q_full), q_item & 1);
        }
        if (ready)
          ready = q_part < 4 ? mbar_test_warp(full + 8 * qslot, qphase) : mbar_test_warp(rope_full + 8 * rslot, rphase);
        if (ready) {
          tmem_fence_after();
          const uint32_t d = tmem + buf * N;
          if (q_part < 4) {
            if (elect_one()) {
#pragma unroll
              for (int c = 0; c < L::kPieces; ++c) {
                const uint64_t ka = umma_desc(base + L::kSlotAt + qslot * L::kSlot + c * L::kPiece, 16, 1024);
                const uint64_t qa = umma_desc(base + L::kQAt + (q_part * L::kPieces + c) * (N * 128), 16, 1024);
#pragma unroll
                for (int k = 0; k < 4; ++k)  // 32 bytes of K each
#pragma unroll
                  for (int x = 0; x < kParts; ++x)
                    umma_ss<kFp8>(d, ka + 2 * k, qa + 2 * k + x * (5 * N * 8), kIdescS,
                                  q_part > 0 || c > 0 || k > 0 || x > 0);
              }
            }
            __syncwarp();
            ++q_part;
            if (++qslot == L::kSlots) { qslot = 0; qphase ^= 1; }
          } else {
            if (elect_one()) {
              const uint64_t ka = umma_desc(base + L::kRopeAt + rslot * L::kPiece, 16, 1024);
              const uint64_t qa = umma_desc(base + L::kQAt + 4 * L::kPieces * (N * 128), 16, 1024);
#pragma unroll
              for (int k = 0; k < (kFp8 ? 2 : 4); ++k)
#pragma unroll
                for (int x = 0; x < kParts; ++x)
                  umma_ss<kFp8>(d, ka + 2 * k, qa + 2 * k + x * (5 * N * 8), kIdescS, true);
              umma_commit(rope_empty + 8 * rslot);
              umma_commit(s_full + 8 * buf);
            }
            __syncwarp();
            if (++rslot == L::kRopeSlots) { rslot = 0; rphase ^= 1; }
            q_part = 0;
            ++qt;
            if (q_tile == 0) ++q_item;
            if (++q_tile == qi.n) {
              q_tile = 0;
              q_more = advance(qi);
            }
          }
          progress = true;
        }
      }
      if (progress) {
        idle = 0;
        t0 = 0;
      } else if (++idle >= 256) {
        idle = 0;
        const uint64_t now = now_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitNs) *stop = 1;
        alive = __all_sync(0xffffffffu, *stop == 0) != 0;
      }
    }
    if (!alive && vt > 0) {  // what was issued ends before the CTA does
      int never = 0;
      mbar_wait(smem_u32(&mi.pv_done), static_cast<int>((vt - 1) & 1), &never);
    }
    __syncwarp();
  } else {
    // ---- softmax and epilogue ----
    Items it(p, share);
    const int rows = p.q_len * p.H;
    const int g0 = group * p.rows_per_group;
    const int n_rows = min(p.rows_per_group, rows - g0);
    const float kv_scale = kFp8 && p.scale != nullptr ? *p.scale : 1.0f;
    const float factor = p.sm_scale * kLog2e * kv_scale;
    constexpr float kSlack = kFp8 ? 2.5f : 8.0f;     // weights up to 2^(kBase + kSlack) <= 448
    constexpr float kBase = kFp8 ? 6.0f : 0.0f;
    const int token = warp * 16 + (lane & 15);       // M = 64: 16 rows in each quarter of the lanes
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    JoinNote note{-1, 0, 0, 0};
    int64_t t = 0;
    bool alive = true;
    bool more = it.next();
    // queries of the first request that has any keys
    auto queries = [&](const Items& x) {
      load_queries<TQ, kParts, N>(p, x.b, g0, n_rows, smem + L::kQAt, mi, factor);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&mi.q_full));
    };
    if (tid < N) mi.step[tid] = (g0 + tid) / p.H;
    bool loaded = false;  // whether the queries of `it` are in place
    while (alive && more) {
      if (it.len > 0 && !loaded) queries(it);
      Items ahead = it;
      const bool more_ahead = ahead.next();
      float l[N];
#pragma unroll
      for (int h = 0; h < N; ++h) l[h] = 0.0f;
      const int n = it.len > 0 ? it.n : 0;
      named_sync<kSoft>(1);  // everybody is done with the last request's references
      if (tid < N) mi.ref[tid] = -INFINITY;
      named_sync<kSoft>(1);  // and the queries' factors are there
      for (int i = 0; i < n; ++i, ++t) {
        const int buf = static_cast<int>(t & 1);
        if (!mbar_wait(smem_u32(&mi.s_full[buf]), static_cast<int>(t >> 1) & 1, stop)) alive = false;
        const int64_t j0 = (it.tile + i) * kDecodeTile;
        // the loading warp's note of the tile is ordered by its first slot's barrier
        if (alive && !mbar_wait(smem_u32(&mi.full[static_cast<int>((4 * t) % L::kSlots)]),
                                static_cast<int>((4 * t) / L::kSlots) & 1, stop))
          alive = false;
        if (named_any<kSoft>(2, !alive)) {
          alive = false;
          break;
        }
        tmem_fence_after();
        const uint64_t mask = mi.mask[t & 7];
        __syncwarp();
        uint32_t raw_s[N];
        if constexpr (N == 16) tmem_ld16(tmem + buf * N + lanes, raw_s);
        else if constexpr (N == 32) tmem_ld32(tmem + buf * N + lanes, raw_s);
        else {
          tmem_ld32(tmem + buf * N + lanes, raw_s);
          tmem_ld32(tmem + buf * N + 32 + lanes, raw_s + 32);
        }
        tmem_wait_ld();
        tmem_pin<N>(raw_s);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&mi.s_free[buf]));
        float s[N];
        const bool there = lane < 16 && (mask >> token & 1) != 0;
        const int j = static_cast<int>(j0) + token;
        const bool edge = j0 + kDecodeTile > it.full_len - p.q_len + 1;  // some row does not see the whole tile
        float over = -INFINITY;
#pragma unroll
        for (int h = 0; h < N; h += 4) {
          const float4 f = kFp8 ? *reinterpret_cast<const float4*>(&mi.factor[h]) : make_float4(factor, factor, factor, factor);
          const float4 r = *reinterpret_cast<const float4*>(&mi.ref[h]);
          s[h] = there ? __uint_as_float(raw_s[h]) * f.x : -INFINITY;
          s[h + 1] = there ? __uint_as_float(raw_s[h + 1]) * f.y : -INFINITY;
          s[h + 2] = there ? __uint_as_float(raw_s[h + 2]) * f.z : -INFINITY;
          s[h + 3] = there ? __uint_as_float(raw_s[h + 3]) * f.w : -INFINITY;
          if (!edge) {
            over = fmaxf(over, fmaxf(fmaxf(s[h] - r.x, s[h + 1] - r.y), fmaxf(s[h + 2] - r.z, s[h + 3] - r.w)));
          }
        }
        if (edge) {
#pragma unroll
          for (int h = 0; h < N; ++h) {
            if (j >= it.full_len - p.q_len + 1 + mi.step[h]) s[h] = -INFINITY;
            // (-inf) - (-inf) is no excess
            if (s[h] != -INFINITY) over = fmaxf(over, s[h] - mi.ref[h]);
          }
        } else if (!there) {
          over = -INFINITY;
        }
        const bool raise = named_any<kSoft>(2, over > kBase + kSlack);
        if (raise) {
          // maximum of every row over the tile's entries
          float* part = reinterpret_cast<float*>(smem + L::kPAt);  // free once the last tile's product is done
          if (t > 0 && !mbar_wait(smem_u32(&mi.pv_done), static_cast<int>(t - 1) & 1, stop)) alive = false;
          tmem_fence_after();
#pragma unroll
          for (int h = 0; h < N; ++h) {
            float top = s[h];
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (lane == 0) part[warp * N + h] = top;
          }
          named_sync<kSoft>(1);
          if (tid < N) {
            const float top = fmaxf(fmaxf(part[tid], part[N + tid]), fmaxf(part[2 * N + tid], part[3 * N + tid]));
            const float old = mi.ref[tid];
            float next = old, a = 1.0f;
            if (top - kBase > old) {  // where the tile raises it at all
              next = top - kBase;
              a = old == -INFINITY ? 0.0f : ex2(old - next);
            }
            mi.ref[tid] = next;
            mi.alpha[tid] = a;
          }
          named_sync<kSoft>(1);
#pragma unroll
          for (int h = 0; h < N; ++h) l[h] *= mi.alpha[h];
          __syncwarp();
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
        }
        // weights
#pragma unroll
        for (int h = 0; h < N; h += 4) {
          const float4 r = *reinterpret_cast<const float4*>(&mi.ref[h]);
          const float rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[h + k] = s[h + k] == -INFINITY ? 0.0f : ex2(s[h + k] - rr[k]);
            l[h + k] += s[h + k];
          }
        }
        // the last tile's product has read its weights
        if (t > 0 && !mbar_wait(smem_u32(&mi.pv_done), static_cast<int>(t - 1) & 1, stop)) alive = false;
        // values past the end of the request may be anything: their weights are 0, so must they be
        const int64_t valid = it.len - j0;
        if (valid < kDecodeTile) {
          const int first = static_cast<int>(valid);
          for (int m = 0; m < 4; ++m) {
            uint8_t* at = smem + L::kSlotAt + static_cast<int>((4 * t + m) % L::kSlots) * L::kSlot;
            for (int x = tid; x < (kDecodeTile - first) * 8 * L::kPieces; x += kSoft) {
              const int piece = x / ((kDecodeTile - first) * 8), y = x % ((kDecodeTile - first) * 8);
              *reinterpret_cast<uint4*>(at + piece * L::kPiece + (first + y / 8) * 128 + (y % 8) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
          }
        }
        if (raise) named_sync<kSoft>(1);  // the maxima's place is where the weights go
        if (lane < 16) {
          uint8_t* row = smem + L::kPAt + token * 128;
          if constexpr (!kFp8) {
#pragma unroll
            for (int u = 0; u < N / 8; ++u)
              *reinterpret_cast<uint4*>(row + ((u ^ (token & 7)) << 4)) =
                  make_uint4(pack2<TQ>(s[8 * u], s[8 * u + 1]), pack2<TQ>(s[8 * u + 2], s[8 * u + 3]),
                             pack2<TQ>(s[8 * u + 4], s[8 * u + 5]), pack2<TQ>(s[8 * u + 6], s[8 * u + 7]));
          } else {
#pragma unroll
            for (int u = 0; u < N / 16; ++u) {
              const int at = (u ^ (token & 7)) << 4;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = part2(s[16 * u + 2 * k], s[16 * u + 2 * k + 1]);
                *reinterpret_cast<uint4*>(row + c * L::kPiece + at) =
                    make_uint4(y[0] | y[1] << 16, y[2] | y[3] << 16, y[4] | y[5] << 16, y[6] | y[7] << 16);
              }
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&mi.p_full));
      }
      if (!alive) break;

      // sums of every row over the lanes, then over the warps
      const bool whole = it.tile == 0 && it.n == it.tiles;
      float* sums = mi.alpha;
      named_sync<kSoft>(1);
      if (tid < N) sums[tid] = 0.0f;
      named_sync<kSoft>(1);
#pragma unroll
      for (int h = 0; h < N; ++h) {
        float x = l[h];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        l[h] = x;
      }
      for (int w = 0; w < 4; ++w) {  // in a fixed order
        if (warp == w && lane == 0) {
#pragma unroll
          for (int h = 0; h < N; ++h) sums[h] += l[h];
        }
        named_sync<kSoft>(1);
      }
      // the next request's queries, while the last product runs
      loaded = false;
      float my_ref = 0.0f, my_sum = 0.0f;
      if (tid < N) {
        my_ref = mi.ref[tid];
        my_sum = sums[tid];
      }
      if (more_ahead && ahead.len > 0) {
        queries(ahead);
        loaded = true;
      }
      float* slot = p.ws.slots + (static_cast<int64_t>(blockIdx.x) * 2 + (it.tile == 0 ? 1 : 0)) * p.slot_floats;
      if (!whole && it.tile == 0 && tid == 0) {
        note.item = it.b;
        note.parts = unit_of(it.piece() + it.tiles - 1, share.total, share.units) - unit + 1;
      }
      if (tid < n_rows) {
        const int rr = g0 + tid;
        if (whole) {
          if (p.lse != nullptr)
            p.lse[static_cast<int64_t>(it.b) * rows + rr] =
                my_sum > 0.0f ? (my_ref + log2f(my_sum)) * kLn2 : -INFINITY;
        } else {
          float* ml = slot + p.rows_per_group * kLatent + 2 * tid;
          ml[0] = my_ref;
          ml[1] = my_sum;
        }
      }
      if (n > 0) {
        if (!mbar_wait(smem_u32(&mi.pv_done), static_cast<int>(t - 1) & 1, stop)) alive = false;
        if (named_any<kSoft>(2, !alive)) {
          alive = false;
          break;
        }
        tmem_fence_after();
      }
      __syncwarp();
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        const int d = m * 128 + warp * 32 + lane;
#pragma unroll 1
        for (int h0 = 0; h0 < N; h0 += 16) {
          uint32_t o[16];
          if (n > 0) {
            tmem_ld16(tmem + (2 + m) * N + h0 + lanes, o);
            tmem_wait_ld();
            tmem_pin<16>(o);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0;
          }
          if (whole) {
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              // even lanes write row k, odd lanes row k + 1, two neighbours' values each
              const float la = sums[h0 + k], lb = sums[h0 + k + 1];
              const float a = __uint_as_float(o[k]) * (la > 0.0f ? kv_scale / la : 0.0f);
              const float b = __uint_as_float(o[k + 1]) * (lb > 0.0f ? kv_scale / lb : 0.0f);
              auto out_at = [&](int h) {
                const int rr = g0 + h;
                return static_cast<TQ*>(p.out) + it.b * p.or_stride + (rr / p.H) * p.ot_stride + (rr % p.H) * p.oh_stride;
              };
              if (p.out_pairs) {
                const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
                const int h = h0 + k + (lane & 1);
                if (h < n_rows)
                  *reinterpret_cast<uint32_t*>(out_at(h) + (d & ~1)) = lane & 1 ? pack2<TQ>(other, b) : pack2<TQ>(a, other);
              } else {
                if (h0 + k < n_rows) out_at(h0 + k)[d] = from_f<TQ>(a);
                if (h0 + k + 1 < n_rows) out_at(h0 + k + 1)[d] = from_f<TQ>(b);
              }
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (h0 + k < n_rows) slot[(h0 + k) * kLatent + d] = __uint_as_float(o[k]) * kv_scale;
          }
        }
      }
      tmem_fence_before();
      it = ahead;
      more = more_ahead;
    }
    if (tid == 0 && p.units > 1) p.ws.notes[blockIdx.x] = note;
    if (tid == 0 && *stop != 0) set_flag(p.err, PMG_FLAG_TIMEOUT);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 5) tmem_free(tmem, kColumns);
}

struct Maps {
  CUtensorMap latent, rope;
};

template <class TQ, int kParts, int N>
int run(const DecodeParams& p, const Maps& maps, int box_rows, void* stream) {
  auto k = decode_tc_kernel<TQ, kParts, N>;
  constexpr int kBytes = Lay<kParts, N>::kBytes;
  const int st = allow_smem(reinterpret_cast<const void*>(k), kBytes);
  if (st != PMG_OK) return st;
  return launch(k, dim3(static_cast<unsigned>(p.units) * p.groups), kThreads, kBytes, stream, p, maps.latent, maps.rope,
                box_rows);
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
         p.qh_stride % 8 == 0;
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
  if (q_dtype == PMG_BF16) return fp8 ? run<bf16, 2>(p, maps, box_rows, stream) : run<bf16, 1>(p, maps, box_rows, stream);
  return fp8 ? run<f16, 3>(p, maps, box_rows, stream) : run<f16, 1>(p, maps, box_rows, stream);
}

}  // namespace pmg_mla
