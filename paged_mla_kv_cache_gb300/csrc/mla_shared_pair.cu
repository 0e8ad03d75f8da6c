// Absorbed latent attention of many rows over a prefix that they share, on pairs
// of SMs: entries of 512 latent and 64 rotated 16-bit values.
//
// Mathematics. A pair of CTAs has 128 query rows, 64 each, and passes tiles of
// 64 entries E: S = Q E^T (128 x 64), P = 2^(S - ref), O += P E[:, :512] (128 x
// 512), unnormalised; references, sums and the parts of split prefixes are as in
// mla_decode_tc_kernel.cuh, the result is the state of a prefix pass
// (mla_decode.cuh).
//
// Bound: the tensor core, from a few hundred rows on. One CTA's products of 64
// rows or entries run at half its rate (2028 multiply-adds a clock measured, of
// 4096) and its 128 x 64 ones at two thirds (2713, bound by the operands' reads);
// the products of a pair, of 128 rows x 64 at 2588 and of 128 x 256 at 4074, bring
// a tile of 64 entries and 128 rows to 1425 clocks, 77% of the full rate. A pair
// splits the second operand of a product: each CTA holds 32 of the tile's
// entries whole, for S, and of all 64 its half of the latent values, for O. Both
// lie at the same place of either CTA, as the joint products need, so half of
// the latent values is there twice; with two tiles in flight that fills shared
// memory (74 KB of queries, 2 x 70 KB, 2 x 8 KB of weights). Measured: 360 us for
// 64 requests of 128 heads over 32768 entries, 1.63 PFLOP/s; all passes of that
// call take 425, with tiles of 64 rows on single SMs (mla_decode_tc_kernel.cuh) 846. Accumulators lie two to
// a row of tensor memory: lanes 0-63 have the entries or values of the first
// CTA's half, lanes 64-127 those of the second's, so two threads share a row.
//
// Roles in each CTA: warps 4 and 7 load, entries for S and for O (as one warp, the
// entries for S waited until the place for O before them was free), warp 5 of the
// pair's first CTA issues all products, warps 5 and 6 of the second tell it what has arrived there, warps 0-3
// do the softmax and the epilogue of their CTA's rows. All waits are bounded; a CTA
// whose wait ran out stops its pair, and the rows of all work that either did not
// finish before become NaN.
#include <algorithm>
#include <type_traits>

#include "mla_decode.cuh"
#include "mla_decode_tc.cuh"
#include "mla_queries.cuh"
#include "mla_sm103.cuh"

namespace pmg_mla {
namespace {

constexpr int kThreads = 256;
constexpr int kSoft = 128;
constexpr int kLatent = 512;               // and 64 rotated ones: kEntry
constexpr int kRows = 64;                  // of a CTA
constexpr int kKeys = kDecodeTile / 2;     // of a tile that a CTA holds whole
constexpr int kKPiece = kKeys * 128;       // 128 bytes of them
constexpr int kQPiece = kRows * 128;
constexpr int kMisc = 2560;

// Shared memory, by the parts of a query: 1 for a 16-bit cache, for an e4m3 one 2 (bf16) or 3 (fp16).
template <int kParts>
struct Lay {
  static constexpr bool kFp8 = kParts > 1;
  static constexpr int kPieces = kFp8 ? 4 : 8;     // of the latent values
  static constexpr int kWeights = kFp8 ? 3 : 1;    // parts of a weight
  static constexpr int kQPart = (kPieces + 1) * kQPiece;
  static constexpr int kK = (kPieces + 1) * kKPiece, kV = kPieces * kKPiece;  // (V: both halves' half of the values)
  static constexpr int kStage = kK + kV;
  // Weights of two tiles: 16-bit ones one behind the other, of e5m2 parts 64 bytes of a row each.
  static constexpr int kPNext = kFp8 ? 64 : kRows * 128, kPPart = kRows * 128;
  static constexpr int kPAt = kQPart * kParts;
  static constexpr int kStageAt = kPAt + (kFp8 ? kWeights : 2) * kPPart;
  static constexpr int kMiscAt = kStageAt + 2 * kStage;
  static constexpr int kBytes = kMiscAt + kMisc + 512;
  static_assert(kBytes <= 232448, "fits");
};
constexpr int kColumns = 512, kSAt = 256;  // O: 256 columns, then two S of 32

struct Misc {
  uint64_t k_full[2], v_full[2], k_peer[2], v_peer[2], k_empty[2], v_empty[2], s_full[2], s_free[2], m_full[4], p_full[2], q_full, q_empty, end;
  uint64_t mask[4];    // entries of a tile that exist, by tile & 3
  float factor[kRows]; // e4m3: what a row's raw scores are multiplied by
  union {
    struct {
      int64_t scratch[33], found[2];
    };
    float tops[kSoft];
    float sums[kSoft];
  };
  uint32_t tmem;
  int32_t stop, never;
  int32_t bad_from;    // the first item that a timeout of either CTA touched
};
static_assert(sizeof(Misc) <= kMisc, "fits");

// ---- pairs of CTAs ----------------------------------------------------------------

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// where `addr` of this CTA is in CTA `rank` of the pair
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_arrive(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// mbar_wait for what either CTA arrives at; a wait that runs out stops both (stop: this CTA's word, peer: the other's).
__device__ __forceinline__ void pair_wait(uint32_t bar, uint32_t parity, uint32_t stop, uint32_t peer) {
  asm volatile(
      "{\n\t"
      ".reg .pred p;\n\t"
      ".reg .b32 s;\n\t"
      ".reg .b64 t0, t1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
      "@p bra DONE%=;\n\t"
      "mov.u64 t0, %%globaltimer;\n\t"
      "AGAIN%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
      "@p bra DONE%=;\n\t"
      "ld.volatile.shared.b32 s, [%2];\n\t"
      "setp.ne.b32 p, s, 0;\n\t"
      "@p bra DONE%=;\n\t"
      "mov.u64 t1, %%globaltimer;\n\t"
      "sub.u64 t1, t1, t0;\n\t"
      "setp.lt.u64 p, t1, 2000000000;\n\t"
      "@p bra AGAIN%=;\n\t"
      "mov.b32 s, 1;\n\t"
      "st.volatile.shared.b32 [%2], s;\n\t"
      "st.shared::cluster.b32 [%3], s;\n\t"
      "DONE%=:\n\t"
      "}" ::"r"(bar),
      "r"(parity), "r"(stop), "r"(peer)
      : "memory");
}

// All products of the kernel are a pair's.
template <bool kFp8>
__device__ __forceinline__ void pair_umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  if constexpr (kFp8) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
  }
}
// arrives at the same barrier of both CTAs when every product issued so far by this thread is done
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// A whole sector: lanes write rows of their own.
__device__ __forceinline__ void store32(float* to, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

template <class T, int kParts>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    shared_pair_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap map,
                       const __grid_constant__ CUtensorMap rope_map, const __grid_constant__ CUtensorMap q_map, int box_rows) {
  using L = Lay<kParts>;
  constexpr bool kFp8 = L::kFp8;
  constexpr int kK = L::kK, kStage = L::kStage, kStageAt = L::kStageAt, kPieces = L::kPieces;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc& mi = *reinterpret_cast<Misc*>(smem + L::kMiscAt);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = cta_rank();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      for (uint64_t* b : {&mi.k_full[i], &mi.v_full[i], &mi.k_peer[i], &mi.v_peer[i], &mi.k_empty[i], &mi.v_empty[i], &mi.s_full[i]})
        mbar_init(smem_u32(b), 1);
      mbar_init(smem_u32(&mi.s_free[i]), 8);
      mbar_init(smem_u32(&mi.p_full[i]), 8);
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&mi.m_full[i]), 1);
    mbar_init(smem_u32(&mi.q_full), kFp8 ? kSoft / 32 : 1);
    mbar_init(smem_u32(&mi.q_empty), 1);
    mbar_init(smem_u32(&mi.end), 1);
    mi.stop = mi.never = 0;
    mi.bad_from = INT32_MAX;
    mbar_fence_init();
    tma_prefetch(&map);
    tma_prefetch(&rope_map);
    if (!kFp8) tma_prefetch(&q_map);
    if (base & 1023) mi.stop = 1;  // (the swizzled tiles' alignment; the attribute sees to it)
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&mi.tmem)), "n"(kColumns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  const int rpc = p.rows_per_group / 2;  // rows of a CTA
  // rows of queries that no copy fills: 0
  for (int i = tid; i < (kFp8 ? 0 : 9 * (kRows - rpc) * 8); i += kThreads) {
    const int c = i / ((kRows - rpc) * 8), y = i % ((kRows - rpc) * 8);
    *reinterpret_cast<uint4*>(smem + c * kQPiece + rpc * 128 + y * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_async_smem();
  pass_entry<true>(p);
  const int unit = blockIdx.x >> 1;
  const Share share = find_share([&](int b) { return prefix_pieces<kItemCost>(p, b); }, p.R, unit, p.units, mi.scratch, mi.found);
  if (blockIdx.x == 0) note_covered(p, tid, kThreads, *reinterpret_cast<int32_t*>(mi.scratch));
  tmem_fence_before();
  __syncthreads();
  pair_sync();
  tmem_fence_after();
  const uint32_t tmem = mi.tmem, stop = smem_u32(&mi.stop), peer = at_rank(stop, rank ^ 1);
  constexpr int kFmt = !kFp8 && std::is_same<T, bf16>::value ? 1 : 0;
  constexpr uint32_t kIdescS = umma_idesc(kFmt, kFmt, 0, 0, 128, kDecodeTile);
  constexpr uint32_t kIdescO = umma_idesc(kFp8 ? 1 : kFmt, kFmt, 0, 1, 128, 256);  // e5m2 weights of e4m3 values
  const uint32_t k_full = smem_u32(&mi.k_full[0]), v_full = smem_u32(&mi.v_full[0]);
  const uint32_t k_empty = smem_u32(&mi.k_empty[0]), v_empty = smem_u32(&mi.v_empty[0]);
  PrefixItems<kItemCost> it(p, share);
  auto wait = [&](uint32_t bar, uint32_t parity) { pair_wait(bar, parity, stop, peer); };

  if (warp == 4 || warp == 7) {
    // ---- loads ----
    const bool for_s = warp == 4;
    uint32_t t = 0, items = 0;
    int bad = 0;
    bool alive = true;
    const int segs = kDecodeTile / box_rows, half = segs / 2;  // boxes of a tile along its rows: 2, 4 or 8; of a CTA's entries
    const int mine = static_cast<int>(rank) * half;            // the first of them
    while (alive && it.next()) {
      if (it.len == 0) continue;
      const int32_t* table = p.bt + static_cast<int64_t>(it.b) * p.bt_stride;
      const uint32_t len = static_cast<uint32_t>(it.len);
      // lane s < segs looks up the page of box s, one tile ahead of its use (places have no sign: boxes past the end may lie
      // past INT32_MAX)
      auto page_of = [&](uint32_t j) { return lane < segs && j < len ? table[j / static_cast<uint32_t>(p.B)] : -1; };
      uint32_t j = static_cast<uint32_t>(it.tile * kDecodeTile) + lane * box_rows;
      int next_id = page_of(j);
#pragma unroll 1
      for (int i = 0; i < it.n; ++i, ++t, j += kDecodeTile) {
        const uint32_t stage = t & 1, parity = (t >> 1 & 1) ^ 1;
        const bool in = lane < segs && j < len;
        int id = next_id;
        const int row = static_cast<int>(j % static_cast<uint32_t>(p.B));
        next_id = i + 1 < it.n ? page_of(j + kDecodeTile) : -1;
        const bool good = id >= 0 && id < p.num_blocks;
        if (in && !good) {
          bad |= PMG_FLAG_PHYS_BLOCK;
          id = static_cast<int>(p.num_blocks);  // outside: the box is filled with zeros
        }
        const uint32_t goods = __ballot_sync(0xffffffffu, in && good);
        const int n_boxes = __popc(__ballot_sync(0xffffffffu, in)), n_mine = max(0, min(half, n_boxes - mine));
        if (stopped(stop)) {
          alive = false;
          break;
        }
        const uint32_t k_at = base + kStageAt + stage * kStage, v_at = k_at + kK;
        if (for_s) {
          uint64_t mask = 0;  // entries that exist
          for (int s = 0; s < segs; ++s)
            if (goods >> s & 1) mask |= ((1ull << box_rows) - 1) << (s * box_rows);
          const int left = it.len - (it.tile + i) * kDecodeTile;
          if (left < 64) mask &= (1ull << left) - 1;
          if (!kFp8 && i == 0) {  // the row tile's queries, once the products with the ones before are done
            if (items > 0) wait(smem_u32(&mi.q_empty), (items - 1) & 1);
            ++items;
            if (elect_one()) {
              const int r0 = it.row0 + static_cast<int>(rank) * rpc, token = r0 / p.H;
              const uint32_t bar = smem_u32(&mi.q_full);
              mbar_expect(bar, static_cast<uint32_t>(rpc) * kEntry * 2);
#pragma unroll 1
              for (int c = 0; c < 9; ++c)
                tma_load_4d(base + c * kQPiece, &q_map, bar, 64 * c, r0 % p.H, token % p.q_tma, token / p.q_tma);
            }
            __syncwarp();
          }
          wait(k_empty + 8 * stage, parity);
          if (elect_one()) {
            // The mask has barriers of its own, four of them: those of the entries may be a phase ahead of the softmax warps,
            // which then wait in vain. A tile's entries are loaded when the scores two tiles before are done, and those when
            // the softmax warps had read the scores, and the mask, of another two before.
            mi.mask[t & 3] = mask;  // by the lane that arrives
            mbar_arrive(smem_u32(&mi.m_full[t & 3]));
            mbar_expect(k_full + 8 * stage, static_cast<uint32_t>(n_mine * box_rows) * ((kPieces + 1) * 128));
          }
          __syncwarp();
#pragma unroll 1
          for (int s = 0; s < n_mine; ++s) {
            const int sid = __shfl_sync(0xffffffffu, id, mine + s), srow = __shfl_sync(0xffffffffu, row, mine + s);
            if (elect_one()) {
              const uint32_t dst = k_at + s * box_rows * 128, bar = k_full + 8 * stage;
              if (box_rows == kKeys) {
                tma_load_4d(dst, &map, bar, 0, srow, 0, sid);
                tma_load_4d(dst + kPieces / 2 * kKPiece, &map, bar, 0, srow, kPieces / 2, sid);
              } else {
#pragma unroll 1
                for (int c = 0; c < kPieces; ++c) tma_load_4d(dst + c * kKPiece, &map, bar, 0, srow, c, sid);
              }
              tma_load_3d(dst + kPieces * kKPiece, &rope_map, bar, kLatent, srow, sid);
            }
            __syncwarp();
          }
        } else {
          wait(v_empty + 8 * stage, parity);
          if (elect_one()) mbar_expect(v_full + 8 * stage, static_cast<uint32_t>(n_boxes * box_rows) * (kPieces / 2 * 128));
          __syncwarp();
#pragma unroll 1
          for (int s = 0; s < n_boxes; ++s) {
            const int sid = __shfl_sync(0xffffffffu, id, s), srow = __shfl_sync(0xffffffffu, row, s);
            if (elect_one()) {
              const uint32_t dst = v_at + (s / half) * (kPieces / 2 * kKPiece) + (s % half) * box_rows * 128, bar = v_full + 8 * stage;
              const int c0 = static_cast<int>(rank) * (kPieces / 2);
              if (box_rows == kKeys) {
                tma_load_4d(dst, &map, bar, 0, srow, c0, sid);
              } else {
#pragma unroll 1
                for (int c = 0; c < kPieces / 2; ++c) tma_load_4d(dst + c * kKPiece, &map, bar, 0, srow, c0 + c, sid);
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (rank == 0 && for_s) set_flag(p.err, bad);
    // after a timeout, copies in flight land before the CTA ends (`never` is not set: these waits run on)
    if (!alive) {
      const uint32_t never = smem_u32(&mi.never);
      if (items > 0) mbar_wait(smem_u32(&mi.q_full), (items - 1) & 1, never);
      for (uint32_t s = t < 2 ? 0 : t - 2; s < t; ++s) mbar_wait((for_s ? k_full : v_full) + 8 * (s & 1), s >> 1 & 1, never);
    }
  } else if (warp >= 5) {
    if (rank == 1) {
      // ---- tells the first CTA what has arrived here ----
      uint32_t t = 0, items = 0;
      const uint32_t here = warp == 5 ? k_full : v_full;
      const uint32_t there = at_rank(smem_u32(warp == 5 ? &mi.k_peer[0] : &mi.v_peer[0]), 0);
      while (it.next()) {
        if (it.len == 0) continue;
        if (warp == 5) wait(smem_u32(&mi.q_full), items++ & 1);
#pragma unroll 1
        for (int i = 0; i < it.n; ++i, ++t) {
          const uint32_t stage = t & 1;
          wait(here + 8 * stage, t >> 1 & 1);
          if (elect_one()) pair_arrive(there + 8 * stage);
          __syncwarp();
        }
      }
      // (the pair's last arrival here comes before this CTA ends)
      if (warp == 5) mbar_wait(smem_u32(&mi.end), 0, smem_u32(&mi.never));
    } else if (warp == 5) {
      // ---- products ----
      const uint32_t k_peer = smem_u32(&mi.k_peer[0]), v_peer = smem_u32(&mi.v_peer[0]);
      const uint32_t s_full = smem_u32(&mi.s_full[0]), s_free = smem_u32(&mi.s_free[0]);
      uint32_t t = 0, items = 0;
      bool first = false;  // the tile before is a row tile's first
      auto values = [&](uint32_t u) {  // O of tile u
        const uint32_t stage = u & 1, parity = u >> 1 & 1;
        wait((lane == 0 ? smem_u32(&mi.p_full[0]) : lane == 1 ? v_full : v_peer) + 8 * stage, parity);
        __syncwarp();
        tmem_fence_after();
        if (elect_one()) {
          const uint64_t pa = umma_desc(base + L::kPAt + stage * L::kPNext, 16, 1024);
          const uint32_t v = base + kStageAt + stage * kStage + kK;
          constexpr int kSteps = kFp8 ? 1 : 2, kStep = 32 / kSteps;  // products along a half's entries, entries of one
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < 2 * kSteps; ++k) {
              const uint64_t vb = umma_desc(v + k / kSteps * (kPieces / 2 * kKPiece) + n * (kPieces / 4 * kKPiece) + k % kSteps * (kStep * 128),
                                            kKPiece, 1024);
#pragma unroll
              for (int x = 0; x < L::kWeights; ++x)
                pair_umma<kFp8>(tmem + n * 128, pa + 2 * k + x * (L::kPPart / 16), vb, kIdescO, !first || k > 0 || x > 0);
            }
          pair_commit(v_empty + 8 * stage);
        }
        __syncwarp();
      };
      while (it.next()) {
        if (it.len == 0) continue;
        const uint32_t q = items++ & 1;
#pragma unroll 1
        for (int i = 0; i < it.n; ++i, ++t) {
          const uint32_t stage = t & 1, parity = t >> 1 & 1;
          // (queries that the softmax warps convert come after the row tile before them, its last product too)
          const bool early = kFp8 && i == 0;
          if (early && t > 0) values(t - 1);
          if (i == 0) wait(smem_u32(&mi.q_full), q);
          // (the lanes wait for one barrier each: one after the other, each took 80 clocks also where it was there)
          wait((lane == 0 ? k_full : lane == 1 ? k_peer : s_free) + 8 * stage, lane < 2 ? parity : parity ^ 1);
          __syncwarp();
          tmem_fence_after();
          if (elect_one()) {
            const uint32_t d = tmem + kSAt + stage * kKeys;
#pragma unroll
            for (int c = 0; c <= kPieces; ++c) {
              const uint64_t qa = umma_desc(base + c * kQPiece, 16, 1024);
              const uint64_t kb = umma_desc(base + kStageAt + stage * kStage + c * kKPiece, 16, 1024);
#pragma unroll
              for (int k = 0; k < (kFp8 && c == kPieces ? 2 : 4); ++k)  // 32 bytes each; an e4m3 entry's rotated values are 64
#pragma unroll
                for (int x = 0; x < kParts; ++x)
                  pair_umma<kFp8>(d, qa + 2 * k + x * (L::kQPart / 16), kb + 2 * k, kIdescS, c > 0 || k > 0 || x > 0);
            }
            pair_commit(k_empty + 8 * stage);
            pair_commit(s_full + 8 * stage);
            if (i + 1 == it.n) pair_commit(smem_u32(&mi.q_empty));
          }
          __syncwarp();
          if (!early && t > 0) values(t - 1);
          first = i == 0;
        }
      }
      if (t > 0) values(t - 1);
      // everything issued ends before the tensor memory is given back
      if (elect_one()) pair_commit(smem_u32(&mi.end));
      __syncwarp();
      mbar_wait(smem_u32(&mi.end), 0, smem_u32(&mi.never));
    }
  } else {
    // ---- softmax and epilogue ----
    const float kv_scale = kFp8 && p.scale != nullptr ? *p.scale : 1.0f;
    float factor = p.sm_scale * kLog2e * kv_scale;
    const float all_rows = factor;
    constexpr bool kF16 = std::is_same<T, f16>::value;
    constexpr float kCap = kFp8 ? 15.5f : kF16 ? 15.0f : 8.0f;    // weights stay below 2^kCap
    constexpr float kFirst = kFp8 ? 11.0f : kF16 ? 8.0f : 0.0f;   // where a first reference puts the largest
    constexpr float kLater = kFp8 ? 13.0f : kF16 ? 8.0f : 0.0f;   // where a later one does
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const int row = tid & (kRows - 1), half = tid >> 6;  // the thread's row, and which half of its entries and latent values
    const uint32_t s_free = smem_u32(&mi.s_free[0]), p_full = smem_u32(&mi.p_full[0]);
    const uint32_t s_free0 = at_rank(s_free, 0), p_full0 = at_rank(p_full, 0);
    // at a barrier of the first CTA
    auto arrive = [&](uint32_t bar, uint32_t bar0) {
      if (lane == 0) {
        if (rank == 0) mbar_arrive(bar);
        else pair_arrive(bar0);
      }
    };
    uint8_t* p_row = smem + L::kPAt + row * 128;
    JoinNote note{-1, 0, 0, 0};
    uint32_t t = 0;
    int item = 0;
    // the product of the tile before is done
    auto product_done = [&]() {
      if (t > 0) wait(v_empty + 8 * ((t - 1) & 1), (t - 1) >> 1 & 1);
    };
    // For each item: its queries, then the sums of the item before (whose last product runs meanwhile), then its tiles.
    const int first_row = static_cast<int>(rank) * rpc;
    bool more = it.next();
    float* prev_out = nullptr;  // where this thread's half of its row goes
    int prev_n = -1;            // tiles of the item before
    bool prev_row = false;      // whether the row exists
    for (;; ++item) {
      float ref = -INFINITY, l = 0.0f;
      const int n_rows = more ? min(rpc, it.n_rows - first_row) : 0;
      if (kFp8 && more && it.n > 0) {  // (all products with the queries before are done: their scores have been read)
        load_queries<T, kParts, kRows>(
            [&](int r) {
              const int rr = it.row0 + first_row + r, t = rr / p.H;
              return static_cast<const T*>(p.q) + t / p.q_len * p.qr_stride + t % p.q_len * p.qt_stride + rr % p.H * p.qh_stride;
            },
            n_rows, smem, mi, all_rows);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&mi.q_full));
      }
      if (prev_n >= 0) {
        if (prev_n > 0) product_done();
        __syncwarp();
        tmem_fence_after();
        if (stopped(stop) && tid == 0) {
          const uint32_t at = smem_u32(&mi.bad_from);
          for (uint32_t r = 0; r < 2; ++r)
            asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" ::"r"(at_rank(at, r)), "r"(item - 1) : "memory");
        }
#pragma unroll 1
        for (int c = 0; c < 256; c += 32) {
          uint32_t o[32];
          if (prev_n > 0) {
            tmem_ld32(tmem + c + lanes, o);
            tmem_wait_ld();
            tmem_pin<32>(o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0;
          }
          if constexpr (kFp8) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * kv_scale);
          }
          if (prev_row) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) store32(prev_out + c + k, o + k);
          }
        }
        tmem_fence_before();
      }
      if (!more) break;
      if (kFp8 && it.n > 0) {
        named_sync<kSoft>(1);
        factor = mi.factor[row];
      }
#pragma unroll 1
      for (int i = 0; i < it.n; ++i, ++t) {
        const uint32_t stage = t & 1, parity = t >> 1 & 1;
        wait(smem_u32(&mi.m_full[t & 3]), t >> 2 & 1);
        wait(smem_u32(&mi.s_full[0]) + 8 * stage, parity);
        __syncwarp();
        tmem_fence_after();
        uint32_t raw_s[32];
        tmem_ld32(tmem + kSAt + stage * kKeys + lanes, raw_s);
        const uint32_t mask = static_cast<uint32_t>(mi.mask[t & 3] >> (32 * half));
        tmem_wait_ld();
        tmem_pin<32>(raw_s);
        tmem_fence_before();
        __syncwarp();
        arrive(s_free + 8 * stage, s_free0 + 8 * stage);
        float* s = reinterpret_cast<float*>(raw_s);
        alignas(8) float x[32];
        // Scores less the reference, two at a time. A reference of -inf makes +inf of what it meets, which raises it; where a
        // score may be -inf too, it takes the other way.
        const bool all = mask == 0xffffffffu && factor > 0.0f;
        float2* x2 = reinterpret_cast<float2*>(x);
        float over = -INFINITY;
        if (all) {
          const float2 f2 = make_float2(factor, factor), r2 = make_float2(-ref, -ref);
#pragma unroll
          for (int k = 0; k < 16; ++k) x2[k] = fma2(make_float2(s[2 * k], s[2 * k + 1]), f2, r2);
#pragma unroll
          for (int k = 0; k < 16; ++k) over = max3(over, x[2 * k], x[2 * k + 1]);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (!(mask >> k & 1)) s[k] = -INFINITY;
            x[k] = s[k] == -INFINITY ? -INFINITY : fmaf(s[k], factor, -ref);
            over = fmaxf(over, x[k]);
          }
        }
        if (named_any<kSoft>(2, over > kCap)) {
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < 32; ++k) top = fmaxf(top, s[k] == -INFINITY ? -INFINITY : s[k] * factor);
          mi.tops[tid] = top;
          named_sync<kSoft>(1);
          top = fmaxf(top, mi.tops[tid ^ kRows]) - (ref == -INFINITY ? kFirst : kLater);
          named_sync<kSoft>(1);  // (before the place is written again)
          float a = 1.0f;
          if (top > ref) {
            a = ref == -INFINITY ? 0.0f : ex2(ref - top);
            ref = top;
            l *= a;
          }
          if (i > 0) {
            product_done();
            __syncwarp();
            tmem_fence_after();
#pragma unroll 1
            for (int c = 0; c < 256; c += 32) {
              uint32_t o[32];
              tmem_ld32(tmem + c + lanes, o);
              tmem_wait_ld();
              tmem_pin<32>(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
              tmem_st32(tmem + c + lanes, o);
            }
            tmem_wait_st();
            tmem_fence_before();
          }
          const float from = ref == -INFINITY ? 0.0f : ref;  // (nothing but -inf so far)
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = s[k] == -INFINITY ? -INFINITY : fmaf(s[k], factor, -from);
        } else if (ref == -INFINITY) {  // nothing but -inf and NaN so far
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = s[k];
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = ex2(x[k]);
        float2 sum2[2] = {x2[0], x2[1]};
#pragma unroll
        for (int k = 2; k < 16; ++k) sum2[k & 1] = add2(sum2[k & 1], x2[k]);
        l += (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
        // values past the end may be anything: their weights are 0, so must they be
        const int left = it.len - (it.tile + i) * kDecodeTile;
        if (left < kDecodeTile) {
          wait(v_full + 8 * stage, parity);
          uint8_t* v = smem + kStageAt + stage * kStage + kK;
          constexpr int kUnits = kPieces / 2 * 8;  // of 16 bytes, of an entry
          for (int y = tid; y < (kDecodeTile - left) * kUnits; y += kSoft) {
            const int key = left + y / kUnits, u = y % kUnits;
            *reinterpret_cast<uint4*>(v + (key / kKeys) * (kPieces / 2 * kKPiece) + (u >> 3) * kKPiece + (key % kKeys) * 128 + (u & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
        }
        // the product two tiles before has read its weights
        if (t >= 2) wait(v_empty + 8 * stage, parity ^ 1);
        if constexpr (!kFp8) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(p_row + stage * L::kPNext + (((4 * half + j) ^ (row & 7)) << 4)) =
                make_uint4(pack2<T>(x[8 * j], x[8 * j + 1]), pack2<T>(x[8 * j + 2], x[8 * j + 3]),
                           pack2<T>(x[8 * j + 4], x[8 * j + 5]), pack2<T>(x[8 * j + 6], x[8 * j + 7]));
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t w[3][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t a = pack2<f16>(x[16 * j + 4 * k], x[16 * j + 4 * k + 1]), b = pack2<f16>(x[16 * j + 4 * k + 2], x[16 * j + 4 * k + 3]);
#pragma unroll
              for (int part = 0; part < 3; ++part) {
                const uint32_t lo = part < 2 ? e5m2_part(a) : e5m2_last(a), hi = part < 2 ? e5m2_part(b) : e5m2_last(b);
                w[part][k] = (lo & 0xffff) | hi << 16;
              }
            }
#pragma unroll
            for (int part = 0; part < 3; ++part)
              *reinterpret_cast<uint4*>(p_row + part * L::kPPart + (((4 * stage + 2 * half + j) ^ (row & 7)) << 4)) =
                  make_uint4(w[part][0], w[part][1], w[part][2], w[part][3]);
          }
        }
        fence_async_smem();
        __syncwarp();
        arrive(p_full + 8 * stage, p_full0 + 8 * stage);
      }
      // sums of the row's halves, in their order
      mi.sums[tid] = l;
      named_sync<kSoft>(1);
      const float sum = mi.sums[row] + mi.sums[row + kRows];
      named_sync<kSoft>(1);
      const bool whole = it.n == it.tiles;
      // where the rows go: a slot of the workspace, or the state
      float* to = p.ws.slots + (static_cast<int64_t>(unit) * 2 + (it.tile == 0 ? 1 : 0)) * p.slot_floats;
      float* ml = to + p.rows_per_group * kLatent;
      if (whole) {
        to = p.state + static_cast<int64_t>(it.row0) * kLatent;
        ml = p.state_ml + 2 * static_cast<int64_t>(it.row0);
      }
      if (half == 0 && row < n_rows) *reinterpret_cast<float2*>(ml + 2 * (first_row + row)) = make_float2(ref, sum);
      if (whole || it.tile == 0) {
        const int parts = whole ? 0 : unit_of(it.last_piece(), share.total, share.units) - unit + 1;
        if (half == 0 && row < n_rows)
          p.row_notes[it.row0 + first_row + row] = {static_cast<uint16_t>(whole ? 0 : unit), static_cast<uint16_t>(parts), first_row + row};
        if (!whole && tid == 0) note = {it.b, parts, it.row0, it.n_rows};
      }
      prev_out = to + static_cast<int64_t>(first_row + row) * kLatent + half * 256;
      prev_n = it.n;
      prev_row = row < n_rows;
      more = it.next();
    }
    if (tid == 0 && rank == 0) p.ws.notes[unit] = note;
    if (stopped(stop) && tid == 0) set_flag(p.err, PMG_FLAG_TIMEOUT);
  }
  tmem_fence_before();
  __syncthreads();
  pair_sync();
  tmem_fence_after();
  if (warp == 5) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kColumns) : "memory");
  if (mi.bad_from != INT32_MAX) {  // rows of items that a timeout of either CTA touched
    PrefixItems<kItemCost> again(p, share);
    for (int item = 0; again.next(); ++item) {
      const int first_row = static_cast<int>(rank) * rpc;
      if (item < mi.bad_from || tid >= min(rpc, again.n_rows - first_row)) continue;
      float* ml = again.n == again.tiles ? p.state_ml + 2 * static_cast<int64_t>(again.row0)
                                         : p.ws.slots + (static_cast<int64_t>(unit) * 2 + (again.tile == 0 ? 1 : 0)) * p.slot_floats +
                                               p.rows_per_group * kLatent;
      ml[2 * (first_row + tid) + 1] = __uint_as_float(0x7fffffffu);
    }
  }
}

template <class T, int kParts>
int run(const DecodeParams& p, const CUtensorMap& latent, const CUtensorMap& rope, const CUtensorMap& q, int box_rows, void* stream) {
  auto k = shared_pair_kernel<T, kParts>;
  const int st = allow_smem(reinterpret_cast<const void*>(k), Lay<kParts>::kBytes);
  if (st != PMG_OK) return st;
  return launch(k, dim3(static_cast<unsigned>(2 * p.units)), kThreads, Lay<kParts>::kBytes, stream, p, latent, rope, q, box_rows);
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

}  // namespace

// A CTA's queries as one box of the copy engine: whole tokens, or whole parts of one, at most an eighth of the CTA's rows
// empty. The box is one of new tokens of a request, of whole requests, or, where the tokens of all requests lie at one
// stride, of any of them.
struct QueryBox {
  int rows;                 // 0: there is none
  uint32_t heads, tokens, reqs;
  bool flat;                // one dimension of tokens
};
static QueryBox query_box(const DecodeParams& p) {
  const int rows = p.H <= kRows ? kRows / p.H * p.H : p.H % kRows == 0 ? kRows : 0;
  if (rows < 56 || (p.qh_stride == 0 && p.H > 1)) return {0, 0, 0, 0, false};
  const int heads = std::min(p.H, rows), n = rows / heads;  // (a part of a token: one)
  const bool in = p.q_len % n == 0, over = n % p.q_len == 0;
  if ((in || over) && (p.qt_stride > 0 || p.q_len == 1) && (p.qr_stride > 0 || p.reqs == 1))
    return {rows, static_cast<uint32_t>(heads), static_cast<uint32_t>(in ? n : p.q_len), static_cast<uint32_t>(in ? 1 : n / p.q_len), false};
  if (p.qt_stride > 0 && (p.reqs == 1 || p.qr_stride == p.q_len * p.qt_stride))
    return {rows, static_cast<uint32_t>(heads), static_cast<uint32_t>(n), 1, true};
  return {0, 0, 0, 0, false};
}

bool prefix_pair_takes(const DecodeParams& p, int q_dtype, int cache_dtype) {
  return static_cast<int64_t>(p.reqs) * p.q_len * p.H > kRows && (cache_dtype == PMG_FP8_E4M3 || query_box(p).rows > 0);
}

int prefix_pair(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream) {
  const bool fp8 = cache_dtype == PMG_FP8_E4M3;  // whose queries the softmax warps convert, row by row
  const QueryBox qb = fp8 ? QueryBox{kRows, 0, 0, 0, false} : query_box(p);
  p.rows_per_group = 2 * qb.rows;
  p.groups = 1;
  p.units = sms / 2;
  // a pair's slot is two CTAs'
  p.slot_floats = (static_cast<int64_t>(p.rows_per_group) * (kLatent + 2) + 7) / 8 * 8;
  static_assert(2 * kRows * (kLatent + 2) <= 2 * kSlotFloats, "fits");
  const CUtensorMapDataType type = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : q_dtype == PMG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int box_rows = gcd(p.B, kKeys), ec = fp8 ? 1 : 2;
  const uint64_t page = static_cast<uint64_t>(p.B), blocks = static_cast<uint64_t>(p.num_blocks);
  const uint64_t row_stride = static_cast<uint64_t>(p.tok_stride) * ec, blk_stride = static_cast<uint64_t>(p.blk_stride) * ec;
  const uint32_t piece = 128 / ec, pieces = kLatent / piece, box = static_cast<uint32_t>(box_rows);
  CUtensorMap latent, rope, q;
  // the latent part as pieces of 128 bytes; the rotated part from the whole row (an e4m3 one is half a piece, and what lies
  // past the row reads as 0)
  int st = tensor_map<4>(&latent, type, p.cache, {piece, page, pieces, blocks}, {row_stride, 128, blk_stride},
                         {piece, box, box_rows == kKeys ? pieces / 2 : 1, 1});
  if (st == PMG_OK) st = tensor_map<3>(&rope, type, p.cache, {kEntry, page, blocks}, {row_stride, blk_stride}, {piece, box, 1});
  if (st != PMG_OK) return st;
  q = rope;
  p.q_tma = 0;
  if (fp8)
    return q_dtype == PMG_BF16 ? run<bf16, 2>(p, latent, rope, q, box_rows, stream) : run<f16, 3>(p, latent, rope, q, box_rows, stream);
  const uint64_t reqs = static_cast<uint64_t>(p.reqs), tokens = static_cast<uint64_t>(p.q_len) * (qb.flat ? reqs : 1);
  p.q_tma = qb.flat ? INT32_MAX : p.q_len;  // new tokens of the dimension before the last
  // (the stride of a dimension of one is not used; it has to be a valid one all the same)
  st = tensor_map<4>(&q, type, p.q, {kEntry, static_cast<uint64_t>(p.H), tokens, qb.flat ? 1 : reqs},
                     {p.H > 1 ? p.qh_stride * 2ull : kEntry * 2ull, tokens > 1 ? p.qt_stride * 2ull : kEntry * 2ull,
                      !qb.flat && reqs > 1 ? p.qr_stride * 2ull : kEntry * 2ull},
                     {64, qb.heads, qb.tokens, qb.reqs});
  if (st != PMG_OK) return st;
  return q_dtype == PMG_BF16 ? run<bf16, 1>(p, latent, rope, q, box_rows, stream) : run<f16, 1>(p, latent, rope, q, box_rows, stream);
}

}  // namespace pmg_mla
