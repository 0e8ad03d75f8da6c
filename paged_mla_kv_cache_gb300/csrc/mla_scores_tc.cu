// Upper bounds of the scores of the cache's pages on the fifth-generation
// tensor core: entries of 576 16-bit values.
//
// Mathematics: with q+ = max(q, 0) and q- = min(q, 0) the bound of a page for a
// row of queries is q+ . hi + q- . lo. For a tile of 64 pages and N rows that
// is one product of 64 x 1152 and 1152 x N values (S = HI Q+^T + LO Q-^T) with
// the pages on the M side, so that a lane of tensor memory holds all rows'
// bounds of its page and the largest over the heads needs no other lane. A NaN
// there may be an infinite bound's product with the 0 of the other half: such
// scores are taken again at the share's end, each by a warp (score_sum_odd).
//
// Bound by the bounds' bytes (2304 a page) as long as there are few rows; by the
// rate of the products of 64 lanes, half of the full one, from about 64 heads
// on. A tile's bounds (147 KB) come by asynchronous copies, page by page
// through the block table, and stay in shared memory while the rows pass in
// chunks of N: the rows' pieces of 64 columns are split by sign on their way
// from registers into a ring of two to four stages. A piece of the next tile's
// bounds is asked for as soon as the last product with the one in its place is
// done.
//
// Roles: warps 0-7 load and split queries, warps 8-11 take the largest over the
// heads, warps 12-15 copy bounds, warp 16 issues products. The flat list of tiles
// of all requests is cut into equal shares, a CTA each.
//
// Measured: 43 us for 256 requests of 128 heads and 1024 to 32768 entries on
// pages of 64 (the bytes alone are 18), 6.7 us for 1875 pages of one request, 6.3 us for a
// few pages, which is three loads one after the other (lengths, page ids, bounds).
#include <algorithm>

#include "mla_scores.cuh"
#include "mla_sm103.cuh"

namespace pmg_mla {
namespace {

constexpr int kLoaders = 256, kReaders = 128, kCopiers = 128;
constexpr int kThreads = kLoaders + kReaders + kCopiers + 32;
constexpr int kLoadWarps = kLoaders / 32, kCopyWarp = kLoadWarps + kReaders / 32, kIssuer = kThreads / 32 - 1;
constexpr int kEntry = 576;
constexpr int kPieces = kEntry / 64;        // of 128 bytes
constexpr int kPiece = kScoreTile * 128;    // 64 pages of one piece
constexpr int kTurn = 3;                    // steps between a load of queries and their split: pieces come in turns of so many
static_assert(kPieces % kTurn == 0, "whole turns");
constexpr int kHalfway = 5;

template <int N>
struct Lay {
  static constexpr int kStages = N == 128 ? 2 : 4;  // of queries: 64 KB
  // Accumulators of a row and page: hi and lo, and of each the first kHalfway pieces and the others, as far as tensor
  // memory reaches twice. The tensor core cuts a sum at every addition, and all of these have one sign: one sum of 72
  // additions was off by 1.2e-6 of the score, four of 16 or 20 by 3e-7.
  static constexpr int kSums = N == 128 ? 2 : 4;
  static constexpr int kStage = 2 * N * 128;
  static constexpr int kStageAt = 2 * kPieces * kPiece;
  static constexpr int kBytes = kStageAt + kStages * kStage + 1024;
  static_assert(kBytes <= 232448 - 1024, "fits beside the barriers");
};

struct Misc {
  uint64_t page_full[kPieces], page_empty[kPieces], full[4], empty[4], s_full[2], s_free[2], end;
  int64_t scratch[33], found[2];
  float shift[kReaders / 32][128];  // of a chunk's rows, each reading warp's own
  uint32_t tmem;
  int32_t stop, never;
};

// Walks the tiles of a share.
struct Tiles {
  const ScoreParams* p;
  int64_t at, end;
  int64_t skip;
  int r;
  int64_t tile, last;   // the current one, the end of the request's in this share
  int64_t pages;
  SparseLen len;
  __device__ Tiles(const ScoreParams& p_, const Share& s) : p(&p_), at(s.begin), end(s.end), skip(s.offset), r(s.item - 1) {
    tile = last = pages = 0;
    len = SparseLen{0, 0, 0};
  }
  __device__ bool next() {
    if (++tile < last) return true;
    do {
      if (at >= end) return false;
      ++r;
      len = sparse_len(p->seq, r, p->bt_stride, p->B);
      pages = score_pages(*p, len);
      const int64_t tiles = score_tiles(pages);
      const int64_t n = min(max(tiles, static_cast<int64_t>(1)) - skip, end - at);
      tile = skip;
      last = min(skip + n, tiles);
      at += n;
      skip = 0;
    } while (tile >= last);
    return true;
  }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

template <class T, int N>
__global__ void __launch_bounds__(kThreads, 1) scores_tc_kernel(const __grid_constant__ ScoreParams p) {
  using L = Lay<N>;
  constexpr int kStages = L::kStages, kSums = L::kSums;
  extern __shared__ uint8_t raw[];
  __shared__ Misc mi;
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  constexpr int kColumns = 2 * kSums * N;
  if (tid == 0) {
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(smem_u32(&mi.page_full[i]), kCopiers);
      mbar_init(smem_u32(&mi.page_empty[i]), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&mi.full[i]), kLoadWarps);
      mbar_init(smem_u32(&mi.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&mi.s_full[i]), 1);
      mbar_init(smem_u32(&mi.s_free[i]), 4);
    }
    mbar_init(smem_u32(&mi.end), 1);
    mi.stop = mi.never = 0;
    mbar_fence_init();
  }
  if (warp == kIssuer) tmem_alloc(smem_u32(&mi.tmem), kColumns);
  pdl_entry();
  const Share share = find_share([&](int r) { return score_pieces(p, r); }, p.R, blockIdx.x, p.units, mi.scratch, mi.found);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = mi.tmem, stop = smem_u32(&mi.stop);
  const uint32_t full = smem_u32(&mi.full[0]), empty = smem_u32(&mi.empty[0]);
  const uint32_t s_full = smem_u32(&mi.s_full[0]), s_free = smem_u32(&mi.s_free[0]);
  const int rows = p.q_len * p.H, chunks = (rows + N - 1) / N;

  if (warp == kIssuer) {
    // ---- products ----
    constexpr int kFmt = std::is_same<T, bf16>::value ? 1 : 0;
    constexpr uint32_t kIdesc = umma_idesc(kFmt, kFmt, 0, 0, kScoreTile, N);
    Tiles it(p, share);
    uint32_t step = 0, chunk = 0, tile = 0;
    for (; it.next(); ++tile) {
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++chunk) {
        const uint32_t buf = chunk & 1, d = tmem + buf * (kSums * N);
        if (chunk >= 2) mbar_wait(s_free + 8 * buf, ((chunk >> 1) + 1) & 1, stop);
#pragma unroll 1
        for (int k = 0; k < kPieces; ++k, ++step) {
          const uint32_t stage = step % kStages;
          // (a barrier a lane; a tile's bounds are the same phase in all of its chunks)
          mbar_wait(lane == 0 ? smem_u32(&mi.page_full[k]) : full + 8 * stage, lane == 0 ? tile & 1 : step / kStages & 1, stop);
          __syncwarp();
          fence_async_smem();  // (the barriers order the loading warps' writes before it)
          tmem_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint64_t a = umma_desc(base + (2 * k + half) * kPiece, 16, 1024);
              const uint64_t b = umma_desc(base + L::kStageAt + stage * L::kStage + half * (N * 128), 16, 1024);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                umma_ss<false>(d + (half + (kSums == 2 || k < kHalfway ? 0 : 2)) * N, a + 2 * x, b + 2 * x, kIdesc,
                               (k > 0 && (kSums == 2 || k != kHalfway)) || x > 0);
            }
            umma_commit(empty + 8 * stage);
            if (c + 1 == chunks) umma_commit(smem_u32(&mi.page_empty[k]));
            if (k + 1 == kPieces) umma_commit(s_full + 8 * buf);
          }
          __syncwarp();
        }
      }
    }
    if (elect_one()) umma_commit(smem_u32(&mi.end));
    __syncwarp();
    mbar_wait(smem_u32(&mi.end), 0, smem_u32(&mi.never));
  } else if (warp < kLoadWarps) {
    // ---- loads ----
    const int unit = tid & 7, row0 = tid >> 3;  // a 16-byte unit of every kApart-th row of a piece
    constexpr int kApart = kLoaders / 8;
    // queries: units of 16 bytes of this thread's rows of a chunk, kTurn steps ahead
    constexpr int kRows = N < kApart ? 1 : N / kApart;
    const bool splits = N >= kApart || row0 < N;
    uint4 x[kTurn][kRows];
    const T* rows_at[kRows];  // of the chunk whose queries are loaded, or NULL
    auto begin = [&](int r, int c) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int rr = c * N + row0 + kApart * i;
        rows_at[i] = splits && rr < rows ? reinterpret_cast<const T*>(p.q) + r * p.qr_stride + (rr / p.H) * p.qt_stride +
                                     (rr % p.H) * p.qh_stride + unit * 8
                               : nullptr;
      }
    };
    auto load = [&](uint4 (&y)[kRows], int k) {
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        y[i] = rows_at[i] != nullptr ? *reinterpret_cast<const uint4*>(rows_at[i] + k * 64) : make_uint4(0, 0, 0, 0);
    };
    Tiles next(p, share);  // the tile after the one that is filled
    bool more = next.next();
    int r = next.r;  // request of the tile that is filled
    bool next_more = more && next.next();
    uint32_t step = 0;
    if (more) {
      begin(r, 0);
#pragma unroll
      for (int k = 0; k < kTurn; ++k) load(x[k], k);
    }
    while (more) {
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
#pragma unroll 1
        for (int k0 = 0; k0 < kPieces; k0 += kTurn) {
#pragma unroll
          for (int turn = 0; turn < kTurn; ++turn, ++step) {
            const int k = k0 + turn;
            const uint32_t stage = step % kStages;
            if (step >= kStages) mbar_wait(empty + 8 * stage, (step / kStages + 1) & 1, stop);
            // queries by sign
            uint8_t* at = smem + L::kStageAt + stage * L::kStage;
#pragma unroll
            for (int y = 0; y < kRows; ++y) {
              const int row = row0 + kApart * y;
              const uint32_t w[4] = {x[turn][y].x, x[turn][y].y, x[turn][y].z, x[turn][y].w};
              uint32_t u[4], d[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t below = (w[j] >> 15 & 0x00010001u) * 0xffffu;
                u[j] = w[j] & ~below;
                d[j] = w[j] & below;
              }
              const int place = row * 128 + ((unit ^ (row & 7)) << 4);
              if (splits) {
                *reinterpret_cast<uint4*>(at + place) = make_uint4(u[0], u[1], u[2], u[3]);
                *reinterpret_cast<uint4*>(at + N * 128 + place) = make_uint4(d[0], d[1], d[2], d[3]);
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(full + 8 * stage);
            // the queries of the step kTurn further on their way
            if (k + kTurn < kPieces) {
              load(x[turn], k + kTurn);
            } else if (c + 1 < chunks || next_more) {
              if (k + kTurn == kPieces) begin(c + 1 < chunks ? r : next.r, c + 1 < chunks ? c + 1 : 0);
              load(x[turn], k + kTurn - kPieces);
            }
          }
        }
      }
      more = next_more;
      r = next.r;
      if (more) next_more = next.next();
    }
  } else if (warp >= kCopyWarp) {
    // ---- bounds ----
    const int at0 = tid - kCopyWarp * 32, unit = at0 & 7, row0 = at0 >> 3;  // a 16-byte unit of every kApart-th row of a piece
    constexpr int kApart = kCopiers / 8, kPageRows = kScoreTile / kApart;
    uint32_t tile = 0;
    for (Tiles it(p, share); it.next(); ++tile) {
      const int32_t* table = p.bt + static_cast<int64_t>(it.r) * p.bt_stride;
      const T* page[kPageRows];
      bool there[kPageRows];
#pragma unroll
      for (int k = 0; k < kPageRows; ++k) {
        const int64_t c = it.tile * kScoreTile + row0 + kApart * k;
        const int32_t id = c < it.pages ? table[c] : -1;
        there[k] = id >= 0 && id < p.num_blocks;
        page[k] = reinterpret_cast<const T*>(p.bounds) + (there[k] ? id : 0) * p.bb_stride + unit * 8;
      }
#pragma unroll 1
      for (int piece = 0; piece < kPieces; ++piece) {
        // where the tile before has had its last product with the piece in this place
        if (tile > 0) mbar_wait(smem_u32(&mi.page_empty[piece]), (tile - 1) & 1, stop);
#pragma unroll
        for (int k = 0; k < kPageRows; ++k) {
          const int row = row0 + kApart * k;
          const uint32_t dst = base + 2 * piece * kPiece + row * 128 + ((unit ^ (row & 7)) << 4);
          copy16(dst, page[k] + piece * 64, there[k]);
          copy16(dst + kPiece, page[k] + p.br_stride + piece * 64, there[k]);
        }
        // arrives when this thread's copies have
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&mi.page_full[piece])) : "memory");
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---- the largest over the heads ----
    const float factor = p.sm_scale * (p.scale != nullptr ? *p.scale : 1.0f);
    const int part = warp - kLoadWarps;  // of the lanes
    int bad = 0;
    bool odd = false;  // a score of this lane is NaN
    uint32_t chunk = 0;
    for (Tiles it(p, share); it.next();) {
      const int64_t c = it.tile * kScoreTile + part * 16 + lane;  // the page of this lane (of the first 16)
      const bool in = lane < 16 && c < it.pages;
      const int32_t id = in ? p.bt[static_cast<int64_t>(it.r) * p.bt_stride + c] : -1;
      const bool good = id >= 0 && id < p.num_blocks;
      if (in && !good) bad |= PMG_FLAG_PHYS_BLOCK;
      const int64_t first = static_cast<int64_t>(it.r) * rows, place = c * p.B;
      float* out = p.scores + static_cast<int64_t>(it.r) * p.q_len * p.s_stride + c;
      float best = -INFINITY;  // of the heads so far of the token at hand
      int token = 0, head = 0;
      auto done = [&]() {
        const bool seen = place < sparse_seen(it.len, token, p.q_len);
        const bool lost = stopped(stop);  // (by all lanes)
        if (in) *out = lost ? __uint_as_float(0x7fffffffu) : good && seen ? best : -INFINITY;
        odd |= isnan(best);
        out += p.s_stride;
        best = -INFINITY;
        head = 0;
        ++token;
      };
#pragma unroll 1
      for (int row = 0; row < rows; row += N, ++chunk) {
        const uint32_t buf = chunk & 1;
        for (int k = lane; k < N; k += 32) mi.shift[part][k] = row + k < rows ? score_shift(p, first + row + k) : 0.0f;
        mbar_wait(s_full + 8 * buf, chunk >> 1 & 1, stop);
        __syncwarp();
        tmem_fence_after();
#pragma unroll 1
        for (int h = 0; h < N; h += 16) {
          uint32_t s[kSums][16];
#pragma unroll
          for (int k = 0; k < kSums; ++k)
            tmem_ld16(tmem + (buf * kSums + k) * N + h + (static_cast<uint32_t>(part * 32) << 16), s[k]);
          const int left = rows - row - h;
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < kSums; ++k) tmem_pin<16>(s[k]);
          float x[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float sum = __uint_as_float(s[0][k]) + __uint_as_float(s[1][k]);
            if constexpr (kSums == 4) sum += __uint_as_float(s[2][k]) + __uint_as_float(s[3][k]);
            x[k] = sum * factor - mi.shift[part][h + k];
          }
          if (left >= 16 && head + 16 <= p.H) {  // one token's
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
#pragma unroll
              for (int k = 0; k < o; ++k) x[k] = max_nan(x[k], x[k + o]);
            best = max_nan(best, x[0]);
            head += 16;
            if (head == p.H) done();
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (k < left) {
                best = max_nan(best, x[k]);
                if (++head == p.H) done();
              }
          }
        }
        tmem_fence_before();
        __syncwarp();  // (the shifts are read too)
        if (lane == 0) mbar_arrive(s_free + 8 * buf);
      }
    }
    if (__any_sync(0xffffffffu, odd) && !stopped(stop)) {  // (scores whose wait ran out stay NaN)
      for (Tiles it(p, share); it.next();) {
        const int64_t c = it.tile * kScoreTile + part * 16 + lane;
        const bool in = lane < 16 && c < it.pages;
        const int32_t id = in ? p.bt[static_cast<int64_t>(it.r) * p.bt_stride + c] : -1;
        float* out = p.scores + static_cast<int64_t>(it.r) * p.q_len * p.s_stride + c;
        const T* q = reinterpret_cast<const T*>(p.q) + it.r * p.qr_stride;
        int64_t row = static_cast<int64_t>(it.r) * rows;
        for (int token = 0; token < p.q_len; ++token, out += p.s_stride, q += p.qt_stride, row += p.H)
          for (uint32_t left = __ballot_sync(0xffffffffu, in && isnan(*out)); left != 0; left &= left - 1) {
            const int at = __ffs(left) - 1;  // whose page it is (one in the cache: others are -inf)
            const T* hi = reinterpret_cast<const T*>(p.bounds) + __shfl_sync(0xffffffffu, id, at) * p.bb_stride;
            float best = -INFINITY;
            for (int h = 0; h < p.H && !isnan(best); ++h)
              best = max_nan(best, score_sum_odd<T, 8>(q + h * p.qh_stride, hi, hi + p.br_stride, kEntry) * factor -
                                       score_shift(p, row + h));
            if (lane == at) *out = best;
          }
      }
    }
    // columns that no token sees anything of, and what is wrong with a length: with a request's last piece
    int64_t at = share.begin, skip = share.offset;
    for (int r = share.item; at < share.end; ++r, skip = 0) {
      const SparseLen len = sparse_len(p.seq, r, p.bt_stride, p.B);
      const int64_t pages = score_pages(p, len), pieces = max(score_tiles(pages), static_cast<int64_t>(1));
      const int64_t n = min(pieces - skip, share.end - at);
      at += n;
      if (skip + n == pieces) {
        bad |= len.bad;
        score_rest(p, r, pages, tid - kLoaders, kReaders);
      }
    }
    if (stopped(stop)) bad |= PMG_FLAG_TIMEOUT;
    set_flag(p.err, bad);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == kIssuer) tmem_free(tmem, kColumns);
}

template <class T, int N>
int run(const ScoreParams& p, void* stream) {
  auto k = scores_tc_kernel<T, N>;
  const int st = allow_smem(reinterpret_cast<const void*>(k), Lay<N>::kBytes);
  if (st != PMG_OK) return st;
  return launch(k, dim3(static_cast<unsigned>(p.units)), kThreads, Lay<N>::kBytes, stream, p);
}
template <class T>
int run(const ScoreParams& p, void* stream) {
  const int rows = p.q_len * p.H;
  return rows <= 16 ? run<T, 16>(p, stream) : rows <= 32 ? run<T, 32>(p, stream)
         : rows <= 64 ? run<T, 64>(p, stream) : run<T, 128>(p, stream);
}

}  // namespace

bool scores_tc_takes(const ScoreParams& p, int dtype) {
  return p.E == kEntry && (dtype == PMG_BF16 || dtype == PMG_FP16) && p.H > 0 && p.num_blocks > 0 && aligned(p.q, 16) &&
         p.qr_stride % 8 == 0 && p.qt_stride % 8 == 0 && p.qh_stride % 8 == 0 && aligned(p.bounds, 16) &&
         p.bb_stride % 8 == 0 && p.br_stride % 8 == 0;
}

int scores_tc(const ScoreParams& p, int dtype, void* stream) {
  return dtype == PMG_BF16 ? run<bf16>(p, stream) : run<f16>(p, stream);
}

}  // namespace pmg_mla
