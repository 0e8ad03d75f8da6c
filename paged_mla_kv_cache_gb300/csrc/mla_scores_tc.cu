// Upper bounds of the scores of the cache's pages on the fifth-generation
// tensor core: entries of 576 16-bit values.
//
// Mathematics: with q+ = max(q, 0) and q- = min(q, 0) the bound of a page for a
// row of queries is q+ . hi + q- . lo. For a tile of 64 pages and N rows that
// is one product of 64 x 1152 and 1152 x N values (S = HI Q+^T + LO Q-^T) with
// the pages on the M side, so that a lane of tensor memory holds all rows'
// bounds of its page and the largest over the heads needs no other lane.
//
// Bound by the bounds' bytes (2304 a page) as long as there are few rows; by the
// rate of the products of 64 lanes, half of the full one, from about 64 heads
// on. A tile's bounds (147 KB) come by asynchronous copies, page by page
// through the block table, and stay in shared memory while the rows pass in
// chunks of N: the rows' pieces of 64 columns are split by sign on their way
// from registers into a ring of four stages. A piece of the next tile's bounds is
// asked for as soon as the last product with the one in its place is done, five
// steps (pieces) before it is multiplied.
//
// Roles: warps 0-3 load, split and take the largest over the heads; warp 4
// issues products. The flat list of tiles of all requests is cut into equal
// shares, a CTA each.
#include <algorithm>

#include "mla_scores.cuh"
#include "mla_sm103.cuh"

namespace pmg_mla {
namespace {

constexpr int kThreads = 160;
constexpr int kLoaders = 128;
constexpr int kEntry = 576;
constexpr int kPieces = kEntry / 64;        // of 128 bytes
constexpr int kPiece = kScoreTile * 128;    // 64 pages of one piece
constexpr int kStages = 4;                  // of queries
constexpr int kLead = kPieces - kStages;    // steps between a piece's copy and its product

template <int N>
struct Lay {
  static constexpr int kStage = 2 * N * 128;
  static constexpr int kStageAt = 2 * kPieces * kPiece;
  static constexpr int kBytes = kStageAt + kStages * kStage + 1024;
  static_assert(kBytes <= 232448 - 1024, "fits beside the barriers");
};

struct Misc {
  uint64_t full[kStages], empty[kStages], s_full[2], s_free[2], end;
  int64_t scratch[33], found[2];
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
      const int64_t pieces = (pages + kScoreTile - 1) / kScoreTile + 1;
      const int64_t n = min(pieces - skip, end - at);
      tile = skip;
      last = min(skip + n, pieces - 1);
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
  extern __shared__ uint8_t raw[];
  __shared__ Misc mi;
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  constexpr int kColumns = 2 * N < 32 ? 32 : 2 * N;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&mi.full[i]), 4);
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
  if (warp == 4) tmem_alloc(smem_u32(&mi.tmem), kColumns);
  pdl_entry();
  const Share share = find_share([&](int r) { return score_pieces(p, r); }, p.R, blockIdx.x, p.units, mi.scratch, mi.found);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = mi.tmem, stop = smem_u32(&mi.stop);
  const uint32_t full = smem_u32(&mi.full[0]), empty = smem_u32(&mi.empty[0]);
  const uint32_t s_full = smem_u32(&mi.s_full[0]), s_free = smem_u32(&mi.s_free[0]);
  const int rows = p.q_len * p.H, chunks = (rows + N - 1) / N;

  if (warp == 4) {
    // ---- products ----
    constexpr int kFmt = std::is_same<T, bf16>::value ? 1 : 0;
    constexpr uint32_t kIdesc = umma_idesc(kFmt, kFmt, 0, 0, kScoreTile, N);
    Tiles it(p, share);
    uint32_t step = 0, chunk = 0;
    while (it.next()) {
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++chunk) {
        const uint32_t buf = chunk & 1, d = tmem + buf * N;
        if (chunk >= 2) mbar_wait(s_free + 8 * buf, ((chunk >> 1) + 1) & 1, stop);
#pragma unroll 1
        for (int k = 0; k < kPieces; ++k, ++step) {
          const uint32_t stage = step % kStages;
          mbar_wait(full + 8 * stage, step / kStages & 1, stop);
          tmem_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint64_t a = umma_desc(base + (2 * k + half) * kPiece, 16, 1024);
              const uint64_t b = umma_desc(base + L::kStageAt + stage * L::kStage + half * (N * 128), 16, 1024);
#pragma unroll
              for (int x = 0; x < 4; ++x) umma_ss<false>(d, a + 2 * x, b + 2 * x, kIdesc, k > 0 || half > 0 || x > 0);
            }
            umma_commit(empty + 8 * stage);
            if (k + 1 == kPieces) umma_commit(s_full + 8 * buf);
          }
          __syncwarp();
        }
      }
    }
    if (elect_one()) umma_commit(smem_u32(&mi.end));
    __syncwarp();
    mbar_wait(smem_u32(&mi.end), 0, smem_u32(&mi.never));
  } else {
    // ---- loads, and the largest over the heads ----
    const float factor = p.sm_scale * (p.scale != nullptr ? *p.scale : 1.0f);
    const int unit = tid & 7, row0 = tid >> 3;  // a 16-byte unit of every 16th row of a piece
    int bad = 0;
    // bounds: of the tile `ahead`, whose pages this thread knows
    Tiles ahead(p, share);
    const T* page[4];
    bool there[4];
    auto look = [&]() {
      const bool more = ahead.next();
      const int32_t* table = p.bt + static_cast<int64_t>(more ? ahead.r : 0) * p.bt_stride;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t c = ahead.tile * kScoreTile + row0 + 16 * k;
        const int32_t id = more && c < ahead.pages ? table[c] : -1;
        there[k] = id >= 0 && id < p.num_blocks;
        page[k] = reinterpret_cast<const T*>(p.bounds) + (there[k] ? id : 0) * p.bb_stride + unit * 8;
      }
      return more;
    };
    auto copy = [&](int piece) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = row0 + 16 * k;
        const uint32_t dst = base + 2 * piece * kPiece + row * 128 + ((unit ^ (row & 7)) << 4);
        copy16(dst, page[k] + piece * 64, there[k]);
        copy16(dst + kPiece, page[k] + p.br_stride + piece * 64, there[k]);
      }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    bool ahead_more = look();
    for (int k = 0; k < kLead; ++k) {
      if (ahead_more) copy(k);
      commit();
    }
    // queries: units of 16 bytes of this thread's rows of a chunk
    constexpr int kRows = N / 16;
    uint4 x[kRows];
    auto load = [&](int r, int c, int k) {
#pragma unroll
      for (int y = 0; y < kRows; ++y) {
        const int rr = c * N + row0 + 16 * y;
        x[y] = make_uint4(0, 0, 0, 0);
        if (rr < rows)
          x[y] = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.q) + r * p.qr_stride + (rr / p.H) * p.qt_stride +
                                                 (rr % p.H) * p.qh_stride + k * 64 + unit * 8);
      }
    };
    // the largest bound so far of this lane's page for the token of the current row
    float best = -INFINITY;
    int token = 0, head = 0;
    Tiles now(p, share), then(p, share);  // the tile that is filled, and the one whose products are read
    bool more = now.next();
    then.next();
    int then_c = 0;
    uint32_t step = 0, chunk = 0, read = 0;
    auto reduce = [&]() {
      const uint32_t buf = read & 1;
      mbar_wait(s_full + 8 * buf, read >> 1 & 1, stop);
      __syncwarp();
      tmem_fence_after();
      const bool lost = stopped(stop);
      const int64_t c = then.tile * kScoreTile + warp * 16 + lane;  // the page of this lane (of the first 16)
      const bool in = lane < 16 && c < then.pages;
      const int32_t id = in ? p.bt[static_cast<int64_t>(then.r) * p.bt_stride + c] : -1;
      const bool good = id >= 0 && id < p.num_blocks;
      if (in && !good) bad |= PMG_FLAG_PHYS_BLOCK;
      const int64_t first = static_cast<int64_t>(then.r) * rows;
#pragma unroll 1
      for (int h = 0; h < N; h += 16) {
        uint32_t s[16];
        tmem_ld16(tmem + buf * N + h + (static_cast<uint32_t>(warp * 32) << 16), s);
        tmem_wait_ld();
        tmem_pin<16>(s);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int rr = then_c * N + h + k;
          if (rr < rows) {
            best = max_nan(best, __uint_as_float(s[k]) * factor - score_shift(p, first + rr));
            if (++head == p.H) {
              const bool seen = c * p.B < sparse_seen(then.len, token, p.q_len);
              if (in)
                p.scores[(static_cast<int64_t>(then.r) * p.q_len + token) * p.s_stride + c] =
                    lost ? __uint_as_float(0x7fffffffu) : good && seen ? best : -INFINITY;
              best = -INFINITY;
              head = 0;
              ++token;
            }
          }
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free + 8 * buf);
      ++read;
      if (++then_c == chunks) {
        then_c = 0;
        token = 0;
        then.next();
      }
    };
    if (more) load(now.r, 0, 0);
    int drop = kLead;  // the next piece of `ahead` to be copied
    while (more) {
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++chunk) {
#pragma unroll 1
        for (int k = 0; k < kPieces; ++k, ++step) {
          const uint32_t stage = step % kStages;
          if (step >= kStages) mbar_wait(empty + 8 * stage, (step / kStages + 1) & 1, stop);
          // the piece that was multiplied kStages steps ago makes room in a tile's last chunk (the first tile's rest
          // has room from the start)
          const bool last_chunk = k >= kStages ? c + 1 == chunks : c == 0;
          if (last_chunk) {
            if (drop == kPieces) {
              drop = 0;
              ahead_more = look();
            }
            if (ahead_more) copy(drop);
            ++drop;
          }
          commit();
          // queries by sign
          uint8_t* at = smem + L::kStageAt + stage * L::kStage;
#pragma unroll
          for (int y = 0; y < kRows; ++y) {
            const int row = row0 + 16 * y;
            uint4 up, down;
            const uint32_t w[4] = {x[y].x, x[y].y, x[y].z, x[y].w};
            uint32_t u[4], d[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t below = (w[j] >> 15 & 0x00010001u) * 0xffffu;
              u[j] = w[j] & ~below;
              d[j] = w[j] & below;
            }
            up = make_uint4(u[0], u[1], u[2], u[3]);
            down = make_uint4(d[0], d[1], d[2], d[3]);
            const int place = row * 128 + ((unit ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(at + place) = up;
            *reinterpret_cast<uint4*>(at + N * 128 + place) = down;
          }
          // the next step's queries on their way
          if (k + 1 < kPieces) load(now.r, c, k + 1);
          else if (c + 1 < chunks) load(now.r, c + 1, 0);
          asm volatile("cp.async.wait_group %0;" ::"n"(kLead) : "memory");
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full + 8 * stage);
        }
        if (chunk > 0) reduce();
      }
      more = now.next();
      if (more) load(now.r, 0, 0);
    }
    if (chunk > 0) reduce();
    asm volatile("cp.async.wait_all;" ::: "memory");
    // columns that no token sees anything of, and what is wrong with a length: with a request's last piece
    int64_t at = share.begin, skip = share.offset;
    for (int r = share.item; at < share.end; ++r, skip = 0) {
      const SparseLen len = sparse_len(p.seq, r, p.bt_stride, p.B);
      const int64_t pages = score_pages(p, len), pieces = (pages + kScoreTile - 1) / kScoreTile + 1;
      const int64_t n = min(pieces - skip, share.end - at);
      at += n;
      if (skip + n == pieces) {
        bad |= len.bad;
        score_rest(p, r, pages, tid, kLoaders);
      }
    }
    if (stopped(stop)) bad |= PMG_FLAG_TIMEOUT;
    set_flag(p.err, bad);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 4) tmem_free(tmem, kColumns);
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
  return rows <= 16 ? run<T, 16>(p, stream) : rows <= 32 ? run<T, 32>(p, stream) : run<T, 64>(p, stream);
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
