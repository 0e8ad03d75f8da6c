// Expanded latent attention on the fifth-generation tensor core: 128 + 64 key
// values, 128 values a head, 16-bit types.
//
// Mathematics. An item is 256 query rows of one head: two halves of 128 rows.
// For a block of 128 keys, S = Q K^T (128 x 128 over 192) for each half, P =
// 2^(S - ref), O += P V. S and O stay in tensor memory (2 x 128 + 2 x 128
// columns: all of it); P is written over S as 16-bit values and is read from
// there by the second product.
//
// Bound: the tensor core. A block costs a half 768 + 512 clocks of products
// against about 128 exponentials a thread, and the halves take turns: while
// one half's softmax runs, the other half's products do. The rotated key part
// is loaded once a token (not once a head) straight from the gathered rows.
// Measured: a causal prompt of 8192 tokens, 32 heads, 528 us (1.30 PFLOP/s, at
// the clocks that the power limit leaves, about 1.7 GHz); 512 rows over 60000
// keys, 16 heads, 250 us (1.26 PFLOP/s). A block takes some 3500 clocks where
// its products alone take 2667 (both operands of the scores come from shared
// memory): the rest is the change between the halves.
//
// Roles: warps 0-3 and 4-7 are the softmax and epilogue of a half each (a row
// a thread, so no maximum or sum ever crosses threads); warp 8 loads; warp 9
// issues products; warps 10 and 11 make the values finite that some row's
// weight of 0 would meet: rows past the end of a request, which may hold
// anything, and infinities and NaN of keys that some row does not see.
//
// A row's reference follows its maximum only when a score passes it by 2^8, so
// the accumulator is rescaled in the first blocks at most. Weights are rounded
// to the type of the values for the second product (2^-8 or 2^-11 of each; the
// sum of weights is of the unrounded ones): wider ones would need the values
// widened too, for products of half the rate. fp16 weights are kept from 2^8 to 2^15
// where the largest ones are, so that one strong key does not push the weights
// of the others below fp16's smallest, 2^-24. Work is cut into
// equal shares of blocks over the whole call (see mla_attn.cuh): causal
// triangles, short and long requests cost every SM the same, and a chunk of
// few rows over a long context uses them all.
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "mla_prefill_tc.cuh"
#include "mla_sm103.cuh"

namespace pmg_mla {
namespace {

constexpr int kThreads = 384;
// registers of a thread: 12 warps are launched with 168, then the last 4 give some to the first 8
constexpr int kRegsUp = 208, kRegsDown = 80;
static_assert(8 * kRegsUp + 4 * kRegsDown <= 12 * 168, "the shares add up to the launch's");
constexpr int kRows = 256, kHalf = 128, kBlock = 128;
constexpr int kNope = 128, kRope = 64, kVal = 128;
constexpr int kPiece = 128 * 128;        // 128 rows of 128 bytes
constexpr int kSlots = 8;                // key and value pieces in flight: 3 + 2 a block
constexpr int kQAt = 0;                  // two halves of three pieces
constexpr int kSlotAt = 6 * kPiece;
constexpr int kMiscAt = kSlotAt + kSlots * kPiece;
constexpr int kMisc = 1024;
constexpr int kBytes = kMiscAt + kMisc + 1024;
static_assert(kBytes <= 232448, "fits");
constexpr int kSlotRow = kVal;           // floats of a row in a join slot, its two sums behind all rows

struct Misc {
  uint64_t k_full[2], v_full[2], k_empty[2], v_empty[2];  // of a block's key and value pieces, by the block's parity
  uint64_t q_full, q_empty, s_full[2], p_full[4], o_done[2], dirty, clean, end;
  int64_t scratch[33], found[2];
  uint32_t tmem;
  int32_t stop, never;
  int32_t spoiled;  // values were set to 0 that rows see: the epilogue adds them
};
static_assert(sizeof(Misc) <= kMisc, "Misc fits");

// keys that row tile t of a request sees at most
__device__ __forceinline__ int keys_of(const PrefillReq& x, int t, int causal) {
  if (!causal) return x.lk;
  const int64_t end = min(static_cast<int64_t>(x.lq), static_cast<int64_t>(t + 1) * kRows);
  return static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(x.lk), x.lk - x.lq + end)));
}
constexpr int kItemCost = 1;  // what an item's beginning and end cost, in blocks
// (rows and keys go up to INT32_MAX: no sum passes it before it is divided)
__device__ __forceinline__ int parts_of(int n, uint32_t size) {
  return static_cast<int>((static_cast<uint32_t>(n) + size - 1) / size);
}
__device__ __forceinline__ int blocks_of(int keys) { return keys > 0 ? parts_of(keys, kBlock) : 1; }
__device__ __forceinline__ int tiles_of(const PrefillReq& x) { return parts_of(x.lq, kRows); }

// pieces of one head of a request
__device__ __forceinline__ int64_t head_pieces(const PrefillReq& x, int causal) {
  const int n = tiles_of(x);
  if (!causal) return static_cast<int64_t>(n) * (kItemCost + blocks_of(x.lk));
  int64_t s = static_cast<int64_t>(n) * kItemCost;
#pragma unroll 1
  for (int t = 0; t < n; ++t) s += blocks_of(keys_of(x, t, causal));
  return s;
}

// Walks the items of a share: (request, head, row tile), blocks [b0, b0 + n) of nb.
struct Items {
  const PrefillParams* p;
  int64_t at, end;
  int r, head, tile;
  PrefillReq x;
  int nb, b0, n;
  int act[2];   // blocks that each half takes part in (of the item's nb)
  int keys;     // keys of the item
  int skip;     // pieces of the item before this share
  int64_t first;  // its first piece
  bool begun;

  __device__ Items(const PrefillParams& p_, const Share& s) : p(&p_), at(s.begin), end(s.end) {
    r = s.item;
    head = tile = nb = b0 = n = keys = 0;
    skip = 0;
    begun = false;
    if (at < end) {
      x = prefill_req(*p, r);
      const int64_t per = head_pieces(x, p->causal);
      head = static_cast<int>(s.offset / per);
      int64_t left = s.offset - head * per;
      for (;;) {
        const int here = kItemCost + blocks_of(keys_of(x, tile, p->causal));
        if (left < here) break;
        left -= here;
        ++tile;
      }
      skip = static_cast<int>(left);
    }
  }
  // the next item of which this share has blocks
  __device__ bool next() {
    do {
      if (at >= end) return false;
      if (begun && ++tile >= tiles_of(x)) {
        tile = 0;
        if (++head >= p->H) {
          head = 0;
          do x = prefill_req(*p, ++r); while (x.lq == 0);
        }
      }
      begun = true;
      keys = keys_of(x, tile, p->causal);
      nb = blocks_of(keys);
      first = at - skip;
      const int take = static_cast<int>(min(static_cast<int64_t>(kItemCost + nb - skip), end - at));
      b0 = max(0, skip - kItemCost);
      n = max(0, skip + take - kItemCost) - b0;
      at += take;
      skip = 0;
    } while (n == 0);
    // the first half's last row may see fewer keys; the second half may not exist
    const int rows = x.lq - tile * kRows;
    int k0 = keys;
    if (p->causal && rows > kHalf)
      k0 = max(0, min(x.lk, x.lk - x.lq + tile * kRows + kHalf));
    act[0] = k0 > 0 ? parts_of(k0, kBlock) : 0;
    act[1] = rows > kHalf && keys > 0 ? nb : 0;
    return true;
  }
  // the piece of the item's last block
  __device__ int64_t last_piece() const { return first + kItemCost + nb - 1; }
  // The first block that reaches past the keys that all rows see: from there on some row has weights of 0, which do not
  // keep infinities and NaN out of a product. The values of these blocks are made finite first.
  __device__ int clean_from() const {
    const int common = p->causal ? max(0, min(x.lk, x.lk - x.lq + 1 + tile * kRows)) : x.lk;
    return common / kBlock;
  }
  // blocks of this share that half h takes part in: [b0, last(h))
  __device__ int last(int h) const { return min(b0 + n, act[h]); }
};

template <class T>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_tc_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_pe,
                      const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Misc& mi = *reinterpret_cast<Misc*>(smem + kMiscAt);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&mi.k_full[i]), 1);
      mbar_init(smem_u32(&mi.v_full[i]), 1);
      mbar_init(smem_u32(&mi.k_empty[i]), 1);
      mbar_init(smem_u32(&mi.v_empty[i]), 1);
    }
    mbar_init(smem_u32(&mi.q_full), 1);
    mbar_init(smem_u32(&mi.q_empty), 1);
    mbar_init(smem_u32(&mi.dirty), 1);
    mbar_init(smem_u32(&mi.clean), 2);
    mbar_init(smem_u32(&mi.end), 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(smem_u32(&mi.s_full[h]), 1);
      mbar_init(smem_u32(&mi.p_full[2 * h]), 4);
      mbar_init(smem_u32(&mi.p_full[2 * h + 1]), 4);
      mbar_init(smem_u32(&mi.o_done[h]), 1);
    }
    mi.stop = mi.never = mi.spoiled = 0;
    mbar_fence_init();
    tma_prefetch(&map_q);
    tma_prefetch(&map_k);
    tma_prefetch(&map_pe);
    tma_prefetch(&map_v);
  }
  if (warp == 9) tmem_alloc(smem_u32(&mi.tmem), 512);
  pdl_entry();

  const int unit = blockIdx.x;
  auto pieces = [&](int r) -> int64_t {
    const PrefillReq x = prefill_req(p, r);
    return x.lq > 0 ? head_pieces(x, p.causal) * p.H : 0;
  };
  const Share share = find_share(pieces, p.R, unit, p.units, mi.scratch, mi.found);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(static_cast<int>(mi.tmem)));  // S of the halves at columns 0 and 128, O at 256 and 384
  const uint32_t stop = smem_u32(&mi.stop);
  constexpr int kFmt = std::is_same<T, bf16>::value ? 1 : 0;
  constexpr uint32_t kIdescS = umma_idesc(kFmt, kFmt, 0, 0, 128, kBlock);
  constexpr uint32_t kIdescO = umma_idesc(kFmt, kFmt, 0, 1, 128, kVal);

  if (warp >= 8) {
    regs_down<kRegsDown>();
    if (warp == 8) {
      // ---- loads ----
      int bad = 0;
      if (unit == 0)
        for (int i = lane; i < p.R; i += 32) bad |= prefill_req(p, i).bad;
      set_flag(p.err, bad);
      Items it(p, share);
      uint32_t items = 0, step = 0;
      const uint32_t k_full = smem_u32(&mi.k_full[0]), v_full = smem_u32(&mi.v_full[0]),
                     k_empty = smem_u32(&mi.k_empty[0]), v_empty = smem_u32(&mi.v_empty[0]);
      // Piece c of block st goes to slot (5 st + c) % 8, where piece c + 2 of block st - 2 was (or c - 3 of st - 1).
      auto wait_old = [&](uint32_t empty, uint32_t back) {
        if (step >= back) mbar_wait(empty + 8 * ((step - back) & 1), (step - back) >> 1 & 1, stop);
        return !stopped(stop);
      };
      auto piece = [&](const CUtensorMap* map, uint32_t full, uint32_t c, int x, int head, int row) {
        if (elect_one())
          tma_load_3d(base + kSlotAt + ((5 * step + c) & (kSlots - 1)) * kPiece, map, full + 8 * (step & 1), x, head, row);
        __syncwarp();
      };
      bool alive = true;
      while (alive && it.next()) {
        if (it.keys == 0) continue;
        if (items > 0) mbar_wait(smem_u32(&mi.q_empty), (items - 1) & 1, stop);
        if (stopped(stop)) break;
        ++items;
        if (elect_one()) {
          const int halves = it.act[1] > 0 ? 2 : 1;
          const uint32_t q_full = smem_u32(&mi.q_full);
          mbar_expect(q_full, halves * 3 * kPiece);
          for (int h = 0; h < halves; ++h)
            for (int c = 0; c < 3; ++c)
              tma_load_3d(base + kQAt + (3 * h + c) * kPiece, &map_q, q_full, 64 * c, it.head,
                          it.x.q0 + it.tile * kRows + h * kHalf);
        }
        __syncwarp();
        // keys that few row tiles share come from HBM (512 rows over 60000 keys: 256 -> 244 us); where many do, they
        // are in L2 and the hints only cost (causal 8192: 525 -> 532 us)
        const bool stream = tiles_of(it.x) <= 4;
        for (int b = it.b0; b < it.b0 + it.n; ++b, ++step) {
          const int row = it.x.k0 + b * kBlock;
          // the pieces of a group share a barrier but come as soon as their own slots are free
          alive = wait_old(k_empty, 2);
          if (!alive) break;
          if (elect_one()) mbar_expect(k_full + 8 * (step & 1), 3 * kPiece);
          __syncwarp();
          piece(&map_k, k_full, 0, 0, it.head, row);
          wait_old(v_empty, 2);
          piece(&map_k, k_full, 1, 64, it.head, row);
          piece(&map_pe, k_full, 2, 0, 0, row);
          alive = wait_old(k_empty, 1);
          if (!alive) {
            ++step;
            break;
          }
          if (elect_one()) mbar_expect(v_full + 8 * (step & 1), 2 * kPiece);
          __syncwarp();
          piece(&map_v, v_full, 3, 0, it.head, row);
          piece(&map_v, v_full, 4, 64, it.head, row);
          if (stream && b + 2 < it.b0 + it.n && elect_one()) {
            // the block after the next on its way into L2: shared memory has room for little more than one
            const int ahead = row + 2 * kBlock;
            tma_prefetch_3d(&map_k, 0, it.head, ahead);
            tma_prefetch_3d(&map_k, 64, it.head, ahead);
            tma_prefetch_3d(&map_v, 0, it.head, ahead);
            tma_prefetch_3d(&map_v, 64, it.head, ahead);
            tma_prefetch_3d(&map_pe, 0, 0, ahead);
          }
          __syncwarp();
        }
      }
      // after a timeout, copies in flight land before the CTA ends (`never` is not set: these waits run on)
      if (stopped(stop)) {
        const uint32_t never = smem_u32(&mi.never);
        for (uint32_t i = 1; i <= 2 && i <= step; ++i) {
          mbar_wait(k_full + 8 * ((step - i) & 1), (step - i) >> 1 & 1, never);
          mbar_wait(v_full + 8 * ((step - i) & 1), (step - i) >> 1 & 1, never);
        }
        if (items > 0) mbar_wait(smem_u32(&mi.q_full), (items - 1) & 1, never);
      }
    } else if (warp == 9) {
      // ---- products ----
      Items it(p, share);
      const uint32_t k_full = smem_u32(&mi.k_full[0]), v_full = smem_u32(&mi.v_full[0]), k_empty = smem_u32(&mi.k_empty[0]),
                     v_empty = smem_u32(&mi.v_empty[0]), s_full = smem_u32(&mi.s_full[0]),
                     p_full = smem_u32(&mi.p_full[0]), o_done = smem_u32(&mi.o_done[0]);
      // piece c of step st in the ring: 5 pieces a step (counted modulo 2^32, a multiple of the ring)
      auto slot_of = [](uint32_t st, uint32_t c) { return (5 * st + c) & (kSlots - 1); };
      auto wait_block = [&](uint32_t full, uint32_t st) { mbar_wait(full + 8 * (st & 1), st >> 1 & 1, stop); };
      // S of half h for the block of step st
      auto scores = [&](int h, uint32_t st) {
        if (elect_one()) {
#pragma unroll
          for (uint32_t c = 0; c < 3; ++c) {
            const uint64_t qa = umma_desc(base + kQAt + (3 * h + c) * kPiece, 16, 1024);
            const uint64_t ka = umma_desc(base + kSlotAt + slot_of(st, c) * kPiece, 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 32 bytes of K each
              umma_ss<false>(tmem + h * kBlock, qa + 2 * k, ka + 2 * k, kIdescS, c > 0 || k > 0);
          }
          umma_commit(s_full + 8 * h);
        }
        __syncwarp();
      };
      // O of half h: the products with keys 64 w to 64 w + 63 of the block
      auto values = [&](int h, int w, uint32_t st, bool first) {
        // the two 64-value pieces of V are two slots, which may wrap around the ring: a product of 64 each then
        const uint32_t d = tmem + 256 + h * kVal, a = tmem + h * kBlock + 32 * w;
        const uint64_t v0 = umma_desc(base + kSlotAt + slot_of(st, 3) * kPiece + w * 8192, kPiece, 1024);
        if (slot_of(st, 4) != 0) {
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_ts(d, a + 8 * k, v0 + 128 * k, kIdescO, !first || w > 0 || k > 0);
            if (w == 1) umma_commit(o_done + 8 * h);
          }
        } else {
          const uint64_t v1 = umma_desc(base + kSlotAt + w * 8192, kPiece, 1024);
          constexpr uint32_t kIdescHalf = umma_idesc(kFmt, kFmt, 0, 1, 128, 64);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              umma_ts(d, a + 8 * k, v0 + 128 * k, kIdescHalf, !first || w > 0 || k > 0);
              umma_ts(d + 64, a + 8 * k, v1 + 128 * k, kIdescHalf, !first || w > 0 || k > 0);
            }
            if (w == 1) umma_commit(o_done + 8 * h);
          }
        }
        __syncwarp();
      };
      uint32_t items = 0, cleans = 0;
      uint32_t step = 0;   // blocks begun
      uint32_t taken = 0;  // parity of the weights taken, a bit a half
      while (uniform(it.next())) {
        if (uniform(it.keys) == 0) continue;
        mbar_wait(smem_u32(&mi.q_full), items++ & 1, stop);
        const int end = uniform(it.b0 + it.n), begin = uniform(it.b0);
        const int clean_from = uniform(it.clean_from());
        // Warps 10 and 11 may look at the values of the block after those that were waited for last: one block at a time,
        // so that neither side falls two phases behind.
        auto clean_next = [&]() {
          if (elect_one()) mbar_arrive(smem_u32(&mi.dirty));
          __syncwarp();
        };
        if (begin >= clean_from) clean_next();
        const int last0 = uniform(it.last(0)), last1 = uniform(it.last(1));
        wait_block(k_full, step);
        tmem_fence_after();
        if (begin < last0) scores(0, step);
        if (begin < last1) scores(1, step);
        if (elect_one()) {
          umma_commit(k_empty + 8 * (step & 1));
          if (begin + 1 == end) umma_commit(smem_u32(&mi.q_empty));
        }
        __syncwarp();
        for (int b = begin; b < end; ++b, ++step) {
          const bool more = b + 1 < end;
          wait_block(v_full, step);
          if (b >= clean_from) mbar_wait(smem_u32(&mi.clean), cleans++ & 1, stop);
          if (more && b + 1 >= clean_from) clean_next();  // early, so that it does not wait: the values are there before
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int last = h ? last1 : last0;
            if (b < last) {
              mbar_wait(p_full + 16 * h, taken >> h & 1, stop);
              tmem_fence_after();
              values(h, 0, step, b == begin);
              mbar_wait(p_full + 16 * h + 8, taken >> h & 1, stop);
              tmem_fence_after();
              values(h, 1, step, b == begin);
              taken ^= 1u << h;
            }
            if (h == 0 && more) {
              wait_block(k_full, step + 1);
              tmem_fence_after();
            }
            if (b + 1 < last) scores(h, step + 1);
          }
          if (elect_one()) {
            umma_commit(v_empty + 8 * (step & 1));
            if (more) umma_commit(k_empty + 8 * ((step + 1) & 1));
            if (b + 2 == end) umma_commit(smem_u32(&mi.q_empty));
          }
          __syncwarp();
        }
      }
      // everything issued ends before the tensor memory is given back
      if (elect_one()) umma_commit(smem_u32(&mi.end));
      __syncwarp();
      mbar_wait(smem_u32(&mi.end), 0, smem_u32(&mi.never));
    } else {
      // ---- values that must not meet a weight of 0: warp 10 takes the first piece of a block, warp 11 the second ----
      Items it(p, share);
      uint32_t step = 0, cleans = 0;
      while (it.next()) {
        if (it.keys == 0) continue;
        const int clean_from = max(it.b0, it.clean_from()), end = it.b0 + it.n;
        step += max(0, min(clean_from, end) - it.b0);
        for (int b = clean_from; b < end; ++b, ++step) {
          mbar_wait(smem_u32(&mi.dirty), cleans++ & 1, stop);
          mbar_wait(smem_u32(&mi.v_full[0]) + 8 * (step & 1), step >> 1 & 1, stop);
          const int slot = static_cast<int>((5 * step + warp - 7) & (kSlots - 1));
          uint4* at = reinterpret_cast<uint4*>(smem + kSlotAt + slot * kPiece);
          const int first = min(kBlock, it.x.lk - b * kBlock);  // rows that belong to the request: the others are 0
          for (int i = first * 8 + lane; i < kBlock * 8; i += 32) at[i] = make_uint4(0, 0, 0, 0);
          if (p.causal) {
            uint32_t odd = 0;
#pragma unroll 8
            for (int i = lane; i < first * 8; i += 32) {
              const uint4 v = at[i];
              odd |= nonfinite<T>(v.x) | nonfinite<T>(v.y) | nonfinite<T>(v.z) | nonfinite<T>(v.w);
            }
            if (__any_sync(0xffffffffu, odd != 0)) {
              for (int i = lane; i < first * 8; i += 32) at[i] = only_finite<T>(at[i]);
              if (lane == 0) *reinterpret_cast<volatile int32_t*>(&mi.spoiled) = 1;
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&mi.clean));
        }
      }
    }
  } else {
    regs_up<kRegsUp>();
    // ---- softmax and epilogue of half h: thread = row ----
    const int h = warp >> 2;
    const int row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + h * kBlock + lanes, o_at = tmem + 256 + h * kVal + lanes;
    const float sc = p.sm_scale * kLog2e;
    constexpr float kFirst = std::is_same<T, f16>::value ? 8.0f : 0.0f;  // where a new reference puts the largest weight
    constexpr float kCap = std::is_same<T, f16>::value ? 15.0f : 8.0f;   // weights stay below 2^kCap
    JoinNote note{-1, 0, 0, 0};
    Items it(p, share);
    uint32_t count = 0;  // blocks taken part in
    while (it.next()) {
      const int i0 = it.tile * kRows + h * kHalf;        // first row of this half within the request
      const int64_t i = i0 + row;
      const int limit = p.causal ? static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(it.x.lk), it.x.lk - it.x.lq + 1 + i)))
                                 : it.x.lk;               // keys this row sees
      // the fewest keys any row of this warp sees
      const int low = __reduce_min_sync(0xffffffffu, limit);
      float ref = -INFINITY, l = 0.0f;
      const int last = it.last(h);
      for (int b = it.b0; b < last; ++b, ++count) {
        mbar_wait(smem_u32(&mi.s_full[h]), count & 1, stop);
        __syncwarp();
        tmem_fence_after();
        uint32_t raw_s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, raw_s + 32 * c);
        tmem_wait_ld();
        tmem_pin<128>(raw_s);
        float* s = reinterpret_cast<float*>(raw_s);
        const int j0 = b * kBlock;
        if (low - j0 < kBlock) {
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if (j0 + k >= limit) s[k] = -INFINITY;
        }
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) m4[c] = max3(s[3 * c], s[3 * c + 1], s[3 * c + 2]);
#pragma unroll
        for (int k = 12; k < 128; k += 2) m4[(k >> 1) & 3] = max3(m4[(k >> 1) & 3], s[k], s[k + 1]);
        const float top = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * sc;
        if (__any_sync(0xffffffffu, top > ref + kCap)) {
          float a = 1.0f;
          const float next = top - kFirst;
          if (next > ref) {
            a = ref == -INFINITY ? 0.0f : ex2(ref - next);
            ref = next;
          }
          l *= a;
          if (b > it.b0) {
            mbar_wait(smem_u32(&mi.o_done[h]), (count - 1) & 1, stop);
            __syncwarp();
            tmem_fence_after();
#pragma unroll 1
            for (int c = 0; c < kVal; c += 16) {
              uint32_t o[16];
              tmem_ld16(o_at + c, o);
              tmem_wait_ld();
              tmem_pin<16>(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
              tmem_st16(o_at + c, o);
            }
          }
        }
        const float r = ref == -INFINITY ? 0.0f : ref;
        const float2 sc2 = make_float2(sc, sc), r2 = make_float2(-r, -r);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float2 x = fma2(make_float2(s[32 * c + 2 * k], s[32 * c + 2 * k + 1]), sc2, r2);
            x = make_float2(ex2(x.x), ex2(x.y));
            sum[k & 1] = add2(sum[k & 1], x);
            w[k] = pack2<T>(x.x, x.y);
          }
          tmem_st16(s_at + 16 * c, w);
          if (c & 1) {  // 64 keys' weights are there: their products may begin
            tmem_wait_st();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&mi.p_full[2 * h + (c >> 1)]));
          }
        }
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
      }

      // epilogue
      const bool whole = it.b0 == 0 && it.n == it.nb;
      const bool some = last > it.b0;
      if (some) {
        mbar_wait(smem_u32(&mi.o_done[h]), (count - 1) & 1, stop);
        __syncwarp();
        tmem_fence_after();
      }
      if (stopped(stop)) l = __uint_as_float(0x7fffffffu);  // a NaN for the row's result and log sum, split or whole
      if (some && *reinterpret_cast<volatile int32_t*>(&mi.spoiled) != 0) {
        // infinities and NaN that were kept out of the products, for the rows that see them
        const int lo = max(it.b0, it.clean_from()) * kBlock;
        const int hi = static_cast<int>(min(static_cast<int64_t>(limit), static_cast<int64_t>(last) * kBlock));
        const T* v0 = static_cast<const T*>(p.v) + static_cast<int64_t>(it.x.k0) * p.vt_stride + it.head * p.vh_stride;
#pragma unroll 1
        for (int c = 0; c < kVal; c += 16) {
          uint32_t o[16];
          __syncwarp();
          tmem_ld16(o_at + c, o);
          tmem_wait_ld();
          tmem_pin<16>(o);
#pragma unroll 1
          for (int j = lo; j < hi; ++j) {
            const uint4* v = reinterpret_cast<const uint4*>(v0 + static_cast<int64_t>(j) * p.vt_stride + c);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t odd = nonfinite<T>(w[k]);
                const float2 two = unpack2<T>(w[k]);
                if (odd & 0xffff) o[8 * q + 2 * k] = __float_as_uint(__uint_as_float(o[8 * q + 2 * k]) + two.x);
                if (odd >> 16) o[8 * q + 2 * k + 1] = __float_as_uint(__uint_as_float(o[8 * q + 2 * k + 1]) + two.y);
              }
            }
          }
          __syncwarp();
          tmem_st16(o_at + c, o);
          tmem_wait_st();
        }
      }
      const bool mine = i < it.x.lq;
      if (!whole && it.b0 == 0 && tid == 0) {
        note.item = it.r;
        note.head = it.head;
        note.tile = it.tile;
        note.parts = unit_of(it.last_piece(), share.total, share.units) - unit + 1;
      }
      float* slot = p.ws.slots + (static_cast<int64_t>(unit) * 2 + (it.b0 == 0 ? 1 : 0)) * kSlotFloats;
      const int64_t t = it.x.q0 + i;
      float now = l != 0.0f ? 1.0f / l : 0.0f, before = 0.0f;
      if (whole && mine) {
        float lse = l != 0.0f ? (ref + log2f(l)) * kLn2 : -INFINITY;
        if (p.prev_lse != nullptr) {
          const Joined g = join_state(lse, p.prev_lse[t * p.H + it.head]);
          now *= g.now;
          before = g.before;
          lse = g.lse;
        }
        if (p.lse != nullptr) p.lse[t * p.H + it.head] = lse;
      } else if (!whole) {
        float* ml = slot + kRows * kSlotRow + 2 * (h * kHalf + row);
        ml[0] = ref;
        ml[1] = l;
      }
      __syncwarp();
#pragma unroll 1
      for (int c = 0; c < kVal; c += 16) {
        uint32_t o[16];
        __syncwarp();
        if (some) {
          tmem_ld16(o_at + c, o);
          tmem_wait_ld();
          tmem_pin<16>(o);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = 0;
        }
        if (!mine) continue;
        if (whole) {
          float y[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] = __uint_as_float(o[k]) * now;
          if (before != 0.0f) {
            const uint4* prev = reinterpret_cast<const uint4*>(static_cast<const T*>(p.prev) + t * p.pt_stride +
                                                               it.head * p.ph_stride + c);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint4 v = prev[q];
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                T e;
                const unsigned short bits = static_cast<unsigned short>(k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xffff);
                memcpy(&e, &bits, 2);
                y[8 * q + k] += before * to_f(e);
              }
            }
          }
          uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + t * p.ot_stride + it.head * p.oh_stride + c);
          out[0] = make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
          out[1] = make_uint4(pack2<T>(y[8], y[9]), pack2<T>(y[10], y[11]), pack2<T>(y[12], y[13]), pack2<T>(y[14], y[15]));
        } else {
          float4* at = reinterpret_cast<float4*>(slot + (h * kHalf + row) * kSlotRow + c);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            at[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]), __uint_as_float(o[4 * k + 2]),
                                __uint_as_float(o[4 * k + 3]));
        }
      }
      tmem_fence_before();
    }
    if (tid == 0) p.ws.notes[unit] = note;
    if (stopped(stop) && tid == 0) set_flag(p.err, PMG_FLAG_TIMEOUT);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 9) tmem_free(tmem, 512);
}

template <class T>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtasPerSm) prefill_join_kernel(const __grid_constant__ PrefillParams p) {
  pdl_entry();
  join_rows(
      p.ws, p.units, 1, kRows, kVal, kSlotFloats,
      [&](const JoinNote& note, int, int row) { return note.tile * kRows + row < prefill_req(p, note.item).lq; },
      [&](const JoinNote& note, int, int row, int d, const float4& a, float top, float l) {
        const int64_t t = static_cast<int64_t>(prefill_req(p, note.item).q0) + note.tile * kRows + row;
        float lse = l != 0.0f ? (top + log2f(l)) * kLn2 : -INFINITY;
        float now = l != 0.0f ? 1.0f / l : 0.0f, before = 0.0f;
        if (p.prev_lse != nullptr) {
          const Joined g = join_state(lse, p.prev_lse[t * p.H + note.head]);
          now *= g.now;
          before = g.before;
          lse = g.lse;
        }
        __syncwarp();  // every lane has read prev_lse, which lse may be
        if (d == 0 && p.lse != nullptr) p.lse[t * p.H + note.head] = lse;
        float y[4] = {a.x * now, a.y * now, a.z * now, a.w * now};
        if (before != 0.0f) {
          const T* prev = static_cast<const T*>(p.prev) + t * p.pt_stride + note.head * p.ph_stride + d;
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] += before * to_f(prev[k]);
        }
        T* out = static_cast<T*>(p.out) + t * p.ot_stride + note.head * p.oh_stride + d;
        *reinterpret_cast<uint2*>(out) = make_uint2(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]));
      });
}

template <class T>
int run(const PrefillParams& p, const CUtensorMap* maps, void* stream) {
  auto k = prefill_tc_kernel<T>;
  int st = allow_smem(reinterpret_cast<const void*>(k), kBytes);
  if (st != PMG_OK) return st;
  st = launch(k, dim3(static_cast<unsigned>(p.units)), kThreads, kBytes, stream, p, maps[0], maps[1], maps[2], maps[3]);
  if (st != PMG_OK) return st;
  return launch(prefill_join_kernel<T>, dim3(static_cast<unsigned>(kJoinCtasPerSm * p.units)), kJoinThreads, 0, stream, p);
}

}  // namespace

bool prefill_tc_takes(const PrefillParams& p, int dtype) {
  auto rows = [](const void* base, int64_t s0, int64_t s1) {
    return aligned(base, 16) && s0 % 8 == 0 && s1 % 8 == 0 && s0 * 2 < (int64_t{1} << 40) && s1 * 2 < (int64_t{1} << 40);
  };
  return p.dn == kNope && p.dr == kRope && p.dv == kVal && (dtype == PMG_BF16 || dtype == PMG_FP16) && p.Tk > 0 &&
         p.sm_scale > 0.0f && rows(p.q, p.qt_stride, p.qh_stride) && rows(p.k, p.kt_stride, p.kh_stride) &&
         rows(p.pe, p.pe_stride, 0) && rows(p.v, p.vt_stride, p.vh_stride) && rows(p.out, p.ot_stride, p.oh_stride) &&
         (p.prev == nullptr || rows(p.prev, p.pt_stride, p.ph_stride)) &&
         // a stride of 0 (one row for all) has no tensor map
         (p.qt_stride > 0 || p.Tq == 1) && (p.qh_stride > 0 || p.H == 1) && (p.kt_stride > 0 || p.Tk == 1) &&
         (p.kh_stride > 0 || p.H == 1) && (p.vt_stride > 0 || p.Tk == 1) && (p.vh_stride > 0 || p.H == 1) &&
         (p.pe_stride > 0 || p.Tk == 1);
}

int prefill_tc(PrefillParams& p, int dtype, int sms, void* stream) {
  p.units = sms;
  const CUtensorMapDataType type = dtype == PMG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap maps[4];
  auto map = [&](CUtensorMap* m, const void* at, int dim, int heads, int rows, int64_t head_stride, int64_t row_stride) {
    // the stride of a dimension of one is not used; it has to be a valid one all the same
    const uint64_t s1 = heads > 1 ? static_cast<uint64_t>(head_stride) * 2 : 512;
    const uint64_t s2 = rows > 1 ? static_cast<uint64_t>(row_stride) * 2 : 512;
    return tensor_map<3>(m, type, at, {static_cast<uint64_t>(dim), static_cast<uint64_t>(heads), static_cast<uint64_t>(rows)},
                         {s1, s2}, {64, 1, 128});
  };
  int st = map(&maps[0], p.q, kNope + kRope, p.H, p.Tq, p.qh_stride, p.qt_stride);
  if (st == PMG_OK) st = map(&maps[1], p.k, kNope, p.H, p.Tk, p.kh_stride, p.kt_stride);
  if (st == PMG_OK) st = map(&maps[2], p.pe, kRope, 1, p.Tk, 0, p.pe_stride);
  if (st == PMG_OK) st = map(&maps[3], p.v, kVal, p.H, p.Tk, p.vh_stride, p.vt_stride);
  if (st != PMG_OK) return st;
  return dtype == PMG_BF16 ? run<bf16>(p, maps, stream) : run<f16>(p, maps, stream);
}

}  // namespace pmg_mla
