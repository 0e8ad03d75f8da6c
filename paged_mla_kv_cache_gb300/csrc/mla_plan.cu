// Block tables, slots and positions of one serving step (pmg_plan_step).
//
// Mathematics: with end = ctx + new, first = ceil(ctx / B) and need =
// ceil(end / B) - first, request r's fresh page j is free[need_0 + ... +
// need_{r-1} + j], and new token t of request r (t counted over all requests)
// sits at position p = ctx_r + t - cu_new[r], in page p / B: a cached page of
// the table where p / B < first, a fresh one otherwise. So slots never wait
// for the table: every thread finds a page's id from the prefix sums alone.
//
// One launch. Requests are taken in groups of 4096, whose prefix sums fit in
// shared memory; a CTA first adds up the groups before its own (64-bit sums),
// scans its own, and then writes its slice of the group's tokens and pages
// with a binary search over the prefix sums. Latency bound: reading the
// lengths, a scan, one dependent read of an id. The scan is repeated by every
// slice instead of passed on: a second launch would cost more than 32 KB read
// from L2. Measured: 2048 ragged requests with 170000 new tokens 10.9 us (3 MB),
// 64 requests of one token 8.1 us, the host's call and one launch. 2048 tokens a
// CTA; 512, 1024, 4096 and 8192 measured slower.
#include <algorithm>

#include "mla_common.cuh"

namespace pmg_mla {
namespace {

constexpr int kThreads = 512;
constexpr int kGroup = 4096;               // requests of one group
constexpr int kPer = kGroup / kThreads;    // requests a thread scans
constexpr int kBatch = 4;                  // tokens of a thread whose page ids are looked up together
constexpr int kTokensPerCta = kBatch * kThreads;

struct PlanParams {
  const int32_t* ctx;
  const int32_t* fresh;  // new lengths
  int32_t R;
  int32_t* bt;
  int64_t bt_stride;
  const int32_t* free_ids;
  int64_t num_free;
  int64_t num_blocks;
  int32_t B;
  int64_t* slots;
  int32_t* positions;
  int32_t* t2s;
  int64_t max_tokens;
  int32_t* cu_new;
  int32_t* seq_lens;
  int32_t* cu_seq;
  int32_t* taken;
  int32_t* err;
  int32_t slices;  // CTAs of a group
  uint32_t magic;  // division by B
  int32_t shift;
};

struct Lens {
  int32_t ctx, fresh;
  int bad;
};

__device__ __forceinline__ Lens lens_of(const PlanParams& p, int64_t r) {
  Lens l{p.ctx[r], p.fresh[r], 0};
  if (l.ctx < 0 || l.fresh < 0) l.bad = PMG_FLAG_LENGTH;
  l.ctx = max(l.ctx, 0);
  l.fresh = max(l.fresh, 0);
  if (l.fresh > INT32_MAX - l.ctx) {
    l.fresh = INT32_MAX - l.ctx;
    l.bad = PMG_FLAG_LENGTH;
  }
  return l;
}

// n / B by one multiply-high, an add and a shift (the invariant-divisor method
// of Granlund and Montgomery, 1994); the host computes magic and shift. Every
// CTA divides twice a request: as plain divisions that took half the kernel.
__device__ __forceinline__ uint32_t page_of(const PlanParams& p, uint32_t n) {
  return static_cast<uint32_t>((static_cast<uint64_t>(__umulhi(p.magic, n)) + n) >> p.shift);
}
__device__ __forceinline__ uint32_t pages_of(const PlanParams& p, uint32_t len) {
  return len == 0 ? 0 : page_of(p, len - 1) + 1;
}

__device__ __forceinline__ int32_t cut(int64_t x) { return static_cast<int32_t>(x < INT32_MAX ? x : INT32_MAX); }

// Exclusive prefix sums of three values over the threads of the block, and the totals.
struct Sums {
  int64_t fresh, seq, page;
};
__device__ __forceinline__ Sums scan_sums(const Sums& x, Sums* scratch, Sums& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, inc.fresh, o), b = __shfl_up_sync(0xffffffffu, inc.seq, o),
                  c = __shfl_up_sync(0xffffffffu, inc.page, o);
    if (lane >= o) {
      inc.fresh += a;
      inc.seq += b;
      inc.page += c;
    }
  }
  __syncthreads();  // scratch is free again
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  Sums before{0, 0, 0};
  all = Sums{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const Sums y = scratch[w];
    if (w == warp) before = all;
    all.fresh += y.fresh;
    all.seq += y.seq;
    all.page += y.page;
  }
  return {before.fresh + inc.fresh - x.fresh, before.seq + inc.seq - x.seq, before.page + inc.page - x.page};
}

// A thread scans kPer neighbours: with one place left out after each kPer, the
// threads of a warp write different banks.
__device__ __forceinline__ int place(int k) { return k + k / kPer; }
constexpr int kPlaces = kGroup + kGroup / kPer + 1;

// last i in [0, n) with a[place(i)] <= key, where the first one is
__device__ __forceinline__ int find(const int64_t* a, int n, int64_t key) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[place(mid)] <= key) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_step_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  int64_t* cu = reinterpret_cast<int64_t*>(smem);   // first new token of each request, by place()
  int64_t* pg = cu + kPlaces;                  // first fresh page of each request
  int32_t* ctx = reinterpret_cast<int32_t*>(pg + kPlaces);  // cached tokens
  __shared__ Sums scratch[kThreads / 32];
  pdl_entry();

  const int group = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
  const int64_t r0 = static_cast<int64_t>(group) * kGroup;
  const int n = static_cast<int>(min(static_cast<int64_t>(kGroup), p.R - r0));
  const uint32_t B = static_cast<uint32_t>(p.B);
  int bad = 0;

  // the groups before this one
  int64_t base_new = 0, base_seq = 0, base_page = 0;
  if (r0 > 0) {
    Sums x{0, 0, 0}, all;
    for (int64_t r = threadIdx.x; r < r0; r += kThreads) {
      const Lens l = lens_of(p, r);
      x.fresh += l.fresh;
      x.seq += static_cast<int64_t>(l.ctx) + l.fresh;
      x.page += pages_of(p, l.ctx + l.fresh) - pages_of(p, l.ctx);
    }
    scan_sums(x, scratch, all);
    base_new = all.fresh;
    base_seq = all.seq;
    base_page = all.page;
  }

  // this group's lengths into shared memory (the new ones in the page sums' place for now); then each thread owns kPer
  // consecutive requests
  int32_t* fresh = reinterpret_cast<int32_t*>(pg);
  for (int k = threadIdx.x; k < n; k += kThreads) {
    const Lens l = lens_of(p, r0 + k);
    bad |= l.bad;
    ctx[place(k)] = l.ctx;
    fresh[place(k)] = l.fresh;
  }
  __syncthreads();
  Sums mine{0, 0, 0};
  int32_t own_ctx[kPer], own_new[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = static_cast<int>(threadIdx.x) * kPer + i;
    own_ctx[i] = k < n ? ctx[place(k)] : 0;
    own_new[i] = k < n ? fresh[place(k)] : 0;
    mine.fresh += own_new[i];
    mine.seq += static_cast<int64_t>(own_ctx[i]) + own_new[i];
    mine.page += pages_of(p, own_ctx[i] + own_new[i]) - pages_of(p, own_ctx[i]);
  }
  Sums all;
  const Sums before = scan_sums(mine, scratch, all);  // (its barriers come before the page sums are written)
  const int64_t tn = all.fresh, ts = all.seq, tp = all.page;
  int64_t cn = base_new + before.fresh, cs = base_seq + before.seq, cp = base_page + before.page;
  const bool writer = slice == 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = static_cast<int>(threadIdx.x) * kPer + i;
    if (k < n) {
      cu[place(k)] = cn;
      pg[place(k)] = cp;
      if (writer) {
        p.cu_new[r0 + k] = cut(cn);
        if (p.cu_seq != nullptr) p.cu_seq[r0 + k] = cut(cs);
        p.seq_lens[r0 + k] = own_ctx[i] + own_new[i];
      }
    }
    cn += own_new[i];
    cs += static_cast<int64_t>(own_ctx[i]) + own_new[i];
    cp += pages_of(p, own_ctx[i] + own_new[i]) - pages_of(p, own_ctx[i]);
  }
  const int64_t end_new = base_new + tn, end_page = base_page + tp;
  const bool last = r0 + n == p.R;
  if (threadIdx.x == 0) {
    if (writer && last) {
      p.cu_new[p.R] = cut(end_new);
      if (p.cu_seq != nullptr) p.cu_seq[p.R] = cut(base_seq + ts);
      if (p.taken != nullptr) *p.taken = cut(min(end_page, p.num_free));
      if (end_new > p.max_tokens || end_new > INT32_MAX || base_seq + ts > INT32_MAX) bad |= PMG_FLAG_CAPACITY;
    }
  }
  __syncthreads();

  // fresh pages of this slice
  {
    const int64_t lo = base_page + tp * slice / p.slices, hi = base_page + tp * (slice + 1) / p.slices;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
      const int k = find(pg, n, i);
      const int64_t column = pages_of(p, ctx[place(k)]) + (i - pg[place(k)]);
      int32_t id = -1;
      if (i >= p.num_free) {
        bad |= PMG_FLAG_NO_BLOCKS;
      } else {
        id = p.free_ids[i];
        if (id < 0 || id >= p.num_blocks) {
          bad |= PMG_FLAG_PHYS_BLOCK;
          id = -1;
        }
      }
      if (column < p.bt_stride) p.bt[(r0 + k) * p.bt_stride + column] = id;
      else bad |= PMG_FLAG_LOGICAL_BLOCK;
    }
  }

  // new tokens of this slice, and the rows past the last token
  if (p.max_tokens > 0 && (p.slots != nullptr || p.positions != nullptr || p.t2s != nullptr)) {
    const int64_t begin = min(base_new, p.max_tokens), end = last ? p.max_tokens : min(end_new, p.max_tokens);
    const int64_t span = end - begin;
    const int64_t lo = begin + span * slice / p.slices, hi = begin + span * (slice + 1) / p.slices;
    // a warp takes 32 kBatch neighbouring tokens: one search for the first, then the requests that begin among the next 32
    const int lane = threadIdx.x & 31;
    for (int64_t w0 = lo + (threadIdx.x >> 5) * (32 * kBatch); w0 < hi; w0 += kBatch * kThreads) {
      int64_t id[kBatch];
      int32_t pos[kBatch], seq[kBatch];
      uint32_t in_page[kBatch];
      int k0 = w0 < end_new ? find(cu, n, w0) : 0;
      // every look-up before the first store
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int64_t tw = w0 + 32 * j, t = tw + lane;
        id[j] = -1;
        pos[j] = seq[j] = -1;
        in_page[j] = 0;
        // token `lane` is in request k0 + c: c beginnings of the next 32 requests are not after it
        const int64_t begin_k = k0 + 1 + lane < n ? cu[place(k0 + 1 + lane)] - tw : 32;
        const int rel = static_cast<int>(min(begin_k, int64_t{32}));
        int c = 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (__shfl_sync(0xffffffffu, rel, c + o - 1) <= lane) c += o;
        if (__shfl_sync(0xffffffffu, rel, 31) <= lane) c = 32;  // (the search ends at 31)
        const int k = c < 32 || t >= end_new ? k0 + c : find(cu, n, t);
        k0 = __shfl_sync(0xffffffffu, k, 31);
        if (t >= hi || t >= end_new) continue;
        seq[j] = static_cast<int32_t>(r0 + k);
        const uint32_t at = static_cast<uint32_t>(ctx[place(k)]) + static_cast<uint32_t>(t - cu[place(k)]);
        pos[j] = static_cast<int32_t>(at);
        if (p.slots == nullptr) continue;
        const uint32_t page = page_of(p, at), first = pages_of(p, ctx[place(k)]);
        in_page[j] = at - page * B;
        if (page >= p.bt_stride) {
          bad |= PMG_FLAG_LOGICAL_BLOCK;
        } else if (page >= first) {
          const int64_t i = pg[place(k)] + (page - first);
          if (i < p.num_free) id[j] = p.free_ids[i];
          if (id[j] >= p.num_blocks) id[j] = -1;  // reported where the table is written
        } else {
          id[j] = p.bt[static_cast<int64_t>(seq[j]) * p.bt_stride + page];
          if (id[j] < 0 || id[j] >= p.num_blocks) {
            bad |= PMG_FLAG_PHYS_BLOCK;
            id[j] = -1;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int64_t t = w0 + 32 * j + lane;
        if (t >= hi) continue;
        if (p.slots != nullptr) p.slots[t] = id[j] < 0 ? -1 : id[j] * p.B + in_page[j];
        if (p.positions != nullptr) p.positions[t] = pos[j];
        if (p.t2s != nullptr) p.t2s[t] = seq[j];
      }
    }
  }
  set_flag(p.err, bad);
}

constexpr int kSmem = kPlaces * 20;

struct Bytes {
  const void* at;
  int64_t n;
};
bool overlap(const Bytes& a, const Bytes& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.at != nullptr && b.at != nullptr && a.n > 0 && b.n > 0 && x < y + static_cast<uintptr_t>(b.n) &&
         y < x + static_cast<uintptr_t>(a.n);
}

}  // namespace
}  // namespace pmg_mla

extern "C" int pmg_plan_step(const int32_t* ctx_lens, const int32_t* new_lens, int32_t num_reqs, int32_t* block_table,
                             int64_t block_table_stride, const int32_t* free_blocks, int64_t num_free,
                             int64_t num_blocks, int32_t block_size, int64_t* slots, int32_t* positions,
                             int32_t* token_to_seq, int64_t max_tokens, int32_t* cu_new, int32_t* seq_lens,
                             int32_t* cu_seq, int32_t* blocks_taken, int32_t* error_flag, void* stream) {
  using namespace pmg_mla;
  if (num_reqs < 0 || block_table_stride < 0 || num_free < 0 || num_blocks < 0 || block_size < 1 || max_tokens < 0)
    return PMG_ERR_ARG;
  if (num_reqs > PMG_MAX_REQS || max_tokens > INT32_MAX || num_blocks > INT32_MAX || num_free > INT32_MAX ||
      block_table_stride > INT32_MAX)
    return PMG_ERR_UNSUPPORTED;
  if (cu_new == nullptr) return PMG_ERR_NULL;
  if (num_reqs > 0 && (ctx_lens == nullptr || new_lens == nullptr || seq_lens == nullptr ||
                       (block_table == nullptr && block_table_stride > 0) || (free_blocks == nullptr && num_free > 0)))
    return PMG_ERR_NULL;
  if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) || !aligned(free_blocks, 4) ||
      !aligned(slots, 8) || !aligned(positions, 4) || !aligned(token_to_seq, 4) || !aligned(cu_new, 4) ||
      !aligned(seq_lens, 4) || !aligned(cu_seq, 4) || !aligned(blocks_taken, 4) || !aligned(error_flag, 4))
    return PMG_ERR_ALIGN;
  // CTAs that have not begun yet read the lengths and the free ids while others write their results
  const int64_t r = num_reqs;
  for (const Bytes& in : {Bytes{ctx_lens, 4 * r}, Bytes{new_lens, 4 * r}, Bytes{free_blocks, 4 * num_free}})
    for (const Bytes& out : {Bytes{block_table, 4 * r * block_table_stride}, Bytes{slots, 8 * max_tokens},
                             Bytes{positions, 4 * max_tokens}, Bytes{token_to_seq, 4 * max_tokens},
                             Bytes{cu_new, 4 * (r + 1)}, Bytes{seq_lens, 4 * r}, Bytes{cu_seq, 4 * (r + 1)},
                             Bytes{blocks_taken, 4}, Bytes{error_flag, 4}})
      if (overlap(in, out)) return PMG_ERR_ARG;
  PlanParams p{ctx_lens, new_lens, num_reqs, block_table, block_table_stride, free_blocks, num_free, num_blocks,
               block_size, slots, positions, token_to_seq, max_tokens, cu_new, seq_lens, cu_seq, blocks_taken,
               error_flag, 1, 0, 0};
  uint32_t l = 0;
  while ((1ull << l) < static_cast<uint64_t>(block_size)) ++l;
  p.magic = static_cast<uint32_t>((((1ull << l) - static_cast<uint64_t>(block_size)) << 32) / static_cast<uint64_t>(block_size) + 1);
  p.shift = static_cast<int32_t>(l);
  int sms = 0;
  int st = sm_count(&sms);
  if (st == PMG_OK) st = allow_smem(reinterpret_cast<const void*>(plan_step_kernel), kSmem);
  if (st != PMG_OK) return st;
  const int64_t groups = std::max<int64_t>(1, (static_cast<int64_t>(num_reqs) + kGroup - 1) / kGroup);
  const int64_t want = (max_tokens + kTokensPerCta * groups - 1) / (kTokensPerCta * groups);
  p.slices = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(want, std::max<int64_t>(1, 2 * sms / groups))));
  return launch(plan_step_kernel, dim3(static_cast<unsigned>(groups * p.slices)), kThreads, kSmem, stream, p);
}
