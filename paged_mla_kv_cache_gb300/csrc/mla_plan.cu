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
// slice instead of passed on: a second launch would cost more than 16 KB read
// from L2.
#include <algorithm>

#include "mla_common.cuh"

namespace pmg_mla {
namespace {

constexpr int kThreads = 512;
constexpr int kGroup = 4096;               // requests of one group
constexpr int kPer = kGroup / kThreads;    // requests a thread scans
constexpr int kTokensPerCta = 2048;

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

__device__ __forceinline__ uint32_t pages_of(uint32_t len, uint32_t B) { return len / B + (len % B != 0 ? 1u : 0u); }

__device__ __forceinline__ int32_t cut(int64_t x) { return static_cast<int32_t>(x < INT32_MAX ? x : INT32_MAX); }

// last i in [0, n) with a[i] <= key, where a[0] <= key
__device__ __forceinline__ int find(const int64_t* a, int n, int64_t key) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= key) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_step_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  int64_t* cu = reinterpret_cast<int64_t*>(smem);   // [n + 1] first new token of each request
  int64_t* pg = cu + (kGroup + 1);                  // [n + 1] first fresh page of each request
  int32_t* ctx = reinterpret_cast<int32_t*>(pg + (kGroup + 1));  // [n]
  __shared__ int64_t scratch[33];
  pdl_entry();

  const int group = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
  const int64_t r0 = static_cast<int64_t>(group) * kGroup;
  const int n = static_cast<int>(min(static_cast<int64_t>(kGroup), p.R - r0));
  const uint32_t B = static_cast<uint32_t>(p.B);
  int bad = 0;

  // the groups before this one
  int64_t base_new = 0, base_seq = 0, base_page = 0;
  if (r0 > 0) {
    int64_t a = 0, b = 0, c = 0;
    for (int64_t r = threadIdx.x; r < r0; r += kThreads) {
      const Lens l = lens_of(p, r);
      a += l.fresh;
      b += static_cast<int64_t>(l.ctx) + l.fresh;
      c += pages_of(l.ctx + l.fresh, B) - pages_of(l.ctx, B);
    }
    block_scan<int64_t>(a, scratch, base_new);
    block_scan<int64_t>(b, scratch, base_seq);
    block_scan<int64_t>(c, scratch, base_page);
  }

  // this group: each thread owns kPer consecutive requests
  int64_t an = 0, as = 0, ap = 0;
  Lens own[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = static_cast<int>(threadIdx.x) * kPer + i;
    own[i] = k < n ? lens_of(p, r0 + k) : Lens{0, 0, 0};
    bad |= own[i].bad;
    an += own[i].fresh;
    as += static_cast<int64_t>(own[i].ctx) + own[i].fresh;
    ap += pages_of(own[i].ctx + own[i].fresh, B) - pages_of(own[i].ctx, B);
  }
  int64_t tn, ts, tp;
  int64_t cn = base_new + block_scan<int64_t>(an, scratch, tn);
  int64_t cs = base_seq + block_scan<int64_t>(as, scratch, ts);
  int64_t cp = base_page + block_scan<int64_t>(ap, scratch, tp);
  const bool writer = slice == 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = static_cast<int>(threadIdx.x) * kPer + i;
    if (k < n) {
      cu[k] = cn;
      pg[k] = cp;
      ctx[k] = own[i].ctx;
      if (writer) {
        p.cu_new[r0 + k] = cut(cn);
        if (p.cu_seq != nullptr) p.cu_seq[r0 + k] = cut(cs);
        p.seq_lens[r0 + k] = own[i].ctx + own[i].fresh;
      }
    }
    cn += own[i].fresh;
    cs += static_cast<int64_t>(own[i].ctx) + own[i].fresh;
    cp += pages_of(own[i].ctx + own[i].fresh, B) - pages_of(own[i].ctx, B);
  }
  const int64_t end_new = base_new + tn, end_page = base_page + tp;
  const bool last = r0 + n == p.R;
  if (threadIdx.x == 0) {
    cu[n] = end_new;
    pg[n] = end_page;
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
      const int64_t column = pages_of(ctx[k], B) + (i - pg[k]);
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
    for (int64_t t = lo + threadIdx.x; t < hi; t += kThreads) {
      int64_t slot = -1;
      int32_t pos = -1, seq = -1;
      if (t < end_new) {
        const int k = find(cu, n, t);
        seq = static_cast<int32_t>(r0 + k);
        const uint32_t at = static_cast<uint32_t>(ctx[k]) + static_cast<uint32_t>(t - cu[k]);
        pos = static_cast<int32_t>(at);
        if (p.slots != nullptr) {
          const uint32_t page = at / B, first = pages_of(ctx[k], B);
          int64_t id = -1;
          if (page < p.bt_stride) {
            if (page >= first) {
              const int64_t i = pg[k] + (page - first);
              if (i < p.num_free) id = p.free_ids[i];
            } else {
              id = p.bt[static_cast<int64_t>(seq) * p.bt_stride + page];
            }
            if (id >= 0 && id < p.num_blocks) slot = id * p.B + at % B;
            else if (page < first) bad |= PMG_FLAG_PHYS_BLOCK;
          } else {
            bad |= PMG_FLAG_LOGICAL_BLOCK;
          }
        }
      }
      if (p.slots != nullptr) p.slots[t] = slot;
      if (p.positions != nullptr) p.positions[t] = pos;
      if (p.t2s != nullptr) p.t2s[t] = seq;
    }
  }
  set_flag(p.err, bad);
}

constexpr int kSmem = (kGroup + 1) * 16 + kGroup * 4;

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
  PlanParams p{ctx_lens, new_lens, num_reqs, block_table, block_table_stride, free_blocks, num_free, num_blocks,
               block_size, slots, positions, token_to_seq, max_tokens, cu_new, seq_lens, cu_seq, blocks_taken,
               error_flag, 1};
  int sms = 0;
  int st = sm_count(&sms);
  if (st == PMG_OK) st = allow_smem(reinterpret_cast<const void*>(plan_step_kernel), kSmem);
  if (st != PMG_OK) return st;
  const int64_t groups = std::max<int64_t>(1, (static_cast<int64_t>(num_reqs) + kGroup - 1) / kGroup);
  const int64_t want = (max_tokens + kTokensPerCta * groups - 1) / (kTokensPerCta * groups);
  p.slices = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(want, std::max<int64_t>(1, 2 * sms / groups))));
  return launch(plan_step_kernel, dim3(static_cast<unsigned>(groups * p.slices)), kThreads, kSmem, stream, p);
}
