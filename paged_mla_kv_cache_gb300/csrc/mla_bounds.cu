// Bounds of the entries of the cache's pages (pmg_block_bounds).
//
// Mathematics: hi[d] = max_j e_j[d], lo[d] = min_j e_j[d] over the entries that
// joined a page, folded into what was known of earlier ones. Maximum and
// minimum are exact in any order and any wider type: 16-bit values are compared
// two at a time as they are, e4m3 ones as the fp16 values that they stand for.
//
// Bound by memory: the new entries once, two rows a touched page. A thread takes
// one 16-byte column unit of a touched page through all of its entries, kAhead of
// them on their way at once, so neighbours read neighbouring units and nothing
// has to meet; the units of all requests' pages are a flat list, cut into equal
// shares, a CTA each. 300000 e4m3 entries take 34 us, 5.4 TB/s of entries and bounds
// (a CTA a page, with groups of threads over its entries that meet in shared
// memory: 44 us at best); a step of 64 requests 3.4 us, one launch. Rows that are
// not whole aligned units take the same threads element by element.
#include <algorithm>

#include "mla_attn.cuh"
#include "mla_long.cuh"
#include "pmg_long.h"

namespace pmg_mla {
namespace {

constexpr int kThreads = 192;
constexpr int kAhead = 16;  // entries of a thread on their way
constexpr int kCtasPerSm = 2;

struct BoundsParams {
  const uint8_t* cache;
  int64_t blk_stride, tok_stride;
  int64_t num_blocks;
  int32_t B, E;
  uint8_t* bounds;
  int64_t bb_stride, br_stride;
  const int32_t* bt;
  int64_t bt_stride;
  const int32_t* ctx;
  const int32_t* seq;
  int32_t R, units;
  int32_t* err;
};

// Places [from, to) that joined a request, as far as its row of the table reaches.
struct Joined {
  int32_t from, to;
  int bad;
};
__device__ __forceinline__ Joined joined(const BoundsParams& p, int r) {
  Joined j{p.ctx != nullptr ? p.ctx[r] : 0, p.seq[r], 0};
  if (j.from < 0 || j.to < 0) j.bad = PMG_FLAG_LENGTH;
  j.from = max(j.from, 0);
  j.to = max(j.to, 0);
  const int64_t room = p.bt_stride * p.B;
  if (j.to > room && j.to > j.from) {
    j.bad |= PMG_FLAG_LOGICAL_BLOCK;
    j.to = static_cast<int32_t>(room);
  }
  return j;
}
__device__ __forceinline__ int64_t joined_pages(const BoundsParams& p, const Joined& j) {
  const uint32_t b = static_cast<uint32_t>(p.B);
  return j.to > j.from ? (static_cast<uint32_t>(j.to) + b - 1) / b - static_cast<uint32_t>(j.from) / b : 0;
}

// One 16-byte unit of entries (kVec) or one element, and its extremes so far.
template <class TC, bool kVec>
struct Extremes {
  static constexpr int kValues = kVec ? 16 / static_cast<int>(sizeof(TC)) : 1;
  static constexpr bool kPacked = kVec && sizeof(TC) < 4;  // two 16-bit values a word
  static constexpr int kWords = kPacked ? kValues / 2 : kValues;
  using Raw = typename std::conditional<kVec, uint4, TC>::type;
  uint32_t hi[kWords], lo[kWords];

  __device__ __forceinline__ void clear() {
    const uint32_t inf = !kPacked ? 0x7f800000u : std::is_same<TC, bf16>::value ? 0x7f807f80u : 0x7c007c00u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      hi[i] = inf | (kPacked ? 0x80008000u : 0x80000000u);
      lo[i] = inf;
    }
  }
  __device__ __forceinline__ static void largest(uint32_t& x, uint32_t a) {
    if constexpr (!kPacked) x = __float_as_uint(max_nan(__uint_as_float(x), __uint_as_float(a)));
    else if constexpr (std::is_same<TC, bf16>::value) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(a));
    else asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(x) : "r"(a));
  }
  __device__ __forceinline__ static void smallest(uint32_t& x, uint32_t a) {
    if constexpr (!kPacked) x = __float_as_uint(min_nan(__uint_as_float(x), __uint_as_float(a)));
    else if constexpr (std::is_same<TC, bf16>::value) asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(a));
    else asm("min.NaN.f16x2 %0, %0, %1;" : "+r"(x) : "r"(a));
  }
  __device__ __forceinline__ void fold(int i, uint32_t a, uint32_t b) {
    largest(hi[i], a);
    smallest(lo[i], b);
  }
  __device__ __forceinline__ void fold(const Raw& x) {
    if constexpr (!kVec) {
      const uint32_t v = __float_as_uint(to_f(x));
      fold(0, v, v);
    } else {
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(TC) == 1) {
          uint32_t a, b;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"(static_cast<uint16_t>(w[i])));
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(static_cast<uint16_t>(w[i] >> 16)));
          fold(2 * i, a, a);
          fold(2 * i + 1, b, b);
        } else {
          fold(i, w[i], w[i]);
        }
      }
    }
  }
  // value k of the unit
  __device__ __forceinline__ static float value(const uint32_t* words, int k) {
    if constexpr (!kPacked) return __uint_as_float(words[k]);
    else if constexpr (std::is_same<TC, bf16>::value)
      return __uint_as_float(k & 1 ? words[k >> 1] & 0xffff0000u : words[k >> 1] << 16);
    else return __half2float(__ushort_as_half(static_cast<unsigned short>(words[k >> 1] >> (k & 1 ? 16 : 0))));
  }
};

template <class TC, class TB, bool kVec>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) bounds_kernel(const __grid_constant__ BoundsParams p) {
  using X = Extremes<TC, kVec>;
  __shared__ int64_t scratch[33], found[2];
  pdl_entry();
  const uint32_t columns = static_cast<uint32_t>(p.E) / X::kValues, B = static_cast<uint32_t>(p.B);
  const Share share = find_share([&](int r) { return joined_pages(p, joined(p, r)) * columns; }, p.R, blockIdx.x, p.units,
                                 scratch, found);
  int bad = 0;
  // The thread's request: units [base, base + n) of the flat list.
  int r = share.item;
  int64_t base = share.begin - share.offset, n = 0;
  Joined j{};
  auto enter = [&]() {
    j = joined(p, r);
    n = joined_pages(p, j) * columns;
    bad |= j.bad;
  };
  const int64_t first = share.begin + threadIdx.x;
  if (first < share.end) enter();
  for (int64_t at = first; at < share.end; at += kThreads) {
    while (at >= base + n) {
      base += n;
      ++r;
      enter();
    }
    const int64_t y = at - base;
    const uint32_t in = static_cast<uint32_t>(y <= UINT32_MAX ? static_cast<uint32_t>(y) / columns : y / columns);
    const uint32_t column = static_cast<uint32_t>(y - static_cast<int64_t>(in) * columns), page = static_cast<uint32_t>(j.from) / B + in;
    const int32_t id = p.bt[static_cast<int64_t>(r) * p.bt_stride + page];
    if (id < 0 || id >= p.num_blocks) {
      bad |= PMG_FLAG_PHYS_BLOCK;
      continue;
    }
    const int64_t place = static_cast<int64_t>(page) * B;  // the page's first
    const int r0 = static_cast<int>(max(static_cast<int64_t>(j.from) - place, static_cast<int64_t>(0)));
    const int r1 = static_cast<int>(min(static_cast<int64_t>(j.to) - place, static_cast<int64_t>(B)));
    const TC* src = reinterpret_cast<const TC*>(p.cache) + id * p.blk_stride + r0 * p.tok_stride + column * X::kValues;
    TB* hi = reinterpret_cast<TB*>(p.bounds) + id * p.bb_stride + column * X::kValues;
    TB* lo = hi + p.br_stride;
    X x;
    x.clear();
    Values<TB, X::kValues> known_hi, known_lo;
    if (r0 > 0) {
      known_hi.load(hi);
      known_lo.load(lo);
    }
#pragma unroll 1
    for (int row = r0; row < r1; row += kAhead) {
      typename X::Raw raw[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)  // (past the last entry: the first of these once more)
        raw[k] = *reinterpret_cast<const typename X::Raw*>(src + (row + k < r1 ? k : 0) * p.tok_stride);
      src += kAhead * p.tok_stride;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) x.fold(raw[k]);
    }
    Values<TB, X::kValues> a, b;
#pragma unroll
    for (int k = 0; k < X::kValues; ++k) {
      float top = X::value(x.hi, k), low = X::value(x.lo, k);
      if (r0 > 0) {
        top = max_nan(top, to_f(known_hi.v[k]));
        low = min_nan(low, to_f(known_lo.v[k]));
      }
      a.v[k] = from_f<TB>(top);  // a value of the entries or of the bounds: nothing is rounded
      b.v[k] = from_f<TB>(low);
    }
    a.store(hi);
    b.store(lo);
  }
  // what is wrong with lengths of requests without pages here
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < p.R; i += gridDim.x * kThreads) bad |= joined(p, i).bad;
  set_flag(p.err, bad);
}

using Kernel = void (*)(const BoundsParams);

template <class TC, class TB>
Kernel pick(bool vec) {
  return vec ? bounds_kernel<TC, TB, true> : bounds_kernel<TC, TB, false>;
}

}  // namespace
}  // namespace pmg_mla

extern "C" int pmg_block_bounds(const void* cache, int64_t cache_block_stride, int64_t cache_token_stride,
                                int64_t num_blocks, int32_t block_size, int32_t entry_dim, int32_t cache_dtype,
                                void* bounds, int64_t bounds_block_stride, int64_t bounds_row_stride,
                                int32_t bounds_dtype, const int32_t* block_table, int64_t block_table_stride,
                                const int32_t* ctx_lens, const int32_t* seq_lens, int32_t num_reqs,
                                int32_t* error_flag, void* stream) {
  using namespace pmg_mla;
  const int ec = elem_bytes(cache_dtype), eb = elem_bytes(bounds_dtype);
  if (ec == 0 || eb < 2 || (cache_dtype != bounds_dtype && cache_dtype != PMG_FP8_E4M3)) return PMG_ERR_DTYPE;
  if (num_reqs < 0 || block_size < 1 || entry_dim < 1 || num_blocks < 0 || block_table_stride < 0) return PMG_ERR_ARG;
  for (const int64_t s : {cache_block_stride, cache_token_stride, bounds_block_stride, bounds_row_stride})
    if (!stride_ok(s)) return PMG_ERR_ARG;
  if (entry_dim > PMG_MAX_ENTRY || num_blocks > INT32_MAX || block_table_stride > INT32_MAX || num_reqs > PMG_MAX_REQS)
    return PMG_ERR_UNSUPPORTED;
  if (num_reqs == 0) return PMG_OK;
  if (seq_lens == nullptr || ((cache == nullptr || bounds == nullptr) && num_blocks > 0) ||
      (block_table == nullptr && block_table_stride > 0))
    return PMG_ERR_NULL;
  if (!aligned(cache, ec) || !aligned(bounds, eb) || !aligned(block_table, 4) || !aligned(ctx_lens, 4) ||
      !aligned(seq_lens, 4) || !aligned(error_flag, 4))
    return PMG_ERR_ALIGN;
  // no two rows that are written overlap: pages lie behind each other, or all largest values before all smallest ones
  // (other threads write them, in no order)
  if (num_blocks > 0 && bounds_row_stride < entry_dim) return PMG_ERR_ARG;
  if (num_blocks > 1 && bounds_block_stride < bounds_row_stride + entry_dim &&
      (bounds_block_stride < entry_dim || (bounds_row_stride - entry_dim) / (num_blocks - 1) < bounds_block_stride))
    return PMG_ERR_ARG;
  int sms = 0;
  const int st = sm_count(&sms);
  if (st != PMG_OK) return st;
  BoundsParams p{};
  p.cache = static_cast<const uint8_t*>(cache);
  p.blk_stride = cache_block_stride;
  p.tok_stride = cache_token_stride;
  p.num_blocks = num_blocks;
  p.B = block_size;
  p.E = entry_dim;
  p.bounds = static_cast<uint8_t*>(bounds);
  p.bb_stride = bounds_block_stride;
  p.br_stride = bounds_row_stride;
  p.bt = block_table;
  p.bt_stride = block_table_stride;
  p.ctx = ctx_lens;
  p.seq = seq_lens;
  p.R = num_reqs;
  p.units = sms * kCtasPerSm;
  p.err = error_flag;
  const bool vec = entry_dim * ec % 16 == 0 && aligned(cache, 16) && cache_block_stride * ec % 16 == 0 &&
                   cache_token_stride * ec % 16 == 0 && aligned(bounds, 16) && bounds_block_stride * eb % 16 == 0 &&
                   bounds_row_stride * eb % 16 == 0;
  Kernel k = nullptr;
  switch (cache_dtype) {
    case PMG_BF16: k = pick<bf16, bf16>(vec); break;
    case PMG_FP16: k = pick<f16, f16>(vec); break;
    case PMG_FP32: k = pick<float, float>(vec); break;
    default:
      k = bounds_dtype == PMG_BF16 ? pick<e4m3, bf16>(vec) : bounds_dtype == PMG_FP16 ? pick<e4m3, f16>(vec) : pick<e4m3, float>(vec);
  }
  return launch(k, dim3(static_cast<unsigned>(p.units)), kThreads, 0, stream, p);
}
