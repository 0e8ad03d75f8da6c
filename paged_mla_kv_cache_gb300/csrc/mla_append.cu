// Norm, rotation and the write of new entries into the paged cache
// (pmg_append).
//
// Mathematics, for each token: y = c * rsqrt(mean(c^2) + eps) * w over the
// latent part; every pair (a, b) of the rotated part, of the shared key and of
// each head's query, goes to (a cos - b sin, b cos + a sin). All in 32 bits,
// one rounding at the store (an e4m3 cache: y / scale, to nearest even,
// saturating).
//
// Bound by memory: an entry in and out, 2 * rope_dim elements a head, one row
// of cosines and sines a token. Measured: 8192 tokens of 128 heads into an e4m3
// cache 59 us (285 MB, 72% of copy bandwidth; a plain copy of the same strided
// 128-byte rows takes 46 us: the rest is mostly the entries, whose warps go
// through a chain of slot, values, sum and store: alone the two launches take
// 12.5 and 43.5 us, so they hardly overlap); 64 tokens
// 7.4 us, the host's call and one launch. One warp takes either a token's entry (the
// latent row stays in registers between the sum and the store, so it is read
// once) or a few heads of a token's queries, for which a lane keeps one set of
// four cosines and sines in registers and issues all its loads before the
// first store. Units are four pairs: 16 bytes of 16-bit values where pairs are
// neighbours, two times 8 bytes where halves are rotated. Rows that are not
// 16-byte aligned or not whole units take the same warps element by element.
#include <algorithm>

#include "mla_common.cuh"

namespace pmg_mla {
namespace {

constexpr int kWarps = 4;          // tasks of a CTA
constexpr int kIters = 4;          // row groups of queries a warp has in flight
constexpr int kMaxLatentUnits = 4; // units of 8 latent values a lane holds: latent_dim up to 1024

struct AppendParams {
  const uint8_t* c_kv;
  int64_t c_stride;
  const uint8_t* k_pe;
  int64_t k_stride;
  const float* weight;
  float eps;
  const float* cos_sin;
  int64_t num_positions;
  const int64_t* slots;
  const int32_t* positions;
  int64_t T;
  int32_t dv, dr;
  uint8_t* cache;
  int64_t blk_stride, tok_stride;
  int64_t num_blocks;
  int32_t B;
  const float* scale;
  const uint8_t* q;
  int64_t qt_stride, qh_stride;
  uint8_t* qo;
  int64_t ot_stride, oh_stride;
  int32_t H;
  int32_t heads_per_task;
  int32_t tasks_per_token;  // 1 entry + query tasks
  int32_t pairs;
  int32_t* err;
};

// N values (a multiple of 4 bytes in all, aligned to their size up to 16)
template <class T, int N>
struct Pack {
  static constexpr int kBytes = N * static_cast<int>(sizeof(T));
  static constexpr int kAlign = kBytes < 16 ? kBytes : 16;
  alignas(kAlign) T v[N];
};

template <class T, int N>
__device__ __forceinline__ void load_n(const T* src, float* x) {
  const Pack<T, N> p = *reinterpret_cast<const Pack<T, N>*>(src);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = to_f(p.v[i]);
}

template <class T, int N>
__device__ __forceinline__ void store_n(T* dst, const float* x) {
  Pack<T, N> p;
  if constexpr (sizeof(T) == 1) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const __nv_fp8x2_storage_t two = __nv_cvt_float2_to_fp8x2(make_float2(x[i], x[i + 1]), __NV_SATFINITE, __NV_E4M3);
      p.v[i].__x = static_cast<__nv_fp8_storage_t>(two & 0xff);
      p.v[i + 1].__x = static_cast<__nv_fp8_storage_t>(two >> 8);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p.v[i] = from_f<T>(x[i]);
  }
  *reinterpret_cast<Pack<T, N>*>(dst) = p;
}

// The four pairs of unit u of a row as they are in memory, and a and b of each.
template <class T>
struct RawPairs {
  Pack<T, 4> lo, hi;  // neighbours: pairs 0, 1 and 2, 3; halves: a and b
};
template <class T>
__device__ __forceinline__ RawPairs<T> load_pairs(const T* row, int u, int half, bool pairs) {
  RawPairs<T> r;
  if (pairs) {
    const Pack<T, 8> p = *reinterpret_cast<const Pack<T, 8>*>(row + 8 * u);
#pragma unroll
    for (int i = 0; i < 4; ++i) { r.lo.v[i] = p.v[i]; r.hi.v[i] = p.v[4 + i]; }
  } else {
    r.lo = *reinterpret_cast<const Pack<T, 4>*>(row + 4 * u);
    r.hi = *reinterpret_cast<const Pack<T, 4>*>(row + half + 4 * u);
  }
  return r;
}
template <class T>
__device__ __forceinline__ void split_pairs(const RawPairs<T>& r, bool pairs, float* a, float* b) {
  if (pairs) {
    a[0] = to_f(r.lo.v[0]); b[0] = to_f(r.lo.v[1]); a[1] = to_f(r.lo.v[2]); b[1] = to_f(r.lo.v[3]);
    a[2] = to_f(r.hi.v[0]); b[2] = to_f(r.hi.v[1]); a[3] = to_f(r.hi.v[2]); b[3] = to_f(r.hi.v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) { a[i] = to_f(r.lo.v[i]); b[i] = to_f(r.hi.v[i]); }
  }
}

template <class T>
__device__ __forceinline__ void store_pairs(T* row, int u, int half, bool pairs, const float* a, const float* b) {
  if (pairs) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[2 * i] = a[i]; x[2 * i + 1] = b[i]; }
    store_n<T, 8>(row + 8 * u, x);
  } else {
    store_n<T, 4>(row + 4 * u, a);
    store_n<T, 4>(row + half + 4 * u, b);
  }
}

__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float x = a * c - b * s, y = b * c + a * s;
  a = x;
  b = y;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What a launch does: entries and queries, or one of them. Large calls launch
// the queries by themselves (below, or here where rows are not whole units).
enum Work : int { kBoth = 0, kEntries = 1, kQueries = 2 };

template <class TS, class TC, bool kVec, int kWork>
__global__ void __launch_bounds__(kWarps * 32, 8) append_kernel(const __grid_constant__ AppendParams p) {
  if constexpr (kWork == kEntries) {
    // the queries' launch that may follow reads what earlier kernels wrote without a wait of its own
    pdl_wait();
    pdl_launch();
  } else {
    pdl_entry();
  }
  const int lane = threadIdx.x & 31;
  // tasks token by token: warps that run together read and write neighbouring rows
  const uint32_t task = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t tasks = kWork == kEntries ? 1 : kWork == kQueries ? p.tasks_per_token - 1 : p.tasks_per_token;
  const int64_t t = kWork == kEntries ? task : task / tasks;
  const int part = kWork == kEntries ? 0 : static_cast<int>(task % tasks) + (kWork == kQueries ? 1 : 0);
  if (t >= p.T) return;
  const int half = p.dr >> 1;
  const bool pairs = p.pairs != 0;
  const int32_t pos = p.positions[t];
  const bool turned = pos >= 0 && pos < p.num_positions;
  const float* cs = p.cos_sin + static_cast<int64_t>(turned ? pos : 0) * p.dr;

  if (kWork == kEntries || (kWork == kBoth && part == 0)) {
    const int64_t slot = p.slots[t];
    if (slot < 0) {
      if (lane == 0 && pos >= p.num_positions) set_flag(p.err, PMG_FLAG_POSITION);
      return;
    }
    const int64_t block = slot <= UINT32_MAX ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.B) : slot / p.B;
    if (!turned || block >= p.num_blocks) {
      if (lane == 0)
        set_flag(p.err, (turned ? 0 : PMG_FLAG_POSITION) | (block < p.num_blocks ? 0 : PMG_FLAG_PHYS_BLOCK));
      return;
    }
    const TS* c = reinterpret_cast<const TS*>(p.c_kv) + t * p.c_stride;
    const TS* kp = reinterpret_cast<const TS*>(p.k_pe) + t * p.k_stride;
    TC* row = reinterpret_cast<TC*>(p.cache) + block * p.blk_stride + (slot - block * p.B) * p.tok_stride;
    const float scale = sizeof(TC) == 1 && p.scale != nullptr ? *p.scale : 1.0f;
    const float inv_n = 1.0f / static_cast<float>(p.dv);
    if constexpr (kVec) {
      Pack<TS, 8> raw[kMaxLatentUnits];
      float a[4], b[4], co[4], si[4];
      const bool turns = lane * 8 < p.dr;
      // every load of the token first
#pragma unroll
      for (int i = 0; i < kMaxLatentUnits; ++i)
        if ((lane + 32 * i) * 8 < p.dv) raw[i] = *reinterpret_cast<const Pack<TS, 8>*>(c + (lane + 32 * i) * 8);
      if (turns) {
        split_pairs(load_pairs(kp, lane, half, pairs), pairs, a, b);
        load_n<float, 4>(cs + 4 * lane, co);
        load_n<float, 4>(cs + half + 4 * lane, si);
      }
      float inv = 1.0f;
      if (p.weight != nullptr) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kMaxLatentUnits; ++i)
          if ((lane + 32 * i) * 8 < p.dv) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float v = to_f(raw[i].v[k]);
              sum += v * v;
            }
          }
        inv = rsqrtf(warp_sum(sum) * inv_n + p.eps);
      }
#pragma unroll
      for (int i = 0; i < kMaxLatentUnits; ++i) {
        const int at = (lane + 32 * i) * 8;
        if (at >= p.dv) continue;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = to_f(raw[i].v[k]);
        if (p.weight != nullptr) {
          float w[8];
          load_n<float, 4>(p.weight + at, w);
          load_n<float, 4>(p.weight + at + 4, w + 4);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = x[k] * inv * w[k];
        }
        if constexpr (sizeof(TC) == 1) {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = x[k] / scale;
        }
        store_n<TC, 8>(row + at, x);
      }
      if (turns) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          rotate(a[k], b[k], co[k], si[k]);
          if constexpr (sizeof(TC) == 1) { a[k] = a[k] / scale; b[k] = b[k] / scale; }
        }
        store_pairs(row + p.dv, lane, half, pairs, a, b);
      }
    } else {
      float inv = 1.0f;
      if (p.weight != nullptr) {
        float sum = 0.0f;
        for (int i = lane; i < p.dv; i += 32) {
          const float v = to_f(c[i]);
          sum += v * v;
        }
        inv = rsqrtf(warp_sum(sum) * inv_n + p.eps);
      }
      for (int i = lane; i < p.dv; i += 32) {
        float v = to_f(c[i]);
        if (p.weight != nullptr) v = v * inv * p.weight[i];
        row[i] = from_f<TC>(sizeof(TC) == 1 ? v / scale : v);
      }
      for (int i = lane; i < half; i += 32) {
        const int ia = pairs ? 2 * i : i, ib = pairs ? 2 * i + 1 : i + half;
        float a = to_f(kp[ia]), b = to_f(kp[ib]);
        rotate(a, b, cs[i], cs[half + i]);
        row[p.dv + ia] = from_f<TC>(sizeof(TC) == 1 ? a / scale : a);
        row[p.dv + ib] = from_f<TC>(sizeof(TC) == 1 ? b / scale : b);
      }
    }
    return;
  }

  // heads of a token's queries
  const int h0 = (part - 1) * p.heads_per_task;
  const int h1 = min(h0 + p.heads_per_task, p.H);
  const TS* q = reinterpret_cast<const TS*>(p.q) + t * p.qt_stride;
  TS* o = reinterpret_cast<TS*>(p.qo) + t * p.ot_stride;
  if constexpr (kVec) {
    const int lanes = p.dr >> 3;      // lanes of a row: a divisor of 32
    const int u = lane & (lanes - 1), step = 32 / lanes;
    const int h = h0 + lane / lanes;
    // the queries do not wait for the position
    RawPairs<TS> raw[kIters];
#pragma unroll
    for (int i = 0; i < kIters; ++i)
      if (h + i * step < h1) raw[i] = load_pairs(q + (h + i * step) * p.qh_stride, u, half, pairs);
    if (!turned) return;  // reported by the entry's warp
    float co[4], si[4];
    load_n<float, 4>(cs + 4 * u, co);
    load_n<float, 4>(cs + half + 4 * u, si);
#pragma unroll
    for (int i = 0; i < kIters; ++i)
      if (h + i * step < h1) {
        float a[4], b[4];
        split_pairs(raw[i], pairs, a, b);
#pragma unroll
        for (int k = 0; k < 4; ++k) rotate(a[k], b[k], co[k], si[k]);
        store_pairs(o + (h + i * step) * p.oh_stride, u, half, pairs, a, b);
      }
  } else {
    if (!turned) return;
    for (int h = h0; h < h1; ++h)
      for (int i = lane; i < half; i += 32) {
        const int ia = pairs ? 2 * i : i, ib = pairs ? 2 * i + 1 : i + half;
        float a = to_f(q[h * p.qh_stride + ia]), b = to_f(q[h * p.qh_stride + ib]);
        rotate(a, b, cs[i], cs[half + i]);
        o[h * p.oh_stride + ia] = from_f<TS>(a);
        o[h * p.oh_stride + ib] = from_f<TS>(b);
      }
  }
}

// The queries of a large call. A warp's rows pass through shared memory with
// asynchronous copies, kStages tasks of kIters row groups in flight: a lane
// waits for its own copies only, and what is in flight costs no registers. (As
// one task a warp, twelve CTAs an SM, the chain of position, angles and values
// left 52% of the memory's rate: 70 us instead of 60 for 8192 tokens of 128
// heads.) Positions are looked up 32 tasks ahead. Two stages in seven or eight CTAs
// an SM measured 63 us, three in five 65, four in four 60.
constexpr int kStages = 3;
constexpr int kQueryCtas = 6;  // an SM

template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(src) : "memory");
}

template <class TS>
struct QueryStage {
  RawPairs<TS> raw[kIters][32];
  float4 co[32], si[32];
};
template <class TS>
constexpr int query_smem() { return kWarps * kStages * static_cast<int>(sizeof(QueryStage<TS>)); }

template <class TS>
__global__ void __launch_bounds__(kWarps * 32, sizeof(TS) == 2 ? kQueryCtas : kQueryCtas / 2)
    append_queries_kernel(const __grid_constant__ AppendParams p) {
  pdl_launch();
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  QueryStage<TS>* stages = reinterpret_cast<QueryStage<TS>*>(smem) + warp * kStages;
  const uint32_t per_token = p.tasks_per_token - 1, tasks = static_cast<uint32_t>(p.T) * per_token;
  const uint32_t warps = gridDim.x * kWarps, first = blockIdx.x * kWarps + warp;
  const uint32_t n = first < tasks ? (tasks - first + warps - 1) / warps : 0;  // this warp's: first + i * warps
  const int half = p.dr >> 1, lanes = p.dr >> 3;
  const bool pairs = p.pairs != 0;
  const int u = lane & (lanes - 1), step = 32 / lanes;
  auto positions = [&](uint32_t i) {  // of tasks i + lane
    return i + lane < n ? p.positions[(first + (i + lane) * warps) / per_token] : -1;
  };
  int32_t now = positions(0), then = positions(32);
  uint32_t seen = 0;  // bit: the tasks in flight, newest first, whose queries are turned
  auto begin = [&](uint32_t i, QueryStage<TS>& s) {
    if (i > 0 && i % 32 == 0) {
      now = then;
      then = positions(i + 32);
    }
    const int32_t pos = __shfl_sync(0xffffffffu, now, i % 32);
    const bool turned = i < n && pos >= 0 && pos < p.num_positions;
    seen = seen << 1 | turned;
    if (turned) {
      const uint32_t task = first + i * warps, t = task / per_token;
      const int h0 = static_cast<int>(task - t * per_token) * p.heads_per_task + lane / lanes;
      const int h1 = min(h0 - lane / lanes + p.heads_per_task, p.H);
      const float* cs = p.cos_sin + static_cast<int64_t>(pos) * p.dr + 4 * u;
      copy_async<16>(&s.co[lane], cs);
      copy_async<16>(&s.si[lane], cs + half);
      const TS* q = reinterpret_cast<const TS*>(p.q) + t * p.qt_stride;
#pragma unroll
      for (int k = 0; k < kIters; ++k)
        if (h0 + k * step < h1) {
          const TS* row = q + (h0 + k * step) * p.qh_stride;
          RawPairs<TS>* dst = &s.raw[k][lane];
          if (pairs && sizeof(TS) == 2) {
            copy_async<16>(dst, row + 8 * u);
          } else {
            copy_async<4 * sizeof(TS)>(&dst->lo, pairs ? row + 8 * u : row + 4 * u);
            copy_async<4 * sizeof(TS)>(&dst->hi, pairs ? row + 8 * u + 4 : row + half + 4 * u);
          }
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  uint32_t ahead = 0, at = 0;
  for (; ahead < kStages - 1; ++ahead) begin(ahead, stages[ahead]);
  for (uint32_t i = 0; i < n; ++i) {
    // the stage of the task before is free: its lanes have their values in registers
    begin(i + kStages - 1, stages[at == 0 ? kStages - 1 : at - 1]);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    if (seen >> (kStages - 1) & 1) {
      const QueryStage<TS>& s = stages[at];
      const uint32_t task = first + i * warps, t = task / per_token;
      const int h0 = static_cast<int>(task - t * per_token) * p.heads_per_task + lane / lanes;
      const int h1 = min(h0 - lane / lanes + p.heads_per_task, p.H);
      TS* o = reinterpret_cast<TS*>(p.qo) + t * p.ot_stride;
      const float4 c4 = s.co[lane], s4 = s.si[lane];
      const float co[4] = {c4.x, c4.y, c4.z, c4.w}, si[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int k = 0; k < kIters; ++k)
        if (h0 + k * step < h1) {
          float a[4], b[4];
          split_pairs(s.raw[k][lane], pairs, a, b);
#pragma unroll
          for (int j = 0; j < 4; ++j) rotate(a[j], b[j], co[j], si[j]);
          store_pairs(o + (h0 + k * step) * p.oh_stride, u, half, pairs, a, b);
        }
    }
    at = at + 1 == kStages ? 0 : at + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  pdl_wait();  // this kernel ends after the one before it
}

template <class TS>
int launch_queries(const AppendParams& p, int sms, void* stream) {
  auto k = append_queries_kernel<TS>;
  const int st = allow_smem(reinterpret_cast<const void*>(k), query_smem<TS>());
  if (st != PMG_OK) return st;
  const int64_t tasks = p.T * (p.tasks_per_token - 1);
  const int64_t ctas = std::min<int64_t>(static_cast<int64_t>(sms) * (sizeof(TS) == 2 ? kQueryCtas : kQueryCtas / 2),
                                         (tasks + kWarps - 1) / kWarps);
  return launch(k, dim3(static_cast<unsigned>(ctas)), kWarps * 32, query_smem<TS>(), stream, p);
}

using Kernel = void (*)(const AppendParams);

template <class TS, class TC, int kWork>
Kernel pick(bool vec) {
  return vec ? append_kernel<TS, TC, true, kWork> : append_kernel<TS, TC, false, kWork>;
}

template <class TS, int kWork>
Kernel pick(int cache_dtype, bool vec) {
  switch (cache_dtype) {
    case PMG_BF16: return pick<TS, bf16, kWork>(vec);
    case PMG_FP16: return pick<TS, f16, kWork>(vec);
    case PMG_FP32: return pick<TS, float, kWork>(vec);
    default: return pick<TS, e4m3, kWork>(vec);
  }
}

template <class TS>
Kernel pick(int cache_dtype, bool vec, Work work) {
  // the queries do not depend on the cache's type
  return work == kBoth ? pick<TS, kBoth>(cache_dtype, vec)
                       : work == kEntries ? pick<TS, kEntries>(cache_dtype, vec) : append_kernel<TS, bf16, false, kQueries>;
}

}  // namespace
}  // namespace pmg_mla

extern "C" int pmg_append(const void* c_kv, int64_t c_kv_stride, const void* k_pe, int64_t k_pe_stride,
                          const float* norm_weight, float eps, const float* cos_sin, int64_t num_positions,
                          const int64_t* slots, const int32_t* positions, int64_t num_tokens, int32_t latent_dim,
                          int32_t rope_dim, int32_t src_dtype, void* cache, int64_t cache_block_stride,
                          int64_t cache_token_stride, int64_t num_blocks, int32_t block_size, int32_t cache_dtype,
                          const float* scale, const void* q_pe, int64_t q_pe_token_stride, int64_t q_pe_head_stride,
                          void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, int32_t heads,
                          int32_t* error_flag, void* stream, uint32_t options) {
  using namespace pmg_mla;
  const int es = elem_bytes(src_dtype), ec = elem_bytes(cache_dtype);
  if (es < 2 || ec == 0) return PMG_ERR_DTYPE;
  if (latent_dim < 1 || rope_dim < 0 || rope_dim % 2 != 0 || num_positions < 0 || num_tokens < 0 || num_blocks < 0 ||
      block_size < 1 || heads < 0 || !(eps >= 0.0f) || (options & ~PMG_OPT_ROPE_PAIRS))
    return PMG_ERR_ARG;
  if (!stride_ok(c_kv_stride) || !stride_ok(k_pe_stride) || !stride_ok(cache_block_stride) ||
      !stride_ok(cache_token_stride) || !stride_ok(q_pe_token_stride) || !stride_ok(q_pe_head_stride) ||
      !stride_ok(q_out_token_stride) || !stride_ok(q_out_head_stride))
    return PMG_ERR_ARG;
  if (num_tokens > INT32_MAX || num_positions > INT32_MAX || num_blocks > INT32_MAX || latent_dim > (1 << 20) ||
      rope_dim > (1 << 20) || heads > (1 << 16))
    return PMG_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PMG_OK;
  if (c_kv == nullptr || slots == nullptr || positions == nullptr || (cache == nullptr && num_blocks > 0) ||
      (rope_dim > 0 && (k_pe == nullptr || (cos_sin == nullptr && num_positions > 0))) ||
      (heads > 0 && rope_dim > 0 && (q_pe == nullptr || q_out == nullptr)))
    return PMG_ERR_NULL;
  if (!aligned(c_kv, es) || !aligned(k_pe, es) || !aligned(norm_weight, 4) || !aligned(cos_sin, 4) ||
      !aligned(slots, 8) || !aligned(positions, 4) || !aligned(cache, ec) || !aligned(scale, 4) ||
      !aligned(q_pe, es) || !aligned(q_out, es) || !aligned(error_flag, 4))
    return PMG_ERR_ALIGN;
  if (rope_dim == 0) {
    heads = 0;
    num_positions = INT32_MAX;  // nothing is looked up
  }
  AppendParams p{};
  p.c_kv = static_cast<const uint8_t*>(c_kv);
  p.c_stride = c_kv_stride;
  p.k_pe = static_cast<const uint8_t*>(k_pe);
  p.k_stride = k_pe_stride;
  p.weight = norm_weight;
  p.eps = eps;
  p.cos_sin = cos_sin;
  p.num_positions = num_positions;
  p.slots = slots;
  p.positions = positions;
  p.T = num_tokens;
  p.dv = latent_dim;
  p.dr = rope_dim;
  p.cache = static_cast<uint8_t*>(cache);
  p.blk_stride = cache_block_stride;
  p.tok_stride = cache_token_stride;
  p.num_blocks = num_blocks;
  p.B = block_size;
  p.scale = scale;
  p.q = static_cast<const uint8_t*>(q_pe);
  p.qt_stride = q_pe_token_stride;
  p.qh_stride = q_pe_head_stride;
  p.qo = static_cast<uint8_t*>(q_out);
  p.ot_stride = q_out_token_stride;
  p.oh_stride = q_out_head_stride;
  p.H = heads;
  p.pairs = (options & PMG_OPT_ROPE_PAIRS) ? 1 : 0;
  p.err = error_flag;
  // whole units at 16-byte aligned rows (8-byte rows of an e4m3 cache); a row
  // of queries takes a power of two of lanes
  auto rows16 = [](const void* base, int bytes, int64_t s0, int64_t s1) {
    const int n = 8 * bytes < 16 ? 8 * bytes : 16;
    return aligned(base, n) && s0 * bytes % n == 0 && s1 * bytes % n == 0;
  };
  const int lanes = rope_dim / 8;
  const bool vec = latent_dim % 8 == 0 && latent_dim <= kMaxLatentUnits * 256 && rope_dim % 8 == 0 && rope_dim > 0 &&
                   lanes <= 32 && (lanes & (lanes - 1)) == 0 && rows16(c_kv, es, c_kv_stride, 0) &&
                   rows16(k_pe, es, k_pe_stride, 0) && rows16(cache, ec, cache_block_stride, cache_token_stride) &&
                   aligned(cos_sin, 16) && aligned(norm_weight, 16) &&
                   (heads == 0 || (rows16(q_pe, es, q_pe_token_stride, q_pe_head_stride) &&
                                   rows16(q_out, es, q_out_token_stride, q_out_head_stride)));
  p.heads_per_task = vec ? kIters * (32 / lanes) : 8;
  p.tasks_per_token = 1 + (heads + p.heads_per_task - 1) / p.heads_per_task;
  auto kernel = [&](Work work) {
    return src_dtype == PMG_BF16 ? pick<bf16>(cache_dtype, vec, work)
           : src_dtype == PMG_FP16 ? pick<f16>(cache_dtype, vec, work) : pick<float>(cache_dtype, vec, work);
  };
  // a warp a task
  const int64_t tasks = p.tasks_per_token;
  if (num_tokens * tasks > INT32_MAX) return PMG_ERR_UNSUPPORTED;
  auto grid = [&](int64_t per_token) { return dim3(static_cast<unsigned>((num_tokens * per_token + kWarps - 1) / kWarps)); };
  // Queries by themselves: 128 heads, back to back on the device, 34 us instead of 40 at 64 MB of queries, 10.3 instead of
  // 10.9 at 16 MB, 6.7 instead of 6.3 at 8 MB; and a second launch takes the host about 2 us.
  if (tasks == 1 || num_tokens * heads * rope_dim * es < (int64_t{16} << 20))
    return launch(kernel(tasks == 1 ? kEntries : kBoth), grid(tasks), kWarps * 32, 0, stream, p);
  const int st = launch(kernel(kEntries), grid(1), kWarps * 32, 0, stream, p);
  if (st != PMG_OK) return st;
  if (!vec) return launch(kernel(kQueries), grid(tasks - 1), kWarps * 32, 0, stream, p);
  int sms = 0;
  const int found = sm_count(&sms);
  if (found != PMG_OK) return found;
  return src_dtype == PMG_BF16   ? launch_queries<bf16>(p, sms, stream)
         : src_dtype == PMG_FP16 ? launch_queries<f16>(p, sms, stream)
                                 : launch_queries<float>(p, sms, stream);
}
