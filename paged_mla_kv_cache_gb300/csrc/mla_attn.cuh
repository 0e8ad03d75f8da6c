// What the attention kernels share: how a flat list of work is cut into equal
// shares, where a share's unfinished rows go, and the kernel body for any
// sizes.
//
// The work of a call is a flat list of equal pieces (a tile of keys for one
// group of rows), request after request, with a few idle pieces before each
// request for what its beginning and end cost. The list is cut into as many
// equal shares as there are units (a unit is the CTAs that run one share, one
// for each group of rows), so long and short requests cost every SM the same.
// A request that a share covers whole is finished there. One that a cut falls
// into leaves, from every share that holds a part of it, the unnormalised
// rows, their running maximum and their sum in the workspace; the share that
// holds its first tile notes how many shares follow, and the join kernel adds
// them up in their order, so results do not depend on timing.
#pragma once

#include "mla_common.cuh"

namespace pmg_mla {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Workspace: one note a CTA, then two slots of unfinished rows a CTA (0: the
// share began inside the request, 1: the share ended inside it).
struct JoinNote {
  int32_t item;         // request that begins in this share and goes on in the next, or -1
  int32_t parts;        // shares that hold it
  int32_t head, tile;   // prefill: which of the request's row tiles
};
constexpr int kNotesPerSm = 4;
constexpr int64_t kSlotFloats = 256 * 130;  // the largest slot: 256 rows of 128 values, or 64 of 512, and two sums each

struct Workspace {
  JoinNote* notes;
  float* slots;
};

inline int64_t workspace_notes(int sms) { return static_cast<int64_t>(sms) * kNotesPerSm * sizeof(JoinNote); }
inline int64_t workspace_bytes(int sms) { return (workspace_notes(sms) + 255) / 256 * 256 + 2 * sms * kSlotFloats * 4; }
inline Workspace workspace_at(void* base, int sms) {
  uint8_t* b = static_cast<uint8_t*>(base);
  return {reinterpret_cast<JoinNote*>(b), reinterpret_cast<float*>(b + (workspace_notes(sms) + 255) / 256 * 256)};
}

struct Share {
  int64_t begin, end;  // flat pieces
  int64_t total;
  int32_t units;       // units that have a share: none of them is empty
  int32_t item;        // the item that holds `begin`
  int64_t offset;      // pieces of it before `begin`
};

// x * a / b for 0 <= a <= b, in 32 bits where they do
__device__ __forceinline__ int64_t scaled(int64_t x, int a, int b) {
  if (x * a <= UINT32_MAX) return static_cast<uint32_t>(x * a) / static_cast<uint32_t>(b);
  return x * a / b;
}

__device__ __forceinline__ Share cut_share(int64_t total, int unit, int units) {
  Share s;
  s.total = total;
  s.units = static_cast<int32_t>(min(static_cast<int64_t>(units), total));
  s.begin = unit < s.units ? scaled(total, unit, s.units) : total;
  s.end = unit < s.units ? scaled(total, unit + 1, s.units) : total;
  return s;
}

// This unit's share of sum over items of pieces(item), found by the whole
// block, or for up to 32 items by every warp for itself. `scratch`: 33 int64,
// `found`: 2 int64, both shared.
template <class F>
__device__ __forceinline__ Share find_share(F pieces, int items, int unit, int units, int64_t* scratch, int64_t* found) {
  const int nt = blockDim.x, tid = threadIdx.x;
  if (items <= 32) {
    const int lane = tid & 31;
    const int64_t mine = lane < items ? pieces(lane) : 0;
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    Share s = cut_share(__shfl_sync(0xffffffffu, inc, 31), unit, units);
    const bool here = inc - mine <= s.begin && s.begin < inc;
    const int at = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    s.item = at < 0 ? items : at;
    s.offset = at < 0 ? 0 : s.begin - __shfl_sync(0xffffffffu, inc - mine, at);
    return s;
  }
  int64_t mine = 0, total = 0;
  for (int i = tid; i < items; i += nt) mine += pieces(i);
  int64_t before = block_scan<int64_t>(mine, scratch, total);
  Share s = cut_share(total, unit, units);
  if (tid == 0) {
    found[0] = items;
    found[1] = 0;
  }
  __syncthreads();
  if (items <= nt) {  // `mine` is one item
    if (before <= s.begin && s.begin < before + mine) {
      found[0] = tid;
      found[1] = s.begin - before;
    }
  } else {
    int64_t run = 0;
    for (int base = 0; base < items; base += nt) {
      const int64_t x = base + tid < items ? pieces(base + tid) : 0;
      int64_t sum;
      const int64_t at = run + block_scan<int64_t>(x, scratch, sum);
      if (at <= s.begin && s.begin < at + x) {
        found[0] = base + tid;
        found[1] = s.begin - at;
      }
      run += sum;
      if (run > s.begin) break;
    }
  }
  __syncthreads();
  s.item = static_cast<int32_t>(found[0]);
  s.offset = found[1];
  return s;
}

// The unit whose share holds flat piece x.
__device__ __forceinline__ int unit_of(int64_t x, int64_t total, int units) {
  int64_t u = x * units / total;
#pragma unroll 1
  while (u + 1 < units && total * (u + 1) / units <= x) ++u;
#pragma unroll 1
  while (u > 0 && total * u / units > x) --u;
  return static_cast<int>(u);
}

// ---- the join -----------------------------------------------------------------

// Sums of the rows that shares cut. Work is one warp for each row and 128
// columns where a request lies in a few shares, and a whole CTA (its warps take
// the shares in turn) where it lies in many: a request cut into a hundred
// parts and a hundred requests cut in two both fill the SMs in one wave. 5 to 12
// us a call: launch, read-back of the parts (up to 40 MB, mostly from L2), and
// the arithmetic of addresses. CTAs of 512 threads, or six or eight an SM, a
// whole row a warp, or references reduced over the lanes, measured slower.
//   part i of a note by CTA c is in the slots of CTA c + i * stride;
//   valid(note, c, row): whether the row exists;
//   emit(note, c, row, d, sums, top, l): columns d to d + 3 of the unnormalised
//   row (to be multiplied by 1 / l), its reference and sum. d is lane * 4 + 128 k:
//   whoever has d == 0 writes the log sum.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinFew = 8;        // parts that one warp adds up
constexpr int kJoinNotes = 512;    // notes at most (a unit has more than one share only while CTAs fit the SMs)
constexpr int kJoinCtasPerSm = 4;

template <class Valid, class Emit>
__device__ __forceinline__ void join_rows(const Workspace& ws, int notes, int stride, int rows, int dv,
                                          int64_t slot_floats, Valid valid, Emit emit) {
  __shared__ int16_t few[kJoinNotes], many[kJoinNotes];
  __shared__ int n_few, n_many;
  __shared__ float4 sums[kJoinThreads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the notes in their order, the same in every CTA: it decides who does what
  if (warp == 0) {
    int a = 0, b = 0;
    for (int i0 = 0; i0 < notes; i0 += 32) {
      const int i = i0 + lane;
      const JoinNote note = i < notes ? ws.notes[i] : JoinNote{-1, 0, 0, 0};
      const bool one = note.item >= 0 && note.parts <= kJoinFew, other = note.item >= 0 && !one;
      const uint32_t ones = __ballot_sync(0xffffffffu, one), others = __ballot_sync(0xffffffffu, other);
      const uint32_t below = (1u << lane) - 1;
      if (one) few[a + __popc(ones & below)] = static_cast<int16_t>(i);
      if (other) many[b + __popc(others & below)] = static_cast<int16_t>(i);
      a += __popc(ones);
      b += __popc(others);
    }
    if (lane == 0) {
      n_few = a;
      n_many = b;
    }
  }
  __syncthreads();
  if (n_few + n_many == 0) return;
  const int quarters = (dv + 127) / 128;
  const bool vec = dv % 4 == 0;
  auto slot_of = [&](int cta, int i) {  // part 0 is the noting share's own end, the others begin their shares
    return ws.slots + ((cta + static_cast<int64_t>(i) * stride) * 2 + (i == 0 ? 1 : 0)) * slot_floats;
  };
  auto values = [&](int cta, int row, int d, int i) {
    const float* o = slot_of(cta, i) + static_cast<int64_t>(row) * dv + d;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (vec) {
      if (d < dv) x = *reinterpret_cast<const float4*>(o);
    } else {
      if (d < dv) x.x = o[0];
      if (d + 1 < dv) x.y = o[1];
      if (d + 2 < dv) x.z = o[2];
      if (d + 3 < dv) x.w = o[3];
    }
    return x;
  };
  // adds parts i0, i0 + step, ... of a row's columns d to d + 3 under the reference `top`
  auto add = [&](int cta, int row, int d, int i0, int parts, int step, float top, float4& a, float& l) {
    const int64_t ml = static_cast<int64_t>(rows) * dv + 2 * row;
#pragma unroll 4
    for (int i = i0; i < parts; i += step) {
      const float* slot = slot_of(cta, i);
      const float m = slot[ml], part_l = slot[ml + 1];
      const float4 x = values(cta, row, d, i);
      if (part_l == 0.0f) continue;  // the row saw nothing there (a NaN among its scores makes a sum of NaN, which counts)
      const float w = exp2f(m - top);
      l += w * part_l;
      a.x += w * x.x;
      a.y += w * x.y;
      a.z += w * x.z;
      a.w += w * x.w;
    }
  };
  auto top_of = [&](int cta, int row, int parts) {
    const int64_t ml = static_cast<int64_t>(rows) * dv + 2 * row;
    float top = -INFINITY;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, slot_of(cta, i)[ml]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
  };
  for (int x = blockIdx.x * kJoinWarps + warp; x < n_few * rows * quarters; x += gridDim.x * kJoinWarps) {
    const int cta = few[x / (rows * quarters)], row = x / quarters % rows, d = x % quarters * 128 + lane * 4;
    const JoinNote note = ws.notes[cta];
    if (!valid(note, cta, row)) continue;
    // four parts at a time, all of their loads before any is used; every lane has the references and sums
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f, top = -INFINITY;
    for (int i0 = 0; i0 < note.parts; i0 += 4) {
      float4 o[4];
      float m[4], part_l[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool in = i0 + k < note.parts;
        const float* ml = slot_of(cta, in ? i0 + k : 0) + static_cast<int64_t>(rows) * dv + 2 * row;
        m[k] = in ? ml[0] : -INFINITY;
        part_l[k] = in ? ml[1] : 0.0f;
        o[k] = in ? values(cta, row, d, i0 + k) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      const float next = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), top);
      if (i0 > 0 && l != 0.0f) {
        const float keep = exp2f(top - next);
        l *= keep;
        a.x *= keep;
        a.y *= keep;
        a.z *= keep;
        a.w *= keep;
      }
      top = next;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (part_l[k] == 0.0f) continue;
        const float w = exp2f(m[k] - top);
        l += w * part_l[k];
        a.x += w * o[k].x;
        a.y += w * o[k].y;
        a.z += w * o[k].z;
        a.w += w * o[k].w;
      }
    }
    __syncwarp();
    if (d < dv) emit(note, cta, row, d, a, top, l);
  }
  for (int x = blockIdx.x; x < n_many * rows * quarters; x += gridDim.x) {
    const int cta = many[x / (rows * quarters)], row = x / quarters % rows, d = x % quarters * 128 + lane * 4;
    const JoinNote note = ws.notes[cta];
    if (!valid(note, cta, row)) continue;  // the same for the whole CTA
    const float top = top_of(cta, row, note.parts);
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
    add(cta, row, d, warp, note.parts, kJoinWarps, top, a, l);
    __shared__ float sums_l[kJoinWarps];
    sums[tid] = a;
    if (lane == 0) sums_l[warp] = l;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int k = 1; k < kJoinWarps; ++k) {
        const float4 y = sums[k * 32 + lane];
        a.x += y.x;
        a.y += y.y;
        a.z += y.z;
        a.w += y.w;
        l += sums_l[k];
      }
      if (d < dv) emit(note, cta, row, d, a, top, l);
    }
    __syncthreads();
  }
}

// ---- the body for any sizes -------------------------------------------------

constexpr int kGenRows = 8;    // rows of one pass: a warp each
constexpr int kGenKeys = 32;   // keys of a tile: a lane each
constexpr int kGenThreads = kGenRows * 32;
constexpr int kGenCols = PMG_MAX_ENTRY / kGenThreads;  // value columns of a thread

struct GenSmem {
  float* q;      // [kGenRows][E]
  float* k;      // [kGenKeys][E + 1]
  float* p;      // [kGenRows][kGenKeys]
  float* scale;  // [kGenRows]
};

inline int general_smem(int E) { return (kGenRows * E + kGenKeys * (E + 1) + kGenRows * kGenKeys + kGenRows) * 4; }

__device__ __forceinline__ GenSmem general_smem_at(uint8_t* base, int E) {
  GenSmem s;
  s.q = reinterpret_cast<float*>(base);
  s.k = s.q + kGenRows * E;
  s.p = s.k + kGenKeys * (E + 1);
  s.scale = s.p + kGenRows * kGenKeys;
  return s;
}

// Keys [j0, j1) for up to 8 rows whose queries are in s.q: one pass with the
// running maximum m (log2 domain) and sum l of each row, all in 32 bits.
//   load(j, e): element e of key j, or NaN-free 0;  seen(row, j);
//   value(j - tile, j, d): element d of the value of key j (only called where some row sees j)
template <class Load, class Seen, class Value>
__device__ __forceinline__ void general_rows(const GenSmem& s, int E, int dv, int64_t j0, int64_t j1, float sm_log2,
                                             Load load, Seen seen, Value value, float (&acc)[kGenRows][kGenCols],
                                             float& m, float& l) {
  const int tid = threadIdx.x, lane = tid & 31, row = tid >> 5;
#pragma unroll
  for (int r = 0; r < kGenRows; ++r)
#pragma unroll
    for (int c = 0; c < kGenCols; ++c) acc[r][c] = 0.0f;
  m = -INFINITY;
  l = 0.0f;
  for (int64_t t = j0; t < j1; t += kGenKeys) {
    const int n = static_cast<int>(min(static_cast<int64_t>(kGenKeys), j1 - t));
    __syncthreads();
    for (int j = row; j < kGenKeys; j += kGenRows)
      for (int e = lane; e < E; e += 32) s.k[j * (E + 1) + e] = j < n ? load(t + j, e) : 0.0f;
    __syncthreads();
    const bool mine = lane < n && seen(row, t + lane);
    float x = 0.0f;
    for (int e = 0; e < E; ++e) x += s.q[row * E + e] * s.k[lane * (E + 1) + e];
    x = mine ? x * sm_log2 : -INFINITY;
    float top = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float next = fmaxf(m, top);
    const float base = next == -INFINITY ? 0.0f : next;
    const float w = mine ? exp2f(x - base) : 0.0f;
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float keep = m == -INFINITY ? 0.0f : exp2f(m - base);
    l = l * keep + sum;
    m = next;
    s.p[row * kGenKeys + lane] = w;
    if (lane == 0) s.scale[row] = keep;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kGenRows; ++r)
#pragma unroll
      for (int c = 0; c < kGenCols; ++c) acc[r][c] *= s.scale[r];
    for (int j = 0; j < n; ++j) {
      float w8[kGenRows];
      bool any = false;
#pragma unroll
      for (int r = 0; r < kGenRows; ++r) {
        w8[r] = s.p[r * kGenKeys + j];
        any |= w8[r] != 0.0f;
      }
      if (!any) continue;
#pragma unroll
      for (int c = 0; c < kGenCols; ++c) {
        const int d = tid + c * kGenThreads;
        if (d < dv) {
          const float v = value(j, t + j, d);
#pragma unroll
          for (int r = 0; r < kGenRows; ++r)
            if (w8[r] != 0.0f) acc[r][c] += w8[r] * v;
        }
      }
    }
  }
}

}  // namespace pmg_mla
