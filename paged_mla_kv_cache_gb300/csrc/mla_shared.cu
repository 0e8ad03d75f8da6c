// Absorbed latent attention of requests behind shared prefixes
// (pmg_latent_decode_shared): the C entry.
//
// Mathematics: a row's weights over its prefix and over its own entries have
// sums (o1, m1, l1) and (o2, m2, l2), unnormalised under references m; with m =
// max(m1, m2) and w_i = 2^(m_i - m), out = (w1 o1 + w2 o2) / (w1 l1 + w2 l2).
//
// The prefix is a product of few entries with the rows of many requests, which
// is bound by the tensor core from a few hundred rows on; the own entries are a
// decode as before. Two passes leave (o, m, l) of every row (mla_decode.cuh), in
// 32 bits: 2 KB a row and pass, written and read once, mostly in L2. The join adds
// them up, and the parts of rows whose keys several shares held, in their order.
// The passes run beside each other where the first leaves SMs free. (Each with a
// join of its own, the second's rows joined as they were finished: four launches
// one after the other, 33 us for four requests behind 513 entries.)
#include <algorithm>

#include "mla_decode.cuh"
#include "pmg_long.h"

namespace pmg_mla {
namespace {

// What a pass left.
struct PassRows {
  Workspace ws;
  int64_t slot_floats;
  int32_t slot_rows, stride, notes;  // rows of a slot, CTAs between the parts of a row, CTAs that may have noted one
  const float* state;
  const float* state_ml;
  const RowNote* rows;
};

struct JoinParams {
  PassRows pass[2];        // prefixes, own entries
  const int32_t* covered;
  int32_t rows, H, q_len, dv;
  void* out;
  int64_t or_stride, ot_stride, oh_stride;
  float* lse;
};

// A warp takes a row's next 128 columns. Rows that a pass left in many parts are
// taken by a whole CTA, from the list of the CTAs that noted one, its warps the
// parts in turn: more than kJoinFew for each time that the CTAs would have to
// take a task (a CTA takes about 3 us a task, a warp 1 us and 0.2 a part; 1024 rows
// of 10 parts took 20 us as tasks of CTAs).
template <class TQ>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtasPerSm) shared_join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ float4 sums[kJoinThreads];
  __shared__ float sums_l[kJoinWarps], tops[kJoinWarps];
  pdl_entry();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int dv = p.dv, quarters = (dv + 127) / 128, per_req = p.q_len * p.H;
  const bool vec = dv % 4 == 0;
  const int covered0 = p.covered[0] * per_req, covered1 = p.covered[1] * per_req;
  // which notes are of rows in many parts, looked up by all threads at once: thread t notes t, t + 256, ...
  const int n0 = p.pass[0].notes, notes = n0 + p.pass[1].notes;
  const int64_t turns = (static_cast<int64_t>(p.rows) * quarters + gridDim.x - 1) / gridDim.x;
  const int few = static_cast<int>(min(kJoinFew * turns, static_cast<int64_t>(INT32_MAX)));
  uint32_t mine = 0;
#pragma unroll
  for (int k = 0; k < 2 * kJoinNotes / kJoinThreads; ++k) {
    const int i = tid + k * kJoinThreads;
    if (i < notes) {
      const JoinNote& note = p.pass[i < n0 ? 0 : 1].ws.notes[i < n0 ? i : i - n0];
      if (note.item >= 0 && note.parts > few) mine |= 1u << k;
    }
  }
  // parts of a row: of its prefix, then of its own entries
  struct Row {
    RowNote note[2];
    int n[2];
  };
  auto row_of = [&](int row) {
    Row r;
    const bool has = row >= covered0 && row < covered1;
    r.note[0] = has ? p.pass[0].rows[row] : RowNote{0, 0, 0};
    r.note[1] = p.pass[1].rows[row];
    r.n[0] = has ? max(static_cast<int>(r.note[0].parts), 1) : 0;
    r.n[1] = max(static_cast<int>(r.note[1].parts), 1);
    return r;
  };
  // reference and sum of part i, and its columns d to d + 3
  auto place = [&](const Row& r, int row, int i, const float*& ml) {
    const int k = i < r.n[0] ? 0 : 1;
    const PassRows& x = p.pass[k];
    const RowNote note = k == 0 ? r.note[0] : r.note[1];
    i -= k == 0 ? 0 : r.n[0];
    if (note.parts == 0) {
      ml = x.state_ml + 2 * static_cast<int64_t>(row);
      return x.state + static_cast<int64_t>(row) * dv;
    }
    // part 0 is the noting share's own end, the others begin their shares
    const float* slot = x.ws.slots + ((note.cta + static_cast<int64_t>(i) * x.stride) * 2 + (i == 0 ? 1 : 0)) * x.slot_floats;
    ml = slot + static_cast<int64_t>(x.slot_rows) * dv + 2 * note.row;
    return slot + static_cast<int64_t>(note.row) * dv;
  };
  auto values = [&](const float* o, int d) {
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (vec) {
      if (d < dv) y = *reinterpret_cast<const float4*>(o + d);
    } else {
      if (d < dv) y.x = o[d];
      if (d + 1 < dv) y.y = o[d + 1];
      if (d + 2 < dv) y.z = o[d + 2];
      if (d + 3 < dv) y.w = o[d + 3];
    }
    return y;
  };
  auto scale = [](float4& a, float& l, float w) {
    l *= w;
    a.x *= w;
    a.y *= w;
    a.z *= w;
    a.w *= w;
  };
  auto add = [](float4& a, float& l, float w, const float4& x, float part_l) {
    l += w * part_l;
    a.x += w * x.x;
    a.y += w * x.y;
    a.z += w * x.z;
    a.w += w * x.w;
  };
  auto emit = [&](int row, int d, const float4& a, float top, float l) {
    if (d >= dv) return;
    if (d == 0 && p.lse != nullptr) p.lse[row] = l != 0.0f ? (top + log2f(l)) * kLn2 : -INFINITY;
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    const int req = row / per_req, rr = row - req * per_req;
    TQ* out = static_cast<TQ*>(p.out) + req * p.or_stride + (rr / p.H) * p.ot_stride + (rr % p.H) * p.oh_stride + d;
    const float y[4] = {a.x * inv, a.y * inv, a.z * inv, a.w * inv};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (d + k < dv) out[k] = from_f<TQ>(y[k]);
  };
  // Sums of parts i0, i0 + step, ... of a row, kAhead at a time, all of their loads before any is used; every lane has the
  // references and sums.
  constexpr int kAhead = 4;
  auto sum = [&](const Row& r, int row, int d, int i0, int step, float4& a, float& l, float& top) {
    a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    l = 0.0f;
    top = -INFINITY;
    const int parts = r.n[0] + r.n[1];
    for (; i0 < parts; i0 += kAhead * step) {
      float4 o[kAhead];
      float m[kAhead], part_l[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        m[k] = -INFINITY;
        part_l[k] = 0.0f;
        o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i0 + k * step < parts) {
          const float* ml;
          const float* from = place(r, row, i0 + k * step, ml);
          m[k] = ml[0];  // (slots of odd rows and columns: not aligned to two)
          part_l[k] = ml[1];
          o[k] = values(from, d);
        }
      }
      // (a part whose sum is 0 saw nothing: its reference may be anything; a NaN among the scores makes a sum of NaN, which counts)
      float next = top;
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (part_l[k] != 0.0f) next = fmaxf(next, m[k]);
      if (l != 0.0f) scale(a, l, exp2f(top - next));
      top = next;
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (part_l[k] != 0.0f) add(a, l, exp2f(m[k] - top), o[k], part_l[k]);
    }
  };
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * kJoinWarps + warp; x < static_cast<int64_t>(p.rows) * quarters;
       x += gridDim.x * kJoinWarps) {
    const int row = static_cast<int>(x / quarters), d = static_cast<int>(x % quarters) * 128 + lane * 4;
    const Row r = row_of(row);
    if (r.n[0] > few || r.n[1] > few) continue;
    float4 a;
    float l, top;
    sum(r, row, d, 0, 1, a, l, top);
    emit(row, d, a, top, l);
  }
  // rows in many parts, if there are any (all of this is the same for a whole CTA)
  if (!__syncthreads_or(mine != 0)) return;
  __shared__ uint8_t is_many[2 * kJoinNotes];
  __shared__ uint16_t many[2 * kJoinNotes];
  __shared__ int n_many;
#pragma unroll
  for (int k = 0; k < 2 * kJoinNotes / kJoinThreads; ++k) is_many[tid + k * kJoinThreads] = mine >> k & 1;
  __syncthreads();
  if (warp == 0) {  // in the order of the notes
    int n = 0;
    for (int i0 = 0; i0 < notes; i0 += 32) {
      const bool one = is_many[i0 + lane];
      const uint32_t ones = __ballot_sync(0xffffffffu, one);
      if (one) many[n + __popc(ones & ((1u << lane) - 1))] = static_cast<uint16_t>(i0 + lane);
      n += __popc(ones);
    }
    if (lane == 0) n_many = n;
  }
  __syncthreads();
  int at = 0;  // tasks before those of the note at hand: CTAs take them in turn
  for (int y = 0; y < n_many; ++y) {
    const int i = many[y], k = i < n0 ? 0 : 1;
    const JoinNote note = p.pass[k].ws.notes[k == 0 ? i : i - n0];
    const int tasks = note.tile * quarters, begin = (static_cast<int>(blockIdx.x) - at % static_cast<int>(gridDim.x) + gridDim.x) % gridDim.x;
    at += tasks;
    for (int x = begin; x < tasks; x += gridDim.x) {
      const int row = note.head + x / quarters, d = x % quarters * 128 + lane * 4;
      const Row r = row_of(row);
      if (k == 1 && r.n[0] > few) continue;  // done with its prefix's
      float4 a;
      float l, top;
      sum(r, row, d, warp, kJoinWarps, a, l, top);
      sums[tid] = a;
      if (lane == 0) {
        sums_l[warp] = l;
        tops[warp] = top;
      }
      __syncthreads();
      if (warp == 0) {
        float all = -INFINITY;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w)
          if (sums_l[w] != 0.0f) all = fmaxf(all, tops[w]);
        a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        l = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w)
          if (sums_l[w] != 0.0f) add(a, l, exp2f(tops[w] - all), sums[w * 32 + lane], sums_l[w]);
        emit(row, d, a, all, l);
      }
      __syncthreads();
    }
  }
}

// The workspace: one of the attention calls for each pass, then what both leave of all rows, and the covered requests.
struct StateBytes {
  int64_t second, sums[2], ml[2], rows[2], covered, end;
  StateBytes(int sms, int64_t n, int32_t dv) {
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    second = up(workspace_bytes(sms));
    int64_t at = 2 * second;
    for (int i = 0; i < 2; ++i) {
      sums[i] = at;
      ml[i] = up(sums[i] + n * dv * 4);
      rows[i] = up(ml[i] + n * 8);
      at = up(rows[i] + n * static_cast<int64_t>(sizeof(RowNote)));
    }
    covered = at;
    end = covered + 256;
  }
};

PassRows rows_of(const DecodeParams& p) {
  return {p.ws, p.slot_floats, p.rows_per_group, p.groups, p.units > 1 ? p.units * p.groups : 0, p.state, p.state_ml, p.row_notes};
}

}  // namespace
}  // namespace pmg_mla

extern "C" int64_t pmg_shared_workspace(int64_t rows, int32_t latent_dim) {
  using namespace pmg_mla;
  int sms = 0;
  if (rows < 0 || rows > INT32_MAX || latent_dim < 1 || latent_dim > PMG_MAX_ENTRY || sm_count(&sms) != PMG_OK) return -1;
  return StateBytes(sms, rows, latent_dim).end;
}

extern "C" int pmg_latent_decode_shared(
    const void* q, int64_t q_req_stride, int64_t q_token_stride, int64_t q_head_stride, const void* cache,
    int64_t cache_block_stride, int64_t cache_token_stride, int64_t num_blocks, const int32_t* prefix_table,
    int64_t prefix_table_stride, const int32_t* prefix_lens, const int32_t* cu_groups, int32_t num_groups,
    const int32_t* block_table, int64_t block_table_stride, const int32_t* seq_lens, int32_t num_reqs, int32_t q_len,
    int32_t heads, int32_t latent_dim, int32_t rope_dim, int32_t block_size, int32_t q_dtype, int32_t cache_dtype,
    const float* scale, float sm_scale, void* out, int64_t out_req_stride, int64_t out_token_stride,
    int64_t out_head_stride, float* lse, void* workspace, int64_t workspace_bytes_given, int32_t* error_flag,
    void* stream, uint32_t options) {
  using namespace pmg_mla;
  DecodeParams p;
  int st = decode_params(p, q, q_req_stride, q_token_stride, q_head_stride, cache, cache_block_stride, cache_token_stride,
                         num_blocks, block_table, block_table_stride, seq_lens, num_reqs, q_len, heads, latent_dim,
                         rope_dim, block_size, q_dtype, cache_dtype, scale, sm_scale, out, out_req_stride,
                         out_token_stride, out_head_stride, lse, workspace, error_flag, options);
  if (st != PMG_OK) return st;
  if (num_groups < 0 || prefix_table_stride < 0) return PMG_ERR_ARG;
  if (num_groups > PMG_MAX_REQS || prefix_table_stride > INT32_MAX) return PMG_ERR_UNSUPPORTED;
  if (p.R == 0) return PMG_OK;
  const int64_t rows = static_cast<int64_t>(num_reqs) * q_len * heads;
  if (rows > INT32_MAX) return PMG_ERR_UNSUPPORTED;
  if (num_groups > 0 && (prefix_lens == nullptr || cu_groups == nullptr || (prefix_table == nullptr && prefix_table_stride > 0)))
    return PMG_ERR_NULL;
  if (!aligned(prefix_table, 4) || !aligned(prefix_lens, 4) || !aligned(cu_groups, 4) || !aligned(workspace, 256))
    return PMG_ERR_ALIGN;
  int sms = 0;
  st = sm_count(&sms);
  if (st != PMG_OK) return st;
  const StateBytes at(sms, rows, latent_dim);
  if (workspace_bytes_given < at.end) return PMG_ERR_ARG;
  p.ws = workspace_at(workspace, sms);
  if (num_groups == 0) return decode_alone(p, q_dtype, cache_dtype, sms, stream, options);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  auto keep = [&](DecodeParams& x, int i) {
    x.ws = workspace_at(base + i * at.second, sms);
    x.state = reinterpret_cast<float*>(base + at.sums[i]);
    x.state_ml = reinterpret_cast<float*>(base + at.ml[i]);
    x.row_notes = reinterpret_cast<RowNote*>(base + at.rows[i]);
    x.covered = reinterpret_cast<int32_t*>(base + at.covered);
  };
  DecodeParams prefix = p;
  prefix.cu = cu_groups;
  prefix.reqs = num_reqs;
  prefix.R = num_groups;
  prefix.bt = prefix_table;
  prefix.bt_stride = prefix_table_stride;
  prefix.seq_lens = prefix_lens;
  keep(prefix, 0);
  keep(p, 1);
  st = run_prefix(prefix, q_dtype, cache_dtype, sms, stream, options);
  if (st == PMG_OK) st = run_decode(p, q_dtype, cache_dtype, sms, stream, options);
  if (st != PMG_OK) return st;
  JoinParams j{};
  j.pass[0] = rows_of(prefix);
  j.pass[1] = rows_of(p);
  j.covered = p.covered;
  j.rows = static_cast<int32_t>(rows);
  j.H = heads;
  j.q_len = q_len;
  j.dv = latent_dim;
  j.out = out;
  j.or_stride = out_req_stride;
  j.ot_stride = out_token_stride;
  j.oh_stride = out_head_stride;
  j.lse = lse;
  const auto join = q_dtype == PMG_BF16 ? shared_join_kernel<bf16> : q_dtype == PMG_FP16 ? shared_join_kernel<f16> : shared_join_kernel<float>;
  return launch(join, dim3(static_cast<unsigned>(kJoinCtasPerSm * sms)), kJoinThreads, 0, stream, j);
}
