// Absorbed latent attention over the paged cache (pmg_latent_decode): the
// kernel for any sizes, the join of split requests, and the C entry.
//
// Mathematics: with e_j the entries of a request, s_j = sm_scale q . e_j over
// the whole entry, out = sum_j exp(s_j - lse) e_j[0:latent]. Softmax runs in
// base 2 (scores are multiplied by sm_scale * log2 e once) with a running
// maximum, so an entry is read once for both products.
#include <algorithm>

#include "mla_decode.cuh"
#include "mla_decode_tc.cuh"

namespace pmg_mla {
namespace {

// Any sizes, types, strides and pages. A CTA takes 8 rows (a warp each) and
// tiles of 32 keys held in shared memory in 32 bits; scores are dot products
// of a lane, values are summed by columns of a thread. It is bound by shared
// memory reads of the scores (one 4-byte word a multiply), far above the
// cache's bytes: it exists for what the tensor-core kernel does not take. As a
// prefix pass it takes 16 requests of 16 heads behind 4096 entries in 1.05 ms with
// their own 100 entries and the join (on the tensor core 36 us).
template <class TQ, class TC, bool kPrefix>
__global__ void __launch_bounds__(kGenThreads) decode_general_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t scratch[33], found[2];
  pass_entry<kPrefix>(p);
  const int E = p.dv + p.dr;
  const GenSmem s = general_smem_at(smem, E);
  const int unit = kPrefix ? blockIdx.x : blockIdx.x / p.groups, group = kPrefix ? 0 : blockIdx.x % p.groups;
  const Share share = find_share(
      [&](int b) -> int64_t {
        if constexpr (kPrefix) return prefix_pieces<0>(p, b);
        else return decode_tiles(p, b);
      },
      p.R, unit, p.units, scratch, found);
  const int tid = threadIdx.x, lane = tid & 31, row = tid >> 5;
  if constexpr (kPrefix) {
    if (blockIdx.x == 0) note_covered(p, tid, kGenThreads, *reinterpret_cast<int32_t*>(scratch));
  }
  const int rows = p.q_len * p.H;
  const int g0 = group * p.rows_per_group;
  const float scale = sizeof(TC) == 1 && p.scale != nullptr ? *p.scale : 1.0f;
  const bool keeps = kPrefix || p.state != nullptr;  // rows are left for the join over shared prefixes
  JoinNote note{-1, 0, 0, 0};
  int bad = 0;
  int64_t at = share.begin;
  int64_t tile = share.offset;
  PrefixItems<0> it(p, share);
  for (int b = share.item; at < share.end; ++b, tile = 0) {
    DecodeLen len;
    int64_t tiles, n, row0;  // tiles of the item and of this share, the item's first row of all rows of the call
    int n_rows;
    if constexpr (kPrefix) {
      if (!it.next()) break;
      b = it.b;
      len = {it.full_len, it.len, 0};
      tile = it.tile;
      tiles = max(it.tiles, 1);
      n = it.len > 0 ? it.n : 1;
      row0 = it.row0;
      n_rows = it.n_rows;
    } else {
      len = decode_len(p, b);
      tiles = decode_tiles(p, b);
      n = min(tiles - tile, share.end - at);
      row0 = static_cast<int64_t>(b) * rows + g0;
      n_rows = min(p.rows_per_group, rows - g0);
    }
    bad |= len.bad;
    __syncthreads();
    {
      const int64_t rr = row0 + row, t = rr / p.H;  // a warp loads the row that it scores
      const TQ* q = reinterpret_cast<const TQ*>(p.q) + t / p.q_len * p.qr_stride + t % p.q_len * p.qt_stride + rr % p.H * p.qh_stride;
      for (int e = lane; e < E; e += 32) s.q[row * E + e] = row < n_rows ? to_f(q[e]) : 0.0f;
    }
    const int limit_row = min(g0 + row, rows - 1);
    const int64_t limit = kPrefix ? len.full : static_cast<int64_t>(len.full) - p.q_len + 1 + limit_row / p.H;  // keys this row sees
    const int32_t* table = p.bt + static_cast<int64_t>(b) * p.bt_stride;
    auto block_at = [&](int64_t j) { return table[static_cast<uint32_t>(j) / static_cast<uint32_t>(p.B)]; };
    auto load = [&](int64_t j, int e) -> float {
      const int32_t id = block_at(j);
      if (id < 0 || id >= p.num_blocks) {
        bad |= PMG_FLAG_PHYS_BLOCK;
        return 0.0f;
      }
      return scale * to_f(reinterpret_cast<const TC*>(p.cache)[id * p.blk_stride + (j % p.B) * p.tok_stride + e]);
    };
    auto seen = [&](int, int64_t j) {
      const int32_t id = block_at(j);
      return j < limit && id >= 0 && id < p.num_blocks;
    };
    auto value = [&](int j, int64_t, int d) { return s.k[j * (E + 1) + d]; };
    float acc[kGenRows][kGenCols], m, l;
    general_rows(s, E, p.dv, tile * kDecodeTile, min((tile + n) * kDecodeTile, static_cast<int64_t>(len.use)),
                 p.sm_scale * kLog2e, load, seen, value, acc, m, l);
    const bool whole = tile == 0 && n == tiles;
    const int parts = whole || tile > 0 ? 0 : unit_of(at + tiles - 1, share.total, share.units) - unit + 1;
    if (parts > 0) note = {b, parts, keeps ? static_cast<int32_t>(row0) : 0, keeps ? n_rows : 0};
    // where the rows go that are not finished here: a slot of the workspace, or the state of a pass
    float* slot = p.ws.slots + (static_cast<int64_t>(blockIdx.x) * 2 + (tile == 0 ? 1 : 0)) * p.slot_floats;
    float* slot_ml = slot + p.rows_per_group * p.dv;
    const bool finished = whole && !keeps;
    if (whole && keeps) {
      slot = p.state + row0 * p.dv;
      slot_ml = p.state_ml + 2 * row0;
    }
    __syncthreads();
    if (lane == 0) {  // what every row is multiplied by, and its log sum
      s.scale[row] = finished ? (l != 0.0f ? 1.0f / l : 0.0f) : 1.0f;
      if (row < n_rows) {
        if (finished && p.lse != nullptr) p.lse[row0 + row] = l != 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
        if (!finished) {
          slot_ml[2 * row] = m;
          slot_ml[2 * row + 1] = l;
        }
        if (keeps && (whole || tile == 0))
          p.row_notes[row0 + row] = {static_cast<uint16_t>(whole ? 0 : blockIdx.x), static_cast<uint16_t>(parts), row};
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kGenRows; ++r) {
      if (r >= n_rows) continue;
      const int rr = g0 + r;
      TQ* out = reinterpret_cast<TQ*>(p.out) + b * p.or_stride + (rr / p.H) * p.ot_stride + (rr % p.H) * p.oh_stride;
#pragma unroll
      for (int c = 0; c < kGenCols; ++c) {
        const int d = tid + c * kGenThreads;
        if (d >= p.dv) continue;
        if (finished) out[d] = from_f<TQ>(acc[r][c] * s.scale[r]);
        else slot[r * p.dv + d] = acc[r][c];
      }
    }
    at += n;
  }
  if (tid == 0 && p.units > 1) p.ws.notes[blockIdx.x] = note;  // one unit cuts nothing
  set_flag(p.err, bad);
  pass_exit<kPrefix>(p);
}

template <class TQ>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtasPerSm) decode_join_kernel(const __grid_constant__ DecodeParams p) {
  pdl_entry();
  const int rows = p.q_len * p.H;
  auto row_of = [&](int cta, int row) { return cta % p.groups * p.rows_per_group + row; };
  join_rows(
      p.ws, p.units * p.groups, p.groups, p.rows_per_group, p.dv, p.slot_floats,
      [&](const JoinNote&, int cta, int row) { return row_of(cta, row) < rows; },
      [&](const JoinNote& note, int cta, int row, int d, const float4& a, float top, float l) {
        const int rr = row_of(cta, row);
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        if (d == 0 && p.lse != nullptr)
          p.lse[static_cast<int64_t>(note.item) * rows + rr] = l != 0.0f ? (top + log2f(l)) * kLn2 : -INFINITY;
        TQ* out = static_cast<TQ*>(p.out) + note.item * p.or_stride + (rr / p.H) * p.ot_stride + (rr % p.H) * p.oh_stride + d;
        const float y[4] = {a.x * inv, a.y * inv, a.z * inv, a.w * inv};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (d + k < p.dv) out[k] = from_f<TQ>(y[k]);
      });
}

using Kernel = void (*)(const DecodeParams);

template <bool kPrefix>
Kernel general_kernel(int q_dtype, int cache_dtype) {
  const bool fp8 = cache_dtype == PMG_FP8_E4M3;
  switch (q_dtype) {
    case PMG_BF16: return fp8 ? decode_general_kernel<bf16, e4m3, kPrefix> : decode_general_kernel<bf16, bf16, kPrefix>;
    case PMG_FP16: return fp8 ? decode_general_kernel<f16, e4m3, kPrefix> : decode_general_kernel<f16, f16, kPrefix>;
    default: return fp8 ? decode_general_kernel<float, e4m3, kPrefix> : decode_general_kernel<float, float, kPrefix>;
  }
}

template <bool kPrefix>
int run_general(DecodeParams& p, int q_dtype, int cache_dtype, void* stream) {
  p.slot_floats = (static_cast<int64_t>(p.rows_per_group) * (p.dv + 2) + 3) / 4 * 4;
  const Kernel k = general_kernel<kPrefix>(q_dtype, cache_dtype);
  const int st = allow_smem(reinterpret_cast<const void*>(k), general_smem(PMG_MAX_ENTRY));
  if (st != PMG_OK) return st;
  return launch(k, dim3(static_cast<unsigned>(p.units) * p.groups), kGenThreads, general_smem(p.dv + p.dr), stream, p);
}

}  // namespace
}  // namespace pmg_mla

namespace pmg_mla {

int decode_params(DecodeParams& p, const void* q, int64_t q_req_stride, int64_t q_token_stride, int64_t q_head_stride,
                  const void* cache, int64_t cache_block_stride, int64_t cache_token_stride, int64_t num_blocks,
                  const int32_t* block_table, int64_t block_table_stride, const int32_t* seq_lens, int32_t num_reqs,
                  int32_t q_len, int32_t heads, int32_t latent_dim, int32_t rope_dim, int32_t block_size,
                  int32_t q_dtype, int32_t cache_dtype, const float* scale, float sm_scale, void* out,
                  int64_t out_req_stride, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                  void* workspace, int32_t* error_flag, uint32_t options) {
  p = DecodeParams{};
  const int eq = elem_bytes(q_dtype), ec = elem_bytes(cache_dtype);
  if (eq < 2 || ec == 0 || (cache_dtype != q_dtype && cache_dtype != PMG_FP8_E4M3)) return PMG_ERR_DTYPE;
  if (num_reqs < 0 || q_len < 0 || heads < 0 || latent_dim < 1 || rope_dim < 0 || block_size < 1 || num_blocks < 0 ||
      block_table_stride < 0 || !(sm_scale >= 0.0f) || (options & ~PMG_OPT_FORCE_GENERAL))
    return PMG_ERR_ARG;
  for (const int64_t s : {q_req_stride, q_token_stride, q_head_stride, cache_block_stride, cache_token_stride,
                          out_req_stride, out_token_stride, out_head_stride})
    if (!stride_ok(s)) return PMG_ERR_ARG;
  if (static_cast<int64_t>(latent_dim) + rope_dim > PMG_MAX_ENTRY || num_blocks > INT32_MAX ||
      block_table_stride > INT32_MAX || num_reqs > PMG_MAX_REQS ||
      static_cast<int64_t>(q_len) * heads > (1 << 20))
    return PMG_ERR_UNSUPPORTED;
  if (num_reqs == 0 || q_len == 0 || heads == 0) return PMG_OK;
  if (q == nullptr || out == nullptr || seq_lens == nullptr || workspace == nullptr ||
      (cache == nullptr && num_blocks > 0) || (block_table == nullptr && block_table_stride > 0))
    return PMG_ERR_NULL;
  if (!aligned(q, eq) || !aligned(out, eq) || !aligned(cache, ec) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(scale, 4) || !aligned(lse, 4) || !aligned(workspace, 16) ||
      !aligned(error_flag, 4))
    return PMG_ERR_ALIGN;
  p.q = q;
  p.qr_stride = q_req_stride;
  p.qt_stride = q_token_stride;
  p.qh_stride = q_head_stride;
  p.cache = cache;
  p.blk_stride = cache_block_stride;
  p.tok_stride = cache_token_stride;
  p.num_blocks = num_blocks;
  p.bt = block_table;
  p.bt_stride = block_table_stride;
  p.seq_lens = seq_lens;
  p.R = num_reqs;
  p.q_len = q_len;
  p.H = heads;
  p.dv = latent_dim;
  p.dr = rope_dim;
  p.B = block_size;
  p.scale = scale;
  p.sm_scale = sm_scale;
  p.out = out;
  p.or_stride = out_req_stride;
  p.ot_stride = out_token_stride;
  p.oh_stride = out_head_stride;
  p.lse = lse;
  p.err = error_flag;
  return PMG_OK;
}

int run_decode(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream, uint32_t options) {
  const int rows = p.q_len * p.H;
  int st;
  if (!(options & PMG_OPT_FORCE_GENERAL) && decode_tc_takes(p, q_dtype, cache_dtype)) {
    st = decode_tc(p, q_dtype, cache_dtype, sms, stream);
  } else {
    p.rows_per_group = std::min(rows, kGenRows);
    p.groups = (rows + p.rows_per_group - 1) / p.rows_per_group;
    // as many shares as fill the SMs; more groups than that run whole requests
    p.units = std::max(1, sms / p.groups);
    st = run_general<false>(p, q_dtype, cache_dtype, stream);
  }
  return st;
}

int run_prefix(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream, uint32_t options) {
  int st;
  if (!(options & PMG_OPT_FORCE_GENERAL) && decode_tc_takes(p, q_dtype, cache_dtype)) {
    st = prefix_tc(p, q_dtype, cache_dtype, sms, stream);
  } else {
    p.rows_per_group = kGenRows;
    p.groups = 1;
    p.units = sms;
    st = run_general<true>(p, q_dtype, cache_dtype, stream);
  }
  return st;
}

int decode_alone(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream, uint32_t options) {
  const int st = run_decode(p, q_dtype, cache_dtype, sms, stream, options);
  if (st != PMG_OK || p.units == 1) return st;
  const Kernel join = q_dtype == PMG_BF16 ? decode_join_kernel<bf16>
                      : q_dtype == PMG_FP16 ? decode_join_kernel<f16> : decode_join_kernel<float>;
  return launch(join, dim3(static_cast<unsigned>(kJoinCtasPerSm * sms)), kJoinThreads, 0, stream, p);
}

}  // namespace pmg_mla

extern "C" int64_t pmg_attention_workspace(void) {
  int sms = 0;
  if (pmg_mla::sm_count(&sms) != PMG_OK) return -1;
  return pmg_mla::workspace_bytes(sms);
}

extern "C" int pmg_latent_decode(const void* q, int64_t q_req_stride, int64_t q_token_stride, int64_t q_head_stride,
                                 const void* cache, int64_t cache_block_stride, int64_t cache_token_stride,
                                 int64_t num_blocks, const int32_t* block_table, int64_t block_table_stride,
                                 const int32_t* seq_lens, int32_t num_reqs, int32_t q_len, int32_t heads,
                                 int32_t latent_dim, int32_t rope_dim, int32_t block_size, int32_t q_dtype,
                                 int32_t cache_dtype, const float* scale, float sm_scale, void* out,
                                 int64_t out_req_stride, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                                 void* workspace, int64_t workspace_bytes_given, int32_t* error_flag, void* stream,
                                 uint32_t options) {
  using namespace pmg_mla;
  DecodeParams p;
  int st = decode_params(p, q, q_req_stride, q_token_stride, q_head_stride, cache, cache_block_stride, cache_token_stride,
                         num_blocks, block_table, block_table_stride, seq_lens, num_reqs, q_len, heads, latent_dim,
                         rope_dim, block_size, q_dtype, cache_dtype, scale, sm_scale, out, out_req_stride,
                         out_token_stride, out_head_stride, lse, workspace, error_flag, options);
  if (st != PMG_OK || p.R == 0) return st;
  int sms = 0;
  st = sm_count(&sms);
  if (st != PMG_OK) return st;
  if (workspace_bytes_given < workspace_bytes(sms)) return PMG_ERR_ARG;
  p.ws = workspace_at(workspace, sms);
  return decode_alone(p, q_dtype, cache_dtype, sms, stream, options);
}
