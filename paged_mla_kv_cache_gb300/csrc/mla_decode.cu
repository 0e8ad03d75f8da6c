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
// cache's bytes: it exists for what the tensor-core kernel does not take.
template <class TQ, class TC>
__global__ void __launch_bounds__(kGenThreads) decode_general_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t scratch[33], found[2];
  pdl_entry();
  const int E = p.dv + p.dr;
  const GenSmem s = general_smem_at(smem, E);
  const int unit = blockIdx.x / p.groups, group = blockIdx.x % p.groups;
  const Share share = find_share([&](int b) { return decode_tiles(p, b); }, p.R, unit, p.units, scratch, found);
  const int tid = threadIdx.x, lane = tid & 31, row = tid >> 5;
  const int rows = p.q_len * p.H;
  const int g0 = group * p.rows_per_group;
  const int n_rows = min(p.rows_per_group, rows - g0);
  const float scale = sizeof(TC) == 1 && p.scale != nullptr ? *p.scale : 1.0f;
  JoinNote note{-1, 0, 0, 0};
  int bad = 0;
  int64_t at = share.begin;
  int64_t tile = share.offset;
  for (int b = share.item; at < share.end; ++b, tile = 0) {
    const DecodeLen len = decode_len(p, b);
    bad |= len.bad;
    const int64_t tiles = decode_tiles(p, b);
    const int64_t n = min(tiles - tile, share.end - at);
    __syncthreads();
    for (int i = tid; i < n_rows * E; i += kGenThreads) {
      const int rr = g0 + i / E;
      s.q[i] = to_f(reinterpret_cast<const TQ*>(p.q)[b * p.qr_stride + (rr / p.H) * p.qt_stride + (rr % p.H) * p.qh_stride + i % E]);
    }
    for (int i = n_rows * E + tid; i < kGenRows * E; i += kGenThreads) s.q[i] = 0.0f;
    const int limit_row = min(g0 + row, rows - 1);
    const int64_t limit = static_cast<int64_t>(len.full) - p.q_len + 1 + limit_row / p.H;  // keys this row sees
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
    if (!whole && tile == 0) {
      note.item = b;
      note.parts = unit_of(at + tiles - 1, share.total, share.units) - unit + 1;
    }
    float* slot = p.ws.slots + (static_cast<int64_t>(blockIdx.x) * 2 + (tile == 0 ? 1 : 0)) * p.slot_floats;
    __syncthreads();
    if (lane == 0) {  // what every row is multiplied by, and its log sum
      s.scale[row] = whole ? (l != 0.0f ? 1.0f / l : 0.0f) : 1.0f;
      if (row < n_rows) {
        const int rr = g0 + row;
        if (whole && p.lse != nullptr)
          p.lse[static_cast<int64_t>(b) * rows + rr] = l != 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
        if (!whole) {
          float* ml = slot + p.rows_per_group * p.dv + 2 * row;
          ml[0] = m;
          ml[1] = l;
        }
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
        if (whole) out[d] = from_f<TQ>(acc[r][c] * s.scale[r]);
        else slot[r * p.dv + d] = acc[r][c];
      }
    }
    at += n;
  }
  if (tid == 0 && p.units > 1) p.ws.notes[blockIdx.x] = note;  // one unit cuts nothing
  set_flag(p.err, bad);
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

Kernel general_kernel(int q_dtype, int cache_dtype) {
  const bool fp8 = cache_dtype == PMG_FP8_E4M3;
  switch (q_dtype) {
    case PMG_BF16: return fp8 ? decode_general_kernel<bf16, e4m3> : decode_general_kernel<bf16, bf16>;
    case PMG_FP16: return fp8 ? decode_general_kernel<f16, e4m3> : decode_general_kernel<f16, f16>;
    default: return fp8 ? decode_general_kernel<float, e4m3> : decode_general_kernel<float, float>;
  }
}

}  // namespace
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
  int sms = 0;
  int st = sm_count(&sms);
  if (st != PMG_OK) return st;
  if (workspace_bytes_given < workspace_bytes(sms)) return PMG_ERR_ARG;
  DecodeParams p{};
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
  p.ws = workspace_at(workspace, sms);
  p.err = error_flag;
  const int rows = q_len * heads;
  if (!(options & PMG_OPT_FORCE_GENERAL) && decode_tc_takes(p, q_dtype, cache_dtype)) {
    st = decode_tc(p, q_dtype, cache_dtype, sms, stream);
  } else {
    p.rows_per_group = std::min(rows, kGenRows);
    p.groups = (rows + p.rows_per_group - 1) / p.rows_per_group;
    // as many shares as fill the SMs; more groups than that run whole requests
    p.units = std::max(1, sms / p.groups);
    p.slot_floats = (static_cast<int64_t>(p.rows_per_group) * (p.dv + 2) + 3) / 4 * 4;
    const int E = p.dv + p.dr;
    const Kernel k = general_kernel(q_dtype, cache_dtype);
    st = allow_smem(reinterpret_cast<const void*>(k), general_smem(PMG_MAX_ENTRY));
    if (st != PMG_OK) return st;
    st = launch(k, dim3(static_cast<unsigned>(p.units) * p.groups), kGenThreads, general_smem(E), stream, p);
  }
  if (st != PMG_OK || p.units == 1) return st;
  const Kernel join = q_dtype == PMG_BF16 ? decode_join_kernel<bf16>
                      : q_dtype == PMG_FP16 ? decode_join_kernel<f16> : decode_join_kernel<float>;
  return launch(join, dim3(static_cast<unsigned>(kJoinCtasPerSm * sms)), kJoinThreads, 0, stream, p);
}
