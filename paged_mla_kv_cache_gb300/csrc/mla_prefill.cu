// Expanded latent attention of a chunk of new tokens (pmg_latent_prefill): the
// kernel for any sizes and the C entry.
//
// Mathematics: s_ij = sm_scale (q_i[:nope] . k_j + q_i[nope:] . pe_j), out_i =
// sum_j softmax_j(s_ij) v_j, joined with an earlier state by their log sums.
// The rotated key part stays one row a token: it is never copied out to the
// heads.
#include <algorithm>

#include "mla_prefill.cuh"
#include "mla_prefill_tc.cuh"

namespace pmg_mla {
namespace {

// Any sizes, types and strides: a CTA takes 8 query rows of one head at a time
// (see general_rows). It exists for what the tensor-core kernel does not take.
template <class T>
__global__ void __launch_bounds__(kGenThreads) prefill_general_kernel(const __grid_constant__ PrefillParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t scratch[33], found[2];
  pdl_entry();
  const int E = p.dn + p.dr;
  const GenSmem s = general_smem_at(smem, E);
  auto pieces = [&](int r) -> int64_t {
    return (static_cast<int64_t>(prefill_req(p, r).lq) + kGenRows - 1) / kGenRows * p.H;
  };
  const Share share = find_share(pieces, p.R, blockIdx.x, p.units, scratch, found);
  const int tid = threadIdx.x, lane = tid & 31, row = tid >> 5;
  int64_t offset = share.offset;
  int r = share.item;
  int bad = 0;
  if (blockIdx.x == 0)
    for (int i = tid; i < p.R; i += kGenThreads) bad |= prefill_req(p, i).bad;
  for (int64_t at = share.begin; at < share.end; ++at, ++offset) {
    PrefillReq x = prefill_req(p, r);
    int64_t n = pieces(r);
    while (offset >= n) {
      offset -= n;
      x = prefill_req(p, ++r);
      n = pieces(r);
    }
    const int h = static_cast<int>(offset % p.H);
    const int i0 = static_cast<int>(offset / p.H) * kGenRows;
    const int rows = min(kGenRows, x.lq - i0);
    __syncthreads();
    for (int i = tid; i < kGenRows * E; i += kGenThreads)
      s.q[i] = i < rows * E
                   ? to_f(reinterpret_cast<const T*>(p.q)[(x.q0 + i0 + i / E) * p.qt_stride + h * p.qh_stride + i % E])
                   : 0.0f;
    const int64_t shift = static_cast<int64_t>(x.lk) - x.lq + 1;
    const int64_t limit = p.causal ? min(static_cast<int64_t>(x.lk), shift + i0 + min(row, rows - 1)) : x.lk;
    const int64_t j1 = p.causal ? min(static_cast<int64_t>(x.lk), shift + i0 + rows - 1) : x.lk;
    const T* kb = reinterpret_cast<const T*>(p.k) + x.k0 * p.kt_stride + h * p.kh_stride;
    const T* pb = reinterpret_cast<const T*>(p.pe) + x.k0 * p.pe_stride;
    const T* vb = reinterpret_cast<const T*>(p.v) + x.k0 * p.vt_stride + h * p.vh_stride;
    auto load = [&](int64_t j, int e) {
      return to_f(e < p.dn ? kb[j * p.kt_stride + e] : pb[j * p.pe_stride + (e - p.dn)]);
    };
    auto seen = [&](int, int64_t j) { return j < limit; };
    auto value = [&](int, int64_t j, int d) { return to_f(vb[j * p.vt_stride + d]); };
    float acc[kGenRows][kGenCols], m, l;
    general_rows(s, E, p.dv, 0, j1, p.sm_scale * kLog2e, load, seen, value, acc, m, l);
    __syncthreads();
    if (lane == 0) {
      float lse = l != 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
      float now = l != 0.0f ? 1.0f / l : 0.0f, before = 0.0f;
      if (row < rows) {
        const int64_t at_lse = static_cast<int64_t>(x.q0 + i0 + row) * p.H + h;
        if (p.prev_lse != nullptr) {
          const Joined g = join_state(lse, p.prev_lse[at_lse]);
          now *= g.now;
          before = g.before;
          lse = g.lse;
        }
        if (p.lse != nullptr) p.lse[at_lse] = lse;
      }
      s.scale[row] = now;
      s.p[row] = before;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGenRows; ++i) {
      if (i >= rows) continue;
      const int64_t t = x.q0 + i0 + i;
      T* out = reinterpret_cast<T*>(p.out) + t * p.ot_stride + h * p.oh_stride;
      const T* prev = reinterpret_cast<const T*>(p.prev) + t * p.pt_stride + h * p.ph_stride;
      const float w = s.p[i];
#pragma unroll
      for (int c = 0; c < kGenCols; ++c) {
        const int d = tid + c * kGenThreads;
        if (d >= p.dv) continue;
        float y = acc[i][c] * s.scale[i];
        if (w != 0.0f) y += w * to_f(prev[d]);
        out[d] = from_f<T>(y);
      }
    }
  }
  set_flag(p.err, bad);
}

using Kernel = void (*)(const PrefillParams);

}  // namespace
}  // namespace pmg_mla

extern "C" int pmg_latent_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_nope,
                                  int64_t k_token_stride, int64_t k_head_stride, const void* k_pe,
                                  int64_t k_pe_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                                  const int32_t* cu_q, const int32_t* cu_k, int32_t num_reqs, int64_t total_q,
                                  int64_t total_k, int32_t heads, int32_t nope_dim, int32_t rope_dim, int32_t v_dim,
                                  int32_t dtype, float sm_scale, void* out, int64_t out_token_stride,
                                  int64_t out_head_stride, float* lse, const void* prev_out,
                                  int64_t prev_token_stride, int64_t prev_head_stride, const float* prev_lse,
                                  void* workspace, int64_t workspace_bytes_given, int32_t* error_flag, void* stream,
                                  uint32_t options) {
  using namespace pmg_mla;
  const int es = elem_bytes(dtype);
  if (es < 2) return PMG_ERR_DTYPE;
  if (num_reqs < 0 || total_q < 0 || total_k < 0 || heads < 0 || nope_dim < 1 || rope_dim < 0 || v_dim < 1 ||
      !(sm_scale >= 0.0f) || (options & ~(PMG_OPT_CAUSAL | PMG_OPT_FORCE_GENERAL)))
    return PMG_ERR_ARG;
  for (const int64_t s : {q_token_stride, q_head_stride, k_token_stride, k_head_stride, k_pe_stride, v_token_stride,
                          v_head_stride, out_token_stride, out_head_stride, prev_token_stride, prev_head_stride})
    if (!stride_ok(s)) return PMG_ERR_ARG;
  if (static_cast<int64_t>(nope_dim) + rope_dim > PMG_MAX_ENTRY || v_dim > PMG_MAX_ENTRY || total_q > INT32_MAX ||
      total_k > INT32_MAX || num_reqs > PMG_MAX_REQS || heads > (1 << 16))
    return PMG_ERR_UNSUPPORTED;
  if (num_reqs == 0 || total_q == 0 || heads == 0) return PMG_OK;
  if (q == nullptr || out == nullptr || cu_q == nullptr || cu_k == nullptr || workspace == nullptr ||
      (total_k > 0 && (k_nope == nullptr || v == nullptr || (k_pe == nullptr && rope_dim > 0))) ||
      (prev_out == nullptr) != (prev_lse == nullptr))
    return PMG_ERR_NULL;
  if (!aligned(q, es) || !aligned(k_nope, es) || !aligned(k_pe, es) || !aligned(v, es) || !aligned(out, es) ||
      !aligned(prev_out, es) || !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4) || !aligned(prev_lse, 4) ||
      !aligned(workspace, 16) || !aligned(error_flag, 4))
    return PMG_ERR_ALIGN;
  int sms = 0;
  int st = sm_count(&sms);
  if (st != PMG_OK) return st;
  if (workspace_bytes_given < workspace_bytes(sms)) return PMG_ERR_ARG;
  PrefillParams p{};
  p.q = q;
  p.qt_stride = q_token_stride;
  p.qh_stride = q_head_stride;
  p.k = k_nope;
  p.kt_stride = k_token_stride;
  p.kh_stride = k_head_stride;
  p.pe = k_pe;
  p.pe_stride = k_pe_stride;
  p.v = v;
  p.vt_stride = v_token_stride;
  p.vh_stride = v_head_stride;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.R = num_reqs;
  p.Tq = static_cast<int32_t>(total_q);
  p.Tk = static_cast<int32_t>(total_k);
  p.H = heads;
  p.dn = nope_dim;
  p.dr = rope_dim;
  p.dv = v_dim;
  p.sm_scale = sm_scale;
  p.out = out;
  p.ot_stride = out_token_stride;
  p.oh_stride = out_head_stride;
  p.lse = lse;
  p.prev = prev_out;
  p.pt_stride = prev_token_stride;
  p.ph_stride = prev_head_stride;
  p.prev_lse = prev_lse;
  p.ws = workspace_at(workspace, sms);
  p.err = error_flag;
  p.causal = (options & PMG_OPT_CAUSAL) ? 1 : 0;
  if (!(options & PMG_OPT_FORCE_GENERAL) && prefill_tc_takes(p, dtype)) return prefill_tc(p, dtype, sms, stream);
  const int E = p.dn + p.dr;
  const Kernel k = dtype == PMG_BF16 ? prefill_general_kernel<bf16>
                   : dtype == PMG_FP16 ? prefill_general_kernel<f16> : prefill_general_kernel<float>;
  st = allow_smem(reinterpret_cast<const void*>(k), general_smem(PMG_MAX_ENTRY));
  if (st != PMG_OK) return st;
  const int64_t most = (total_q / kGenRows + num_reqs) * heads;
  p.units = static_cast<int32_t>(std::min<int64_t>(most, 4 * sms));
  return launch(k, dim3(static_cast<unsigned>(p.units)), kGenThreads, general_smem(E), stream, p);
}
