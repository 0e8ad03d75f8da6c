// Parameters of the prefill kernels.
#pragma once

#include "mla_attn.cuh"

namespace pmg_mla {

struct PrefillParams {
  const void* q;
  int64_t qt_stride, qh_stride;
  const void* k;
  int64_t kt_stride, kh_stride;
  const void* pe;
  int64_t pe_stride;
  const void* v;
  int64_t vt_stride, vh_stride;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int32_t R;
  int32_t Tq, Tk;
  int32_t H;
  int32_t dn, dr, dv;
  float sm_scale;
  void* out;
  int64_t ot_stride, oh_stride;
  float* lse;
  const void* prev;
  int64_t pt_stride, ph_stride;
  const float* prev_lse;
  Workspace ws;
  int32_t* err;
  int32_t causal;
  int32_t units;
};

// Rows of request r: [q0, q0 + lq) and [k0, k0 + lk).
struct PrefillReq {
  int32_t q0, lq, k0, lk;
  int bad;
};

__device__ __forceinline__ int32_t clip_rows(int32_t x, int32_t total) { return max(0, min(x, total)); }

__device__ __forceinline__ PrefillReq prefill_req(const PrefillParams& p, int r) {
  const int32_t a = p.cu_q[r], b = p.cu_q[r + 1], c = p.cu_k[r], d = p.cu_k[r + 1];
  PrefillReq x;
  x.bad = (a < 0 || c < 0 || b < a || d < c) ? PMG_FLAG_CU_ORDER : 0;
  x.q0 = clip_rows(a, p.Tq);
  x.k0 = clip_rows(c, p.Tk);
  x.lq = max(0, clip_rows(b, p.Tq) - x.q0);
  x.lk = max(0, clip_rows(d, p.Tk) - x.k0);
  if (x.bad) x.lq = 0;
  return x;
}

// The shares of this call's and the previous state's rows: what each is
// multiplied by, and the joined log sum.
struct Joined {
  float now, before, lse;
};
__device__ __forceinline__ Joined join_state(float lse, float prev) {
  const float top = fmaxf(lse, prev);
  if (top == -INFINITY) return {0.0f, 0.0f, -INFINITY};
  const float a = lse == -INFINITY ? 0.0f : expf(lse - top), b = prev == -INFINITY ? 0.0f : expf(prev - top);
  const float sum = a + b;
  return {a / sum, b / sum, top + logf(sum)};
}

}  // namespace pmg_mla
