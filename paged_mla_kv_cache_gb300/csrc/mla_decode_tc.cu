// Absorbed latent attention on the tensor core: requests over their own entries
// (the kernel of mla_decode_tc_kernel.cuh).
#include "mla_decode_tc.cuh"
#include "mla_decode_tc_kernel.cuh"

namespace pmg_mla {

bool decode_tc_takes(const DecodeParams& p, int q_dtype, int cache_dtype) {
  const int ec = elem_bytes(cache_dtype);
  return p.dv == kLatent && p.dr == kRope && (q_dtype == PMG_BF16 || q_dtype == PMG_FP16) && p.B % 8 == 0 &&
         p.num_blocks > 0 && p.tok_stride > 0 && p.blk_stride > 0 && aligned(p.cache, 16) &&
         p.tok_stride * ec % 16 == 0 && p.blk_stride * ec % 16 == 0 && p.blk_stride * ec < (int64_t{1} << 40) &&
         p.tok_stride * ec < (int64_t{1} << 40) && aligned(p.q, 16) && p.qr_stride % 8 == 0 && p.qt_stride % 8 == 0 &&
         p.qh_stride % 8 == 0 && p.qr_stride < (int64_t{1} << 38) && p.qt_stride < (int64_t{1} << 38) &&
         p.qh_stride < (int64_t{1} << 38);
}

int decode_tc(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream) {
  const int rows = p.q_len * p.H;
  p.groups = (rows + 63) / 64;
  p.rows_per_group = (rows + p.groups - 1) / p.groups;
  p.groups = (rows + p.rows_per_group - 1) / p.rows_per_group;
  p.units = std::max(1, sms / p.groups);
  return launch_tc<false>(p, q_dtype, cache_dtype, stream);
}

}  // namespace pmg_mla
