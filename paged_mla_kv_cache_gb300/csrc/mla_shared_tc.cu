// Absorbed latent attention on the tensor core: groups of requests over their
// prefixes (the kernel of mla_decode_tc_kernel.cuh, as a prefix pass).
#include "mla_decode_tc.cuh"
#include "mla_decode_tc_kernel.cuh"

namespace pmg_mla {

int prefix_tc(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream) {
  const int64_t rows = static_cast<int64_t>(p.reqs) * p.q_len * p.H;
  p.groups = 1;
  p.units = sms;
  // Small calls, where one wave holds every tile of keys of every 16 or 32 rows: their CTAs take less time than one of 64 rows
  // (4 requests of 16 heads behind 513 entries: 20.1 us for all passes instead of 22.3). The host knows neither the lengths
  // nor the groups' sizes: it counts as many tiles as a row of the table has room for, and every row in every group, so calls
  // with a wider table or with several groups may take the larger tiles.
  const int64_t tiles = std::min<int64_t>((p.bt_stride * p.B + kDecodeTile - 1) / kDecodeTile, sms) * p.R;
  for (const int n : {16, 32})
    if ((rows + n - 1) / n * tiles <= sms) {
      p.rows_per_group = static_cast<int32_t>(std::min<int64_t>(rows, p.H <= n ? n / p.H * p.H : n));
      return launch_tc<true>(p, q_dtype, cache_dtype, stream);
    }
  if (sms >= 2 && prefix_pair_takes(p, q_dtype, cache_dtype)) return prefix_pair(p, q_dtype, cache_dtype, sms, stream);
  // whole tokens in a row tile, where that leaves at most an eighth of it empty: its queries are then one box of the copy
  // engine (an e4m3 cache's are converted by the softmax warps anyhow)
  const int whole = p.H <= 64 ? 64 / p.H * p.H : 64;
  const int tile = cache_dtype != PMG_FP8_E4M3 && whole >= 56 ? whole : 64;
  p.rows_per_group = static_cast<int32_t>(std::min<int64_t>(rows, tile));
  return launch_tc<true>(p, q_dtype, cache_dtype, stream);
}

}  // namespace pmg_mla
