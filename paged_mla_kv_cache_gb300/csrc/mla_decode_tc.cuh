// The tensor-core decode kernel (mla_decode_tc_kernel.cuh) over requests
// (mla_decode_tc.cu) and over shared prefixes (mla_shared_tc.cu).
#pragma once

#include "mla_decode.cuh"

namespace pmg_mla {

// Whether it runs for these arguments.
bool decode_tc_takes(const DecodeParams& p, int q_dtype, int cache_dtype);

// Chooses groups and units, and launches it. The join follows as for the general kernel.
int decode_tc(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream);
int prefix_tc(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream);

// A prefix pass on pairs of SMs (mla_shared_pair.cu), where prefix_tc would do as well.
bool prefix_pair_takes(const DecodeParams& p, int q_dtype, int cache_dtype);
int prefix_pair(DecodeParams& p, int q_dtype, int cache_dtype, int sms, void* stream);

}  // namespace pmg_mla
