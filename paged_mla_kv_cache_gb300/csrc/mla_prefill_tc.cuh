// The tensor-core prefill kernel (mla_prefill_tc.cu).
#pragma once

#include "mla_prefill.cuh"

namespace pmg_mla {

// Whether it runs for these arguments.
bool prefill_tc_takes(const PrefillParams& p, int dtype);

// Launches it and the join of what its shares cut.
int prefill_tc(PrefillParams& p, int dtype, int sms, void* stream);

}  // namespace pmg_mla
