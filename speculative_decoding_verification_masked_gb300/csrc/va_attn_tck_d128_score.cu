// The keys-on-lanes attention kernel (va_attn_tck.cuh) with score shaping: d128,
// a cap or slopes.
#include "va_attn_tck.cuh"

namespace va {

cudaError_t launch_attention_tck_d128_score(const AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                            cudaStream_t stream) {
  return launch_tck<128, false, 2>(p, tmk, tmv, grid, stream);
}

}  // namespace va
