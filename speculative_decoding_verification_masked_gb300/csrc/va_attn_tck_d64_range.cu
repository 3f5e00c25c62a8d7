// The keys-on-lanes attention kernel (va_attn_tck.cuh) with score shaping: d64,
// a window or document start.
#include "va_attn_tck.cuh"

namespace va {

cudaError_t launch_attention_tck_d64_range(const AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                           cudaStream_t stream) {
  return launch_tck<64, false, 1>(p, tmk, tmv, grid, stream);
}

}  // namespace va
