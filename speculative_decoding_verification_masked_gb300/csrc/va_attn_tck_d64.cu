// The keys-on-lanes attention kernel (va_attn_tck.cuh): score shaping, d64.
#include "va_attn_tck.cuh"

namespace va {

cudaError_t launch_attention_tck_d64(const AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                     cudaStream_t stream) {
  return p.mod.on == 1 ? launch_tck<64, false, 1>(p, tmk, tmv, grid, stream)
                       : launch_tck<64, false, 2>(p, tmk, tmv, grid, stream);
}

}  // namespace va
