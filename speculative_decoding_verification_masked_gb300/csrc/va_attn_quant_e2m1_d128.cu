// Attention over caches held in e2m1, head size 128.
#include "va_attn_quant.cuh"

namespace va {

cudaError_t launch_attention_e2m1_d128(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                       cudaStream_t stream) {
  return launch_tq<VA_KV_E2M1, 128>(p, tmk, tmv, grid, stream);
}

}  // namespace va
