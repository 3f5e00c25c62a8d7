// Attention over caches held in e4m3, head size 128.
#include "va_attn_quant.cuh"

namespace va {

cudaError_t launch_attention_e4m3_d128(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                       cudaStream_t stream) {
  return launch_tq<VA_KV_E4M3, 128>(p, tmk, tmv, grid, stream);
}

}  // namespace va
