// The keys-on-lanes attention kernel (va_attn_tck.cuh): the instances without
// score shaping, and the choice between all of them.
#include "va_attn_tck.cuh"

namespace va {

cudaError_t launch_attention_tck_d128_range(const AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                            cudaStream_t stream);
cudaError_t launch_attention_tck_d128_score(const AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                            cudaStream_t stream);
cudaError_t launch_attention_tck_d64_range(const AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                           cudaStream_t stream);
cudaError_t launch_attention_tck_d64_score(const AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                           cudaStream_t stream);

size_t attn_tck_smem_required(const AttnParams &p) {
  if (p.D == 64)
    return p.rows_pad <= 16   ? tck_smem_bytes<64, 16>(p)
           : p.rows_pad <= 32 ? tck_smem_bytes<64, 32>(p)
                              : tck_smem_bytes<64, 64>(p);
  return p.rows_pad <= 16   ? tck_smem_bytes<128, 16>(p)
         : p.rows_pad <= 32 ? tck_smem_bytes<128, 32>(p)
                            : tck_smem_bytes<128, 64>(p);
}

cudaError_t launch_attention_tck(const AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                 cudaStream_t stream) {
  if (p.mod.on != 0) {
    auto launch = p.D == 64 ? (p.mod.on == 1 ? launch_attention_tck_d64_range : launch_attention_tck_d64_score)
                            : (p.mod.on == 1 ? launch_attention_tck_d128_range : launch_attention_tck_d128_score);
    return launch(p, tmk, tmv, grid, stream);
  }
  return p.positions != nullptr ? launch_tck<128, true, 0>(p, tmk, tmv, grid, stream)
                                : launch_tck<128, false, 0>(p, tmk, tmv, grid, stream);
}

}  // namespace va
