// Launcher of the attention over caches held in 8 or 4 bits (va_attn_quant.cuh; one
// translation unit per format and head size, so that they compile side by side).
#pragma once

#include "va_kernels.h"

namespace va {

// Rows of a block of packed query rows.
inline int quant_block_rows(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : 64; }

cudaError_t launch_attention_e4m3_d128(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                       cudaStream_t stream);
cudaError_t launch_attention_e4m3_d64(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                      cudaStream_t stream);
cudaError_t launch_attention_e2m1_d128(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                       cudaStream_t stream);
cudaError_t launch_attention_e2m1_d64(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                      cudaStream_t stream);

}  // namespace va
