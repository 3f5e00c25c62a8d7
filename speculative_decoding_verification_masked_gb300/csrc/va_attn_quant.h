// Launcher of the attention over caches held in 8 or 4 bits (va_attn_quant.cuh; one
// translation unit per format and head size, so that they compile side by side).
#pragma once

#include "va_kernels.h"

namespace va {

// Rows of a block of packed query rows.  Blocks of 128 make halves of a tile once for twice
// the rows; their Q and P leave room for two stages of 4-bit rows, not of 8-bit ones, and
// d 64 stays within the workspace of its shape.
constexpr int quant_block_rows(int R, int format, int D) {
  return R <= 16 ? 16 : R <= 32 ? 32 : R > 64 && format == VA_KV_E2M1 && D == 128 ? 128 : 64;
}

cudaError_t launch_attention_e4m3_d128(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                       cudaStream_t stream);
cudaError_t launch_attention_e4m3_d64(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                      cudaStream_t stream);
cudaError_t launch_attention_e2m1_d128(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                       cudaStream_t stream);
cudaError_t launch_attention_e2m1_d64(AttnParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid,
                                      cudaStream_t stream);

}  // namespace va
