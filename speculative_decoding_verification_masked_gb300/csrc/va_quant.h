// Launchers of the per-head norm with rotation (va_norm.cu) and of writing and
// reading caches held in 8 or 4 bits (va_quant.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "verify_attn.h"

namespace va {

// Rows of a [B][T][heads][D] tensor whose heads are contiguous: base pointer and
// strides in elements.
struct TokenRows {
  const void *p;
  long long batch, token;
};

struct NormParams {
  int B, T, Hq, Hkv, D;
  int fp32;                       // element type: 1 = fp32, 0 = bf16
  TokenRows q, k, q_out, k_out;   // (outputs are written)
  const void *q_weight, *k_weight;// [D] or nullptr: no norm
  float eps;
  const int32_t *positions;       // [B][T] or nullptr: no rotation
  // base^(-2i/D) in turns (divided by 2 pi, modulo 1) as a 64-bit binary fraction
  uint64_t turns[128];
};

cudaError_t launch_norm_rope(const NormParams &p, cudaStream_t stream);

struct QuantParams {
  int B, T, Hkv, D;
  int fp32;                       // element type of the plain rows
  int format;                     // va_kv_format
  TokenRows k, v;                 // plain rows (read, or written when reading back)
  void *k_cache, *v_cache;        // quantised rows: dense [B][len_cap][Hkv] or pages [P][page][Hkv]
  int len_cap;                    // dense: max_cache_len; paged: max_pages * page size
  const int32_t *page_table;      // nullptr for the dense cache
  int page_shift, max_pages, num_pages;
  const int32_t *start;           // [B] first slot
  const int32_t *n_tokens;        // [B] or nullptr: T
  int *status;                    // may be nullptr
  int pass_tokens, pass_heads;    // rows of a block's pass, as whole tokens and heads (set by the launcher)
};

cudaError_t launch_quantize_kv(const QuantParams &p, cudaStream_t stream);
cudaError_t launch_dequantize_kv(const QuantParams &p, cudaStream_t stream);

}  // namespace va
