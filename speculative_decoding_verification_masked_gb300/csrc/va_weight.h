// Launcher of the accumulated attention weight (va_weight.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "va_kernels.h"

namespace va {

struct WeightParams {
  int B, T, Hq, Hkv, D;
  va_dtype dtype;
  const void *q, *k;
  int len_cap;                   // dense: max_cache_len; paged: max_pages * page_size
  const int32_t *page_table;     // NULL = dense
  int num_pages, page_shift, max_pages;
  const int32_t *seqlens;        // [B]
  const int32_t *path;           // [B][T] or NULL (node j = j)
  const int32_t *n_accept;       // [B] or NULL (T)
  const float *lse;              // [B][Hq][T]
  float decay;
  float *weight;                 // [B][Hkv][stride]
  int stride;
  int *status;                   // may be NULL
  ModParams mod;                 // in natural units; out_mul holds the scale also when off
  int tma_box;                   // bf16: rows of one TMA box of the cache; 0 = gathered
  int row0;                      // first packed row of this pass
  uint64_t wait_ns;
  int test_stall;                // test hook: as in AttnParams
};

cudaError_t launch_accumulate_weight(const WeightParams &p, const CUtensorMap &tmk, int sms, cudaStream_t stream);

}  // namespace va
