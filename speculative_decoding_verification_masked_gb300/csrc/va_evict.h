// Launcher of the in-place eviction (va_evict.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace va {

struct EvictParams {
  int B, Hkv;
  int row_bytes;                 // bytes of one (token, kv-head) row, a multiple of 16
  void *k, *v;
  int len_cap;                   // dense: max_cache_len; paged: max_pages * page_size
  const int32_t *page_table;     // NULL = dense
  int num_pages, page_shift, max_pages;
  const int32_t *seqlens;        // [B]
  const int32_t *indices;        // [B][Hkv][max_indices]
  const int32_t *n_indices;      // [B][Hkv]
  int max_indices;
  float *weight;                 // [B][Hkv][stride] or NULL
  int stride;
  int32_t *seqlens_out;          // [B]
  void *scratch;                 // evict_scratch_bytes, zero between calls
  int *status;                   // may be NULL
  uint64_t wait_ns;
  int test_drop;                 // test hook: this block announces nothing (-1: off)
};

size_t evict_scratch_bytes(int B, int Hkv, int max_indices);

cudaError_t launch_evict_kv(const EvictParams &p, int sms, cudaStream_t stream);

}  // namespace va
