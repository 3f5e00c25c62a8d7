// Eviction: the cache rows of a keep set are moved to the front of every
// (sequence, kv-head), in place, with the accumulated weight of each row.
//
// indices[b][h][0..n) is strictly increasing, so row j comes from a slot
// idx[j] >= j: moving the rows in order of j never overwrites one that is
// still to be read.  One thread owns one 16-byte column of one (sequence,
// kv-head) of K or V and moves it batch by batch, each batch read before it
// is written.
#include "va_common.cuh"
#include "va_evict.h"
#include "va_kernels.h"

namespace va {

// Kept rows of (b, h); -1 (recorded) when the call leaves the sequence alone.
__device__ __forceinline__ int evict_count(const EvictParams &p, int b, int h, bool record) {
  const int L = __ldg(p.seqlens + b);
  const int n = __ldg(p.n_indices + (size_t)b * p.Hkv + h);
  bool good = L >= 0 && L <= p.len_cap && n >= 0 && n <= min(L, p.max_indices);
  // one new length per sequence: every kv-head keeps the same number of rows
  for (int g = 0; g < p.Hkv; ++g) good = good && n == __ldg(p.n_indices + (size_t)b * p.Hkv + g);
  if (good && p.weight != nullptr) good = L <= p.stride;
  if (!good && record) record_status(p.status, VA_ERR_DEVICE_BOUNDS);
  return good ? n : -1;
}

// Address of (sequence b, logical slot, kv-head h); nullptr (recorded) for a
// page entry out of range.
__device__ __forceinline__ uint8_t *evict_row(const EvictParams &p, uint8_t *base, int b, int slot, int h) {
  size_t row;
  if (p.page_table != nullptr) {
    const int page = __ldg(p.page_table + (size_t)b * p.max_pages + (slot >> p.page_shift));
    if (page < 0 || page >= p.num_pages) {
      record_status(p.status, VA_ERR_DEVICE_BOUNDS);
      return nullptr;
    }
    row = ((size_t)page << p.page_shift) + (size_t)(slot & ((1 << p.page_shift) - 1));
  } else {
    row = (size_t)b * p.len_cap + slot;
  }
  return base + (row * p.Hkv + h) * (size_t)p.row_bytes;
}

__global__ void __launch_bounds__(64) evict_kv_kernel(const EvictParams p) {
  const int b = blockIdx.x, h = blockIdx.y;
  const int chunks = p.row_bytes / 16;
  const int tid = threadIdx.x;
  const int n = evict_count(p, b, h, tid == 0);
  if (n < 0) {
    if (h == 0 && blockIdx.z == 0 && tid == 0) p.seqlens_out[b] = __ldg(p.seqlens + b);
    return;
  }
  const int L = __ldg(p.seqlens + b);
  const int32_t *idx = p.indices + ((size_t)b * p.Hkv + h) * p.max_indices;
  uint8_t *base = static_cast<uint8_t *>(blockIdx.z == 0 ? p.k : p.v);
  constexpr int U = 8;
  auto source = [&](int j) {
    const int s = __ldg(idx + j);
    if (s < j || s >= L) {
      record_status(p.status, VA_ERR_DEVICE_BOUNDS);
      return j;
    }
    return s;
  };
  for (int c = tid; c < chunks; c += 64) {
    for (int j0 = 0; j0 < n; j0 += U) {
      uint4 v[U];
      bool got[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        got[u] = false;
        if (j0 + u < n) {
          const int s = source(j0 + u);
          const uint8_t *r = s != j0 + u ? evict_row(p, base, b, s, h) : nullptr;
          got[u] = r != nullptr;
          if (got[u]) v[u] = *reinterpret_cast<const uint4 *>(r + 16 * c);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!got[u]) continue;
        uint8_t *r = evict_row(p, base, b, j0 + u, h);
        if (r != nullptr) *reinterpret_cast<uint4 *>(r + 16 * c) = v[u];
      }
    }
  }
  if (blockIdx.z == 0 && tid == 0) {
    if (p.weight != nullptr) {
      float *w = p.weight + ((size_t)b * p.Hkv + h) * p.stride;
      for (int j = 0; j < n; ++j) w[j] = w[source(j)];
    }
    if (h == 0) p.seqlens_out[b] = n;
  }
}

size_t evict_scratch_bytes(int B, int Hkv, int max_indices) {
  (void)B, (void)Hkv, (void)max_indices;
  return 256;
}

cudaError_t launch_evict_kv(const EvictParams &p, cudaStream_t stream) {
  evict_kv_kernel<<<dim3((unsigned)p.B, (unsigned)p.Hkv, 2), 64, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace va
