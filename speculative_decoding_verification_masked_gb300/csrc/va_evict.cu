// Eviction: the cache rows of a keep set are moved to the front of every
// (sequence, kv-head), in place, with the accumulated weight of each row.
//
// indices[b][h][0..n) is strictly increasing, so row j comes from a slot
// idx[j] >= j: whoever reads a slot that row j is written to has a number
// <= j.  The rows of a (sequence, kv-head) are cut into chunks; a block reads a
// whole chunk of K, V and weights into shared memory, announces that, waits
// until every lower chunk of the same kv-head has been read too, and only then
// writes.  So all chunks of all kv-heads are read at once, every byte is read
// and written once, and nothing needs a second copy of the cache.
//
// The blocks are all resident (cooperative launch) and take the chunks in
// ascending order, so the lowest unfinished chunk never waits for one that is
// not running; the wait is bounded all the same.  "Read" is one bit a chunk in
// the caller's scratch, 32 chunks a word; the last block to leave clears the
// words it was given.  Where a wait has run out some chunks are not written, and the
// last block takes the new lengths back: no sequence is reported as cut.
//
// Bound by HBM: 2 x 2 x row bytes a kept row (K and V, read and written).
// Chunks of 32 KB and up to six blocks an SM keep 190 KB an SM in flight: 16
// sequences cut to 8192 rows of 8 kv-heads (1.09 GB) take 199 us, 5.5 TB/s, 82%
// of the measured copy rate.  Chunks of half that size took 207 to 218 us, blocks
// of twice the threads 244 us; divisions in the copy loops had cost 268 us.
#include <mutex>

#include "va_common.cuh"
#include "va_evict.h"
#include "va_kernels.h"

namespace va {

constexpr int kEvictThreads = 256;
constexpr int kEvictChunkBytes = 16384;  // of K, and as much of V
constexpr int kEvictMaxRows = 128;

__host__ __device__ inline int evict_rows(int row_bytes) {
  const int r = kEvictChunkBytes / row_bytes;
  return r < kEvictMaxRows ? r : kEvictMaxRows;
}

// scratch: [0] blocks done, [1] a wait ran out; from 256: read bits, the words
// of (sequence, kv-head) bh at bh * words
struct EvictScratchView {
  unsigned *done, *bits;
  int *gave_up;
};
__device__ __forceinline__ EvictScratchView evict_scratch(const EvictParams &p) {
  unsigned *s = static_cast<unsigned *>(p.scratch);
  return {s, s + 64, reinterpret_cast<int *>(s) + 1};
}

__device__ __forceinline__ unsigned ld_acquire_u32(const unsigned *ptr) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ptr) : "memory");
  return v;
}
__device__ __forceinline__ void red_release_or(unsigned *ptr, unsigned v) {
  asm volatile("red.release.gpu.global.or.b32 [%0], %1;" ::"l"(ptr), "r"(v) : "memory");
}

// Kept rows of sequence b (the whole warp); -1 when the call leaves it alone:
// a length or count out of range, or kv-heads that keep different numbers.
__device__ __forceinline__ int evict_count(const EvictParams &p, int b, int L) {
  const int n = __ldg(p.n_indices + (size_t)b * p.Hkv);
  bool good = L >= 0 && L <= p.len_cap && n >= 0 && n <= min(L, p.max_indices);
  if (p.weight != nullptr) good = good && L <= p.stride;
  for (int g = threadIdx.x & 31; g < p.Hkv; g += 32) good = good && n == __ldg(p.n_indices + (size_t)b * p.Hkv + g);
  return __all_sync(0xffffffffu, good) ? n : -1;
}

// Cache row (of Hkv heads) of a logical slot; -1 (recorded) for a page entry out of range.
__device__ __forceinline__ long long evict_row(const EvictParams &p, int b, int slot) {
  if (p.page_table == nullptr) return (long long)b * p.len_cap + slot;
  const int page = __ldg(p.page_table + (size_t)b * p.max_pages + (slot >> p.page_shift));
  if (page < 0 || page >= p.num_pages) {
    record_status(p.status, VA_ERR_DEVICE_BOUNDS);
    return -1;
  }
  return ((long long)page << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
}

__global__ void __launch_bounds__(kEvictThreads) evict_kv_kernel(const EvictParams p, int rows, int words, long long items) {
  extern __shared__ __align__(16) uint8_t smem[];  // K rows, V rows
  __shared__ long long src[kEvictMaxRows], dst[kEvictMaxRows];  // byte offsets in the caches; src -1: not moved
  __shared__ float sw[kEvictMaxRows];
  __shared__ int s_L, s_n, s_go;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = p.B * p.Hkv;
  // a thread keeps one 16-byte column and steps over the rows (threads past the
  // last whole row of columns have none)
  const int cpr = p.row_bytes / 16;
  const int rstep = kEvictThreads / cpr;
  const int r0 = tid / cpr < rstep ? tid / cpr : rows;
  const int col = (tid % cpr) * 16;
  const EvictScratchView sc = evict_scratch(p);
  uint8_t *kbuf = smem + col, *vbuf = smem + rows * p.row_bytes + col;
  uint8_t *kc = static_cast<uint8_t *>(p.k) + col, *vc = static_cast<uint8_t *>(p.v) + col;

  // this thread's index of an item, loaded one item ahead
  auto index_of = [&](long long it) {
    const int j = (int)(it / heads) * rows + tid;
    return it < items && tid < rows && j < p.max_indices ? __ldg(p.indices + (size_t)(it % heads) * p.max_indices + j) : -1;
  };
  int s_next = index_of(blockIdx.x);
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int c = (int)(it / heads), bh = (int)(it % heads);
    const int b = bh / p.Hkv, h = bh % p.Hkv;
    const int j0 = c * rows;
    int s = s_next;
    s_next = index_of(it + gridDim.x);
    if (warp == 0) {
      const int L = __ldg(p.seqlens + b);
      const int n = evict_count(p, b, L);
      if (lane == 0) {
        s_L = L;
        s_n = n;
        if (h == 0 && c == 0) {
          p.seqlens_out[b] = n < 0 ? L : n;
          if (n < 0) record_status(p.status, VA_ERR_DEVICE_BOUNDS);
        }
      }
    }
    __syncthreads();
    const int nr = min(rows, s_n - j0);  // rows of this chunk
    if (nr <= 0) {
      __syncthreads();  // s_n is read before the next item overwrites it
      continue;
    }
    float *w = p.weight != nullptr ? p.weight + (size_t)bh * p.stride : nullptr;
    if (tid < nr) {
      const int j = j0 + tid;
      if (s < j || s >= s_L) {
        record_status(p.status, VA_ERR_DEVICE_BOUNDS);
        s = j;
      }
      const long long d = s != j ? evict_row(p, b, j) : -1, f = d >= 0 ? evict_row(p, b, s) : -1;
      src[tid] = f >= 0 ? (f * p.Hkv + h) * p.row_bytes : -1;
      dst[tid] = (d * p.Hkv + h) * p.row_bytes;
      if (w != nullptr) sw[tid] = w[s];
    }
    __syncthreads();
#pragma unroll 4
    for (int r = r0; r < nr; r += rstep) {
      const long long o = src[r];
      if (o < 0) continue;
      cp_async_16(kbuf + r * p.row_bytes, kc + o, 16);
      cp_async_16(vbuf + r * p.row_bytes, vc + o, 16);
    }
    cp_async_wait_all();
    __syncthreads();
    // announce, then wait for the lower chunks of this kv-head
    if (warp == 0) {
      unsigned *bits = sc.bits + (size_t)bh * words;
      if (lane == 0 && (int)blockIdx.x != p.test_drop) red_release_or(bits + (c >> 5), 1u << (c & 31));
      bool all = true;
      for (int g = lane; g <= c >> 5; g += 32) {
        const unsigned need = g < (c >> 5) ? ~0u : (1u << (c & 31)) - 1u;
        if ((ld_acquire_u32(bits + g) & need) == need) continue;
        const uint64_t t0 = globaltimer_ns();
        while ((ld_acquire_u32(bits + g) & need) != need) {
          if (globaltimer_ns() - t0 > p.wait_ns || *reinterpret_cast<volatile int *>(sc.gave_up) != 0) {
            record_status(p.status, VA_ERR_TIMEOUT);
            atomicExch(sc.gave_up, 1);
            all = false;
            break;
          }
        }
        if (!all) break;
      }
      const bool go = __all_sync(0xffffffffu, all);
      if (lane == 0) s_go = go ? 1 : 0;
    }
    __syncthreads();
    if (s_go) {
#pragma unroll 4
      for (int r = r0; r < nr; r += rstep) {
        if (src[r] < 0) continue;
        const long long o = dst[r];
        *reinterpret_cast<uint4 *>(kc + o) = *reinterpret_cast<const uint4 *>(kbuf + r * p.row_bytes);
        *reinterpret_cast<uint4 *>(vc + o) = *reinterpret_cast<const uint4 *>(vbuf + r * p.row_bytes);
      }
      if (w != nullptr && tid < nr) w[j0 + tid] = sw[tid];
    }
    __syncthreads();
  }
  // the last block out clears the bits for the next call, and takes the lengths back
  // if a wait ran out (every block's are written by its thread 0, before this count)
  if (tid == 0) {
    __threadfence();
    s_go = atomicAdd(sc.done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (s_go) {
    __threadfence();
    if (*reinterpret_cast<volatile int *>(sc.gave_up) != 0)
      for (int b = tid; b < p.B; b += kEvictThreads) p.seqlens_out[b] = __ldg(p.seqlens + b);
    __syncthreads();
    const size_t total = (size_t)heads * words;
    for (size_t i = tid; i < total; i += kEvictThreads) sc.bits[i] = 0u;
    if (tid == 0) {
      *sc.done = 0u;
      *sc.gave_up = 0;
    }
  }
}

static int evict_words(int max_indices, int rows) { return ((max_indices + rows - 1) / rows + 31) / 32; }

size_t evict_scratch_bytes(int B, int Hkv, int max_indices) {
  // the shortest chunks (rows of 1 KB) need the most words
  return 256 + align256(sizeof(unsigned) * (size_t)B * Hkv * evict_words(max_indices, evict_rows(1024)));
}

cudaError_t launch_evict_kv(const EvictParams &p, int sms, cudaStream_t stream) {
  const int rows = evict_rows(p.row_bytes);
  const int words = evict_words(p.max_indices, rows);
  const size_t smem = 2 * (size_t)rows * p.row_bytes;
  const long long items = (long long)p.B * p.Hkv * ((p.max_indices + rows - 1) / rows);
  int dev = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {  // blocks that fit an SM with this much shared memory, asked for once
    static std::mutex mu;
    static int cache[64][kEvictChunkBytes / 16 + 1];
    std::lock_guard<std::mutex> lock(mu);
    int &n = cache[dev & 63][smem / 32];
    if (n == 0) {
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, evict_kv_kernel, kEvictThreads, smem);
      if (e != cudaSuccess) return e;
    }
    per_sm = n;
  }
  const long long most = (long long)sms * (per_sm < 1 ? 1 : per_sm);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < most ? items : most));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kv_kernel, p, rows, words, items);
}

}  // namespace va
