// Accumulated attention weight: how much attention the accepted tokens of a
// step gave to every cached key, summed over the query heads of a kv-head and
// added to a running total.  The totals are the signal by which a cache is
// evicted (verify_build_index takes them as its score).
//
// After acceptance and commit, sequence b holds L_b + a keys and its accepted
// rows i < a (query rows path[i]) sit at positions L_b + i, a plain causal
// chain.  With the rows' log-sum-exp known from the verification call,
//   p(h, i, j) = exp(s(q[path[i]][h], k_j) - lse[h][path[i]]),  j <= L_b + i,
//   w[g][j]    = (j < L_b ? decay * w[g][j] : 0) + sum over h of g and i of p.
// No softmax pass and no V: K is read once, every total by one thread, in a
// fixed order (the result does not depend on the grid).
#include <cuda_bf16.h>
#include <math.h>

#include "va_common.cuh"
#include "va_mod.cuh"
#include "va_weight.h"

namespace va {

// Committed length and accepted tokens of sequence b; false (recorded once)
// when they do not fit the cache or the totals: that sequence is left alone.
__device__ __forceinline__ bool weight_seq(const WeightParams &p, int b, bool record, int &L, int &a) {
  L = __ldg(p.seqlens + b);
  a = p.n_accept != nullptr ? __ldg(p.n_accept + b) : p.T;
  const bool good = L >= 0 && a >= 0 && a <= p.T && L <= min(p.len_cap, p.stride) - a;
  if (!good && record) record_status(p.status, VA_ERR_DEVICE_BOUNDS);
  return good;
}

// Row of slot j of kv-head h (hidden slots may have any page entry: nullptr).
template <typename Tin>
__device__ __forceinline__ const Tin *weight_key(const WeightParams &p, int b, int h, int j, bool record) {
  size_t row;
  if (p.page_table != nullptr) {
    const int page = __ldg(p.page_table + (size_t)b * p.max_pages + (j >> p.page_shift));
    if (page < 0 || page >= p.num_pages) {
      if (record) record_status(p.status, VA_ERR_DEVICE_BOUNDS);
      return nullptr;
    }
    row = ((size_t)page << p.page_shift) + (size_t)(j & ((1 << p.page_shift) - 1));
  } else {
    row = (size_t)b * p.len_cap + j;
  }
  return static_cast<const Tin *>(p.k) + (row * p.Hkv + h) * p.D;
}

// One thread per key, its row in registers, query rows broadcast from shared
// memory.
template <typename Tin, int D>
__global__ void __launch_bounds__(128) weight_simt_kernel(const WeightParams p) {
  constexpr int RC = 16;  // query rows staged at once
  __shared__ float4 sq[RC][D / 4];
  __shared__ float slse[RC], sns[RC];
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  int L, a;
  if (!weight_seq(p, b, blockIdx.x == 0 && h == 0 && tid == 0, L, a)) return;
  const int j0 = blockIdx.x * 128;
  if (j0 >= L + a) return;
  const int j = j0 + tid;
  const int group = p.Hq / p.Hkv, R = group * a;
  // the first slot each accepted row sees rises with the row: row 0's decides
  // whether anything of this tile is seen
  const int lo = mod_first_slot(p.mod, b, 0, L);
  const bool live = j < L + a && j >= lo;
  float k[D];
  const Tin *kr = live ? weight_key<Tin>(p, b, h, j, true) : nullptr;
#pragma unroll
  for (int i = 0; i < D; ++i) k[i] = 0.f;
  if (kr != nullptr) {
#pragma unroll
    for (int i = 0; i < D; i += 4) {
      if constexpr (sizeof(Tin) == 4) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(kr + i));
        k[i] = v.x, k[i + 1] = v.y, k[i + 2] = v.z, k[i + 3] = v.w;
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(kr + i));
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v.x));
        const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v.y));
        k[i] = x.x, k[i + 1] = x.y, k[i + 2] = y.x, k[i + 3] = y.y;
      }
    }
  }
  float acc = 0.f;
  for (int r0 = 0; r0 < R; r0 += RC) {
    __syncthreads();
    for (int e = tid; e < RC * (D / 4); e += 128) {
      const int r = r0 + e / (D / 4), c = e % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < R) {
        const int i = r / group;
        const int t = p.path != nullptr ? __ldg(p.path + (size_t)b * p.T + i) : i;
        if (t >= 0 && t < p.T) {
          const Tin *qr = static_cast<const Tin *>(p.q) + (((size_t)b * p.T + t) * p.Hq + h * group + r % group) * D;
          if constexpr (sizeof(Tin) == 4) {
            v = __ldg(reinterpret_cast<const float4 *>(qr) + c);
          } else {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(qr) + c);
            const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
            const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
            v = make_float4(x.x, x.y, y.x, y.y);
          }
        }
      }
      sq[e / (D / 4)][c] = v;
    }
    if (tid < RC) {
      const int r = r0 + tid;
      float l = INFINITY, ns = 0.f;  // no such row: exp(s - inf) = 0
      if (r < R) {
        const int i = r / group, hq = h * group + r % group;
        const int t = p.path != nullptr ? __ldg(p.path + (size_t)b * p.T + i) : i;
        if (t >= 0 && t < p.T) {
          l = __ldg(p.lse + ((size_t)b * p.Hq + hq) * p.T + t);
          if (l == -INFINITY) l = INFINITY;  // a row that saw no key
          if (p.mod.slopes != nullptr) ns = -__ldg(p.mod.slopes + hq);
        } else if (blockIdx.x == 0) {
          record_status(p.status, VA_ERR_DEVICE_BOUNDS);
        }
      }
      slse[tid] = l;
      sns[tid] = ns;
    }
    __syncthreads();
    const int rn = min(RC, R - r0);
    for (int r = 0; r < rn; ++r) {
      const int i = (r0 + r) / group;
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < D / 4; ++c) {
        const float4 v = sq[r][c];
        s = fmaf(v.x, k[4 * c], s);
        s = fmaf(v.y, k[4 * c + 1], s);
        s = fmaf(v.z, k[4 * c + 2], s);
        s = fmaf(v.w, k[4 * c + 3], s);
      }
      // natural units: the difference s - lse is small where the weight matters
      const float d = (float)(L + i - j);
      const float x = mod_score(p.mod, s, sns[r], d) - slse[r];
      bool see = kr != nullptr && j <= L + i;
      if (p.mod.window > 0) see = see && (j >= L + i - p.mod.window + 1);
      acc += see ? ex2_approx(x * kModLog2e) : 0.f;
    }
  }
  if (j < L + a) {
    float *w = p.weight + ((size_t)b * p.Hkv + h) * p.stride + j;
    *w = j < L ? fmaf(p.decay, *w, acc) : acc;
  }
}

cudaError_t launch_accumulate_weight(const WeightParams &p, cudaStream_t stream) {
  const int keys = p.len_cap < p.stride ? p.len_cap : p.stride;
  const dim3 grid((unsigned)((keys + 127) / 128), (unsigned)p.Hkv, (unsigned)p.B);
  if (p.dtype == VA_DTYPE_FP32)
    weight_simt_kernel<float, 64><<<grid, 128, 0, stream>>>(p);
  else if (p.D == 64)
    weight_simt_kernel<__nv_bfloat16, 64><<<grid, 128, 0, stream>>>(p);
  else
    weight_simt_kernel<__nv_bfloat16, 128><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace va
