// RMS norm of every query and key head and the rotary embedding, in one pass over
// a projection's output, before verification:
//   y = x * rsqrt(mean(x^2) + eps) * w            (weights given)
//   (y_i, y_{i + D/2}) rotated by pos * base^(-2i/D)   (positions given)
// in fp32, rounded once at the end.
//
// One block per token.  D/16 lanes (rounded up to a power of two, LPR) hold a row: a
// lane has the 8 elements from 8c on of the first half and their partners of the
// second, so the rotation stays in the lane and the sum of squares takes log2(LPR)
// shuffles.  Rows are loaded kRows at a time, before the token's angles are known; what a
// token's rows share (cosines and sines, from shared memory, and the weights, from the
// first-level cache) is loaded again for each, which leaves registers for more blocks.
//
// Angles: base^(-2i/D) / 2 pi comes from the host as a 64-bit binary fraction; its
// product with the position modulo 2^64 is the phase modulo one turn, exact to 2^-34
// of a turn for any 32-bit position, without a 64-bit float on the device.
#include "va_common.cuh"
#include "va_quant.h"

namespace va {

constexpr int kNormThreads = 128;

template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&f)[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float *p, const float (&f)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

template <typename T, int LPR>
__global__ void __launch_bounds__(kNormThreads, sizeof(T) == 2 ? 9 : 7) norm_rope_kernel(const NormParams p) {
  constexpr int kPass = kNormThreads / LPR;      // rows of a pass
  constexpr int kRows = sizeof(T) == 2 ? 3 : 2;  // rows of a thread, loads first
  __shared__ __align__(16) float2 cs[128];       // cosine and sine of pair i
  const int tid = threadIdx.x, c = tid % LPR;
  const int half = p.D / 2, rows = p.Hq + p.Hkv;
  const bool act = 8 * c < half;
  const int b = blockIdx.x / p.T, t = blockIdx.x % p.T;
  const T *q = static_cast<const T *>(p.q.p) + (size_t)b * p.q.batch + (size_t)t * p.q.token + 8 * c;
  const T *k = static_cast<const T *>(p.k.p) + (size_t)b * p.k.batch + (size_t)t * p.k.token + 8 * c;
  T *qo = static_cast<T *>(const_cast<void *>(p.q_out.p)) + (size_t)b * p.q_out.batch + (size_t)t * p.q_out.token + 8 * c;
  T *ko = static_cast<T *>(const_cast<void *>(p.k_out.p)) + (size_t)b * p.k_out.batch + (size_t)t * p.k_out.token + 8 * c;

  Eight<T> lo[kRows], hi[kRows];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u * kPass;
      if (r >= rows || !act) continue;
      const T *x = r < p.Hq ? q + (size_t)r * p.D : k + (size_t)(r - p.Hq) * p.D;
      lo[u].load(x);
      hi[u].load(x + half);
    }
  };
  const int r_first = tid / LPR;
  load(r_first);
  if (p.positions != nullptr) {
    const int pos = __ldg(p.positions + blockIdx.x);
    for (int i = tid; i < half; i += kNormThreads) {
      // half turns in [-1, 1)
      const int turn = (int)(((uint64_t)(int64_t)pos * p.turns[i]) >> 32);
      float s, co;
      sincospif((float)turn * 0x1p-31f, &s, &co);
      cs[i] = make_float2(co, s);
    }
    __syncthreads();
  }
  const float inv_d = 1.f / (float)p.D;
  for (int r0 = r_first; r0 - r_first < rows; r0 += kRows * kPass) {
    if (r0 != r_first) load(r0);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u * kPass;
      const bool in = r < rows && act, is_q = r < p.Hq;
      const T *w = static_cast<const T *>(is_q ? p.q_weight : p.k_weight);
      float a[8], e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = e[j] = 0.f;
      if (in) {
        lo[u].get(a);
        hi[u].get(e);
      }
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], fmaf(e[j], e[j], ss));
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!in) continue;
      if (w != nullptr) {
        Eight<T> wl, wh;
        float fl[8], fh[8];
        wl.load(w + 8 * c);
        wh.load(w + 8 * c + half);
        wl.get(fl);
        wh.get(fh);
        const float rs = 1.f / sqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] = a[j] * rs * fl[j];
          e[j] = e[j] * rs * fh[j];
        }
      }
      if (p.positions != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float4 v = *reinterpret_cast<const float4 *>(cs + 8 * c + j);  // (cos, sin) of pairs j and j + 1
          const float a0 = a[j], a1 = a[j + 1];
          a[j] = fmaf(a0, v.x, -(e[j] * v.y));
          e[j] = fmaf(e[j], v.x, a0 * v.y);
          a[j + 1] = fmaf(a1, v.z, -(e[j + 1] * v.w));
          e[j + 1] = fmaf(e[j + 1], v.z, a1 * v.w);
        }
      }
      T *dst = is_q ? qo + (size_t)r * p.D : ko + (size_t)(r - p.Hq) * p.D;
      Eight<T>::store(dst, a);
      Eight<T>::store(dst + half, e);
    }
  }
}

namespace {
template <typename T>
cudaError_t launch_t(const NormParams &p, cudaStream_t stream) {
  const unsigned grid = (unsigned)((long long)p.B * p.T);
  const int lanes = p.D / 16;
  if (lanes <= 4)
    norm_rope_kernel<T, 4><<<grid, kNormThreads, 0, stream>>>(p);
  else if (lanes <= 8)
    norm_rope_kernel<T, 8><<<grid, kNormThreads, 0, stream>>>(p);
  else
    norm_rope_kernel<T, 16><<<grid, kNormThreads, 0, stream>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_norm_rope(const NormParams &p, cudaStream_t stream) {
  return p.fp32 ? launch_t<float>(p, stream) : launch_t<__nv_bfloat16>(p, stream);
}

}  // namespace va
