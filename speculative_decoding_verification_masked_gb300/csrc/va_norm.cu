// RMS norm of every query and key head and the rotary embedding, in one pass over
// a projection's output, before verification:
//   y = x * rsqrt(mean(x^2) + eps) * w            (weights given)
//   (y_i, y_{i + D/2}) rotated by pos * base^(-2i/D)   (positions given)
// in fp32, rounded once at the end.
//
// One block per token.  D/16 lanes (rounded up to a power of two, LPR) hold a row: a
// lane has the 8 elements from 8c on of the first half and their partners of the
// second, so the rotation stays in the lane and the sum of squares takes log2(LPR)
// shuffles.  Weights and angles are folded into four factors a pair, once per token
// and kind of head, in shared memory (an element's weight times the cosine or sine
// that it meets), so a row costs packed products alone: a 16K-token prompt was bound by
// its instructions, not by HBM, and went from 94 to 63 us (5.4 TB/s, 79% of the measured copy
// rate; weights and angles of a pair apart, in registers, before).  Rows are loaded kRows at a time, before the factors are known.
// (Eight blocks an SM leave 64 registers a thread: 8 bytes of spills, 0.3% of the instructions.)
// fp32 rows are bound by HBM: 16384 tokens in 99.7 us, 99% of the copy rate.
//
// Angles: base^(-2i/D) / 2 pi comes from the host as a binary fraction, good to 2^-55 (a
// double; base >= 1), in 64 bits; its product with the position modulo 2^64 is the phase
// modulo one turn, off by |position| 2^-55 for any 32-bit position, without a 64-bit float on
// the device.  The phase is cut to 32 bits (2^-32 of a turn) and rounded to fp32 (2^-26).
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

template <typename T>
__device__ __forceinline__ float weight_at(const void *w, int i) {
  if (w == nullptr) return 1.f;
  if constexpr (sizeof(T) == 2)
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[i]);
  else
    return static_cast<const float *>(w)[i];
}

template <typename T, int LPR>
__global__ void __launch_bounds__(kNormThreads, 8) norm_rope_kernel(const NormParams p) {
  constexpr int kPass = kNormThreads / LPR;      // rows of a pass
  constexpr int kRows = sizeof(T) == 2 ? 3 : 1;  // rows of a thread, loads first
  // [query, key heads][0: (first half by cosine, second half by sine, negated) of two pairs, 1: (second
  // half by cosine, first half by sine)][pair of pairs of a lane][lane]: neighbouring lanes read
  // neighbouring vectors
  __shared__ float4 fac[2][2][4][16];
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
  {
    const int pos = p.positions != nullptr ? __ldg(p.positions + blockIdx.x) : 0;
    for (int i = tid; i < half; i += kNormThreads) {
      float s = 0.f, co = 1.f;
      if (p.positions != nullptr) {
        // half turns in [-1, 1)
        const int turn = (int)(((uint64_t)(int64_t)pos * p.turns[i]) >> 32);
        sincospif((float)turn * 0x1p-31f, &s, &co);
      }
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        const void *w = kind == 0 ? p.q_weight : p.k_weight;
        const float wl = weight_at<T>(w, i), wh = weight_at<T>(w, i + half);
        float *f = reinterpret_cast<float *>(&fac[kind][0][i % 8 / 2][i / 8]) + (i & 1);
        float *g = reinterpret_cast<float *>(&fac[kind][1][i % 8 / 2][i / 8]) + (i & 1);
        f[0] = wl * co;
        f[2] = -(wh * s);
        g[0] = wh * co;
        g[2] = wl * s;
      }
    }
    __syncthreads();
  }
  const float inv_d = 1.f / (float)p.D;
  const bool turned = p.positions != nullptr;
  for (int r0 = r_first; r0 - r_first < rows; r0 += kRows * kPass) {
    if (r0 != r_first) load(r0);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u * kPass;
      const bool in = r < rows && act, is_q = r < p.Hq;
      float2 a[4], e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = e[j] = make_float2(0.f, 0.f);
      if (in) {
        lo[u].get(reinterpret_cast<float(&)[8]>(a));
        hi[u].get(reinterpret_cast<float(&)[8]>(e));
      }
      float2 ss2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) ss2 = fma2(a[j], a[j], fma2(e[j], e[j], ss2));
      float ss = ss2.x + ss2.y;
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!in) continue;
      if ((is_q ? p.q_weight : p.k_weight) != nullptr) {
        // one Newton step: the approximate root alone is off by two units
        const float v = fmaf(ss, inv_d, p.eps), y = rsqrtf(v);
        const float rs = fmaf(fmaf(-(v * y), y, 1.f), 0.5f * y, y);
        const float2 rs2 = v > 0x1p-100f && v < 0x1p100f ? make_float2(rs, rs) : make_float2(1.f / sqrtf(v), 1.f / sqrtf(v));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a[j] = mul2(a[j], rs2);
          e[j] = mul2(e[j], rs2);
        }
      }
      const int kind = is_q ? 0 : 1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 u0 = fac[kind][0][j][c], u1 = fac[kind][1][j][c];
        float2 x = mul2(a[j], make_float2(u0.x, u0.y)), y = mul2(e[j], make_float2(u1.x, u1.y));
        if (turned) {  // (without, an infinity stays out of its partner)
          x = fma2(e[j], make_float2(u0.z, u0.w), x);
          y = fma2(a[j], make_float2(u1.z, u1.w), y);
        }
        a[j] = x;
        e[j] = y;
      }
      T *dst = is_q ? qo + (size_t)r * p.D : ko + (size_t)(r - p.Hq) * p.D;
      Eight<T>::store(dst, reinterpret_cast<const float(&)[8]>(a));
      Eight<T>::store(dst + half, reinterpret_cast<const float(&)[8]>(e));
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
