// Writing rows of K and V into a cache held in 8 or 4 bits, and reading a range
// of slots back (layout and formats: va_quant.cuh).
//
// Both are one pass over the data.  D/16 neighbouring lanes hold a row, 16
// elements (one group of the 4-bit format) each; a row's largest magnitude comes
// from log2(D/16) shuffles, and the first lane writes the row's 16-byte tail.
// A row of 128 bf16 values moves 256 + 144 (80) bytes, and a thread has kRows rows' loads
// in flight.  64K tokens of 8 heads, in us (floor at the measured copy rate): read from 4 bits
// 66 (51), from 8 bits 66 (60), bound by HBM; written in 8 bits 61 (60), in 4 bits 73 (51), which
// issues 82% of all slots (about nine instructions an element, the quotient's exact rounding
// three of them).  A chunk of 11K tokens is one wave of short blocks: 17.8 us to 4 bits from cold
// caches (8.6), with the loads' latency as the largest stall and 68% of the slots issued.
#include "va_common.cuh"
#include "va_quant.cuh"
#include "va_quant.h"

namespace va {

constexpr int kQuantThreads = 128;

// Row (sequence b, logical slot, kv-head h) of a cache; nullptr when a page entry
// is out of range (recorded).
__device__ __forceinline__ uint8_t *quant_row(const QuantParams &p, void *cache, int row_bytes, int b, int slot,
                                              int h) {
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
  return static_cast<uint8_t *>(cache) + (row * p.Hkv + h) * (size_t)row_bytes;
}

// First slot and number of rows of sequence b (0 rows, recorded, when they do not fit).
__device__ __forceinline__ void quant_range(const QuantParams &p, int b, int &start, int &n) {
  start = __ldg(p.start + b);
  n = p.n_tokens != nullptr ? __ldg(p.n_tokens + b) : p.T;
  if (n < 0 || n > p.T || start < 0 || start > p.len_cap - n) {
    record_status(p.status, VA_ERR_DEVICE_BOUNDS);
    n = 0;
  }
}

// Token and head of row r0 + u * kPass of a sequence (heads fastest), walked from row to
// row: a division each was a quarter of the quantising kernel's instructions.
template <int kPass>
struct RowWalk {
  int t, h;
  __device__ __forceinline__ RowWalk(int r, int heads) {
    t = r / heads;
    h = r - t * heads;
  }
  __device__ __forceinline__ void next(const QuantParams &p) {
    t += p.pass_tokens;
    h += p.pass_heads;
    if (h >= p.Hkv) {
      h -= p.Hkv;
      ++t;
    }
  }
};

// 16 consecutive elements as they are in memory, and as fp32.
template <typename T>
struct Sixteen;
template <>
struct Sixteen<__nv_bfloat16> {
  uint4 v[2];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    v[0] = __ldg(reinterpret_cast<const uint4 *>(p));
    v[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
    reinterpret_cast<uint4 *>(p)[0] = v[0];
    reinterpret_cast<uint4 *>(p)[1] = v[1];
  }
  __device__ __forceinline__ void get(float (&f)[16]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        f[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void set(const float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[i] = make_uint4(pack_bf16(f[8 * i], f[8 * i + 1]), pack_bf16(f[8 * i + 2], f[8 * i + 3]),
                        pack_bf16(f[8 * i + 4], f[8 * i + 5]), pack_bf16(f[8 * i + 6], f[8 * i + 7]));
  }
};
template <>
struct Sixteen<float> {
  float4 v[4];
  __device__ __forceinline__ void load(const float *p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __ldg(reinterpret_cast<const float4 *>(p) + i);
  }
  __device__ __forceinline__ void store(float *p) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float4 *>(p)[i] = v[i];
  }
  __device__ __forceinline__ void get(float (&f)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[4 * i] = v[i].x;
      f[4 * i + 1] = v[i].y;
      f[4 * i + 2] = v[i].z;
      f[4 * i + 3] = v[i].w;
    }
  }
  __device__ __forceinline__ void set(const float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  }
};

// Exponent e of the row scale 2^e: the least e >= -126 with amax <= top * 2^e,
// top = 448 = 1.75 * 2^8 (e4m3) or 6 * 448 = 1.3125 * 2^11 (e2m1).
template <int FMT>
__device__ __forceinline__ int row_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  constexpr int kTop = FMT == VA_KV_E4M3 ? 8 : 11;
  constexpr uint32_t kMant = FMT == VA_KV_E4M3 ? 0x600000u : 0x280000u;  // .75, .3125
  const int e = (int)(bits >> 23) - 127 - kTop + ((bits & 0x7fffffu) > kMant ? 1 : 0);
  return max(e, -126);  // (zero and subnormal rows end here)
}

// amax / 6 with the remainder's sign kept in the last bit (rounded to odd), so that
// rounding it to e4m3 is the rounding of the exact quotient.
__device__ __forceinline__ float sixth_to_odd(float y) {
  const float q = __fdiv_rz(y, 6.f);
  return fmaf(q, -6.f, y) != 0.f ? __uint_as_float(__float_as_uint(q) | 1u) : q;
}

// |y| / g for the rounding to e2m1, whose borders m g (m = 0.25, 0.75, .. 5) have at
// most 7 significant bits.
//  bf16 input: y has 8 bits, so y = m g or |y - m g| >= 2^-8 |y|.  The product with
//    the rounded reciprocal is within 2^-22 of the quotient; rounded to 12 bits it is
//    the border itself in the first case and on the right side in the second.
//  fp32 input: the quotient is rounded once from its residual, then moved off a
//    border that it has only been rounded to.
// (q0: y * inv)
template <typename T>
__device__ __forceinline__ float group_quotient(float y, float g, float inv, float q0) {
  if constexpr (sizeof(T) == 2) {
    return __uint_as_float((__float_as_uint(q0) + 0x800u) & 0xfffff000u);
  } else {
    const float a = fabsf(y), qa = fabsf(q0);
    const float q = fmaf(fmaf(-qa, g, a), inv, qa);
    const float r = fmaf(-q, g, a);
    const uint32_t b = __float_as_uint(q);
    // (a zero stays one, with its sign)
    return copysignf(r == 0.f ? q : __uint_as_float((r < 0.f && b != 0 ? b - 1 : b) | 1u), y);
  }
}

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kQuantThreads, 8) quantize_kernel(const QuantParams p) {
  using R = QRow<FMT, D>;
  constexpr int LPR = D / 16;                     // lanes of a row
  constexpr int kPass = kQuantThreads / LPR;      // rows of a pass
  constexpr int kRows = sizeof(T) == 2 ? 4 : 2;   // rows of a thread, loads first
  const int b = blockIdx.y;
  const TokenRows src = blockIdx.z == 0 ? p.k : p.v;
  void *cache = blockIdx.z == 0 ? p.k_cache : p.v_cache;
  const int li = threadIdx.x % LPR;
  int start, n;
  quant_range(p, b, start, n);
  const int rows = n * p.Hkv;  // (T * Hkv < 2^31)
  const T *x = static_cast<const T *>(src.p) + (size_t)b * src.batch + li * 16;
  const int r0 = blockIdx.x * kPass * kRows + threadIdx.x / LPR;
  if (blockIdx.x * kPass * kRows >= rows) return;
  Sixteen<T> in[kRows];
  RowWalk<kPass> at(r0, p.Hkv);
  const RowWalk<kPass> first = at;
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const bool live = r0 + u * kPass < rows;  // (lanes past the end take the first row again)
    in[u].load(x + (size_t)(live ? at.t : 0) * src.token + (size_t)(live ? at.h : 0) * D);
    at.next(p);
  }
  at = first;
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int r = r0 + u * kPass, row_t = at.t, row_h = at.h;
    at.next(p);
    float f[16];
    in[u].get(f);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(f[i]));
    float row = amax;
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) row = max_nan(row, __shfl_xor_sync(0xffffffffu, row, o));
    // a row that holds an infinity or a NaN reads back as NaN
    const bool bad = !(row <= 3.402823466e38f);
    const int e = row_exponent<FMT>(row);
    const float up = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e (normal: e is -126 to 120)
    const uint32_t scale = bad ? 0x7fc00000u : (uint32_t)(e + 127) << 23;
    uint32_t group = 0, code[4] = {0u, 0u, 0u, 0u};
    if (!bad) {
      if constexpr (FMT == VA_KV_E4M3) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t two = __nv_cvt_float2_to_fp8x2(mul2(make_float2(f[2 * i], f[2 * i + 1]), make_float2(up, up)),
                                                        __NV_SATFINITE, __NV_E4M3);
          code[i / 2] |= two << (16 * (i & 1));
        }
      } else {
        group = __nv_cvt_float_to_fp8(sixth_to_odd(amax * up), __NV_SATFINITE, __NV_E4M3);
        const float g = e4m3_to_float(group), inv = g > 0.f ? __frcp_rn(g) : 0.f;  // (g = 0: codes +-0)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 y = mul2(make_float2(f[2 * i], f[2 * i + 1]), make_float2(up, up));
          const float2 q0 = mul2(y, make_float2(inv, inv));
          const uint32_t two = __nv_cvt_float2_to_fp4x2(
              make_float2(group_quotient<T>(y.x, g, inv, q0.x), group_quotient<T>(y.y, g, inv, q0.y)), __NV_E2M1,
              cudaRoundNearest);
          code[i / 4] |= two << (8 * (i & 3));
        }
      }
    }
    uint32_t tail[4] = {scale, 0u, 0u, 0u};
    if constexpr (FMT == VA_KV_E2M1) {
      // the row's group scales, byte i from its lane i
      uint32_t w = group << (8 * (li & 3));
      w |= __shfl_xor_sync(0xffffffffu, w, 1);
      w |= __shfl_xor_sync(0xffffffffu, w, 2);
      if constexpr (D == 128) {
        tail[1] = __shfl_xor_sync(0xffffffffu, w, 4);
        tail[2] = scale;
      } else {
        tail[1] = scale;
      }
      tail[0] = w;
    }
    if (r >= rows) continue;
    uint8_t *dst = quant_row(p, cache, R::kBytes, b, start + row_t, row_h);
    if (dst == nullptr) continue;
    if constexpr (FMT == VA_KV_E4M3)
      reinterpret_cast<uint4 *>(dst)[li] = make_uint4(code[0], code[1], code[2], code[3]);
    else
      reinterpret_cast<uint2 *>(dst)[li] = make_uint2(code[0], code[1]);
    if (li == 0) *reinterpret_cast<uint4 *>(dst + R::kCodeBytes) = make_uint4(tail[0], tail[1], tail[2], tail[3]);
  }
}

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kQuantThreads, 8) dequantize_kernel(const QuantParams p) {
  using R = QRow<FMT, D>;
  constexpr int LPR = D / 16;
  constexpr int kPass = kQuantThreads / LPR;
  constexpr int kRows = 4;
  const int b = blockIdx.y;
  const TokenRows out = blockIdx.z == 0 ? p.k : p.v;
  void *cache = blockIdx.z == 0 ? p.k_cache : p.v_cache;
  const int li = threadIdx.x % LPR;
  int start, n;
  quant_range(p, b, start, n);
  const int rows = n * p.Hkv;
  T *y = static_cast<T *>(const_cast<void *>(out.p)) + (size_t)b * out.batch + li * 16;
  const int r0 = blockIdx.x * kPass * kRows + threadIdx.x / LPR;
  if (blockIdx.x * kPass * kRows >= rows) return;
  uint4 code[kRows], tail[kRows];
  bool live[kRows];
  RowWalk<kPass> at(r0, p.Hkv);
  const RowWalk<kPass> first = at;
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int r = r0 + u * kPass, row_t = at.t, row_h = at.h;
    at.next(p);
    live[u] = false;
    if (r >= rows) continue;
    const uint8_t *src = quant_row(p, cache, R::kBytes, b, start + row_t, row_h);
    if (src == nullptr) continue;
    live[u] = true;
    if constexpr (FMT == VA_KV_E4M3) {
      code[u] = __ldg(reinterpret_cast<const uint4 *>(src) + li);
    } else {
      const uint2 c = __ldg(reinterpret_cast<const uint2 *>(src) + li);
      code[u] = make_uint4(c.x, c.y, 0u, 0u);
    }
    tail[u] = __ldg(reinterpret_cast<const uint4 *>(src + R::kCodeBytes));
  }
  at = first;
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int row_t = at.t, row_h = at.h;
    at.next(p);
    if (!live[u]) continue;
    float f[16];
    const uint32_t w[4] = {code[u].x, code[u].y, code[u].z, code[u].w};
    float s;
    if constexpr (FMT == VA_KV_E4M3) {
      s = __uint_as_float(tail[u].x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 two = __half22float2(e4m3x2_to_half2(w[i / 2] >> (16 * (i & 1)) & 0xffffu));
        f[2 * i] = two.x * s;
        f[2 * i + 1] = two.y * s;
      }
    } else {
      const uint32_t gw = D == 128 && li >= 4 ? tail[u].y : tail[u].x;
      s = __uint_as_float(D == 128 ? tail[u].z : tail[u].y);
      const float g = e4m3_to_float(gw >> (8 * (li & 3)) & 0xffu);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 two = __half22float2(e2m1x2_to_half2(w[i / 4] >> (8 * (i & 3)) & 0xffu));
        f[2 * i] = two.x * g * s;  // (code * g is exact, so is the product with a power of two)
        f[2 * i + 1] = two.y * g * s;
      }
    }
    Sixteen<T> o;
    o.set(f);
    o.store(y + (size_t)row_t * out.token + (size_t)row_h * D);
  }
}

namespace {
template <int FMT, int D, typename T>
cudaError_t launch_t(QuantParams p, bool write, cudaStream_t stream) {
  const int pass = kQuantThreads / (D / 16), per_block = pass * (write && sizeof(T) == 4 ? 2 : 4);
  p.pass_tokens = pass / p.Hkv;
  p.pass_heads = pass % p.Hkv;
  const long long rows = (long long)p.T * p.Hkv;
  const dim3 grid((unsigned)((rows + per_block - 1) / per_block), (unsigned)p.B, 2);
  if (write)
    quantize_kernel<FMT, D, T><<<grid, kQuantThreads, 0, stream>>>(p);
  else
    dequantize_kernel<FMT, D, T><<<grid, kQuantThreads, 0, stream>>>(p);
  return cudaGetLastError();
}
template <int FMT, int D>
cudaError_t launch_d(const QuantParams &p, bool write, cudaStream_t stream) {
  return p.fp32 ? launch_t<FMT, D, float>(p, write, stream) : launch_t<FMT, D, __nv_bfloat16>(p, write, stream);
}
cudaError_t launch_quant(const QuantParams &p, bool write, cudaStream_t stream) {
  if (p.format == VA_KV_E4M3)
    return p.D == 128 ? launch_d<VA_KV_E4M3, 128>(p, write, stream) : launch_d<VA_KV_E4M3, 64>(p, write, stream);
  return p.D == 128 ? launch_d<VA_KV_E2M1, 128>(p, write, stream) : launch_d<VA_KV_E2M1, 64>(p, write, stream);
}
}  // namespace

cudaError_t launch_quantize_kv(const QuantParams &p, cudaStream_t stream) { return launch_quant(p, true, stream); }
cudaError_t launch_dequantize_kv(const QuantParams &p, cudaStream_t stream) { return launch_quant(p, false, stream); }

}  // namespace va
