// Rows of K and V held in 8 or 4 bits: layout and conversions.
//
// A quantised row is one token of one kv-head, a run of kBytes bytes:
//   e4m3  D codes, the row scale s (fp32), 12 zero bytes;       x = code * s
//   e2m1  D/2 bytes of codes (element 2j in the low half of byte j), D/16 group
//         scales g (e4m3), s (fp32), zeros to a multiple of 16;  x = code * g * s
// s is a power of two, so that every step of the conversion is exact but for the
// roundings that the format asks for: a call gives the same bytes as any other
// correctly rounded implementation.  The run is an odd multiple of 16 bytes, so
// 16-byte reads of the same column of consecutive rows go through all banks of
// shared memory, and a row can be moved by whatever moves rows of 16-byte multiples.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "verify_attn.h"

namespace va {

template <int FMT, int D>
struct QRow {
  static constexpr int kCodeBytes = FMT == VA_KV_E4M3 ? D : D / 2;
  static constexpr int kTailBytes = 16;  // group scales, row scale, zeros
  static constexpr int kBytes = kCodeBytes + kTailBytes;
  static constexpr int kScaleOff = kCodeBytes + (FMT == VA_KV_E4M3 ? 0 : D / 16);
  static_assert(kScaleOff + 4 <= kBytes && (kBytes / 16) % 2 == 1, "odd multiple of 16 bytes");
};

// Two e2m1 codes of a byte, or two e4m3 codes of 16 bits, as halves (exact).
__device__ __forceinline__ __half2 e2m1x2_to_half2(uint32_t byte) {
  return __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)byte, __NV_E2M1));
}
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t two) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
}
// The eight e2m1 codes of a word as halves (the conversion reads its byte of the word).
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(w));
}
__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

}  // namespace va
