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
__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

}  // namespace va
