// Pieces shared by the keys-on-lanes attention kernels: row maxima and sums over the
// keys of a warp, TMEM columns as fp32, and their scaling.
#pragma once

#include "va_common.cuh"
#include "va_tcgen05.cuh"

namespace va {

// Row-wise block of a warp: v[N] per lane -> lane holds the warp maximum of
// max(N/32, 1) rows (row j + (N/32)*lane for N >= 32, lane / (32/N) below).
template <int N, int O>
struct WarpScatterMax {
  static __device__ __forceinline__ void run(float *v, int lane) {
    if constexpr (O == 0) {
      return;
    } else if constexpr (N >= 2) {
      constexpr int H = N / 2;
      const bool up = (lane & O) != 0;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float send = up ? v[i] : v[i + H];
        const float keep = up ? v[i + H] : v[i];
        v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, O));
      }
      WarpScatterMax<H, O / 2>::run(v, lane);
    } else {
      v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], O));
      WarpScatterMax<1, O / 2>::run(v, lane);
    }
  }
};

// The same reduce-scatter with sums: lane l ends with the warp's sum of the
// rows WarpScatterMax leaves it.
template <int N, int O>
struct WarpScatterSum {
  static __device__ __forceinline__ void run(float *v, int lane) {
    if constexpr (O == 0) {
      return;
    } else if constexpr (N >= 2) {
      constexpr int H = N / 2;
      const bool up = (lane & O) != 0;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float send = up ? v[i] : v[i + H];
        const float keep = up ? v[i + H] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, O);
      }
      WarpScatterSum<H, O / 2>::run(v, lane);
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], O);
      WarpScatterSum<1, O / 2>::run(v, lane);
    }
  }
};

// NR fp32 columns of this thread's TMEM lane.
template <int NR>
__device__ __forceinline__ void tmem_ld_f(uint32_t taddr, float (&x)[NR]) {
  if constexpr (NR == 8) {
    uint32_t u[8];
    tmem_ld8(taddr, u);
    tmem_ld_wait(u);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(u[j]);
  } else if constexpr (NR == 16) {
    uint32_t u[16];
    tmem_ld16(taddr, u);
    tmem_ld_wait(u);
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = __uint_as_float(u[j]);
  } else {
#pragma unroll
    for (int h = 0; h < NR / 32; ++h) {
      uint32_t u[32];
      tmem_ld32(taddr + 32 * h, u);
      tmem_ld_wait(u);
#pragma unroll
      for (int j = 0; j < 32; ++j) x[32 * h + j] = __uint_as_float(u[j]);
    }
  }
}

// Multiply column j of this lane's NR columns at taddr by a[j].
template <int NR>
__device__ __forceinline__ void tmem_scale_cols(uint32_t taddr, const float *a) {
  if constexpr (NR == 16) {
    uint32_t u[16];
    tmem_ld16(taddr, u);
    tmem_ld_wait(u);
#pragma unroll
    for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * a[j]);
    tmem_st16(taddr, u);
  } else {
    // 16 columns at a time, each stored before the next is loaded: this rare
    // path then needs few registers next to the 64-row softmax state
#pragma unroll
    for (int h = 0; h < NR / 16; ++h) {
      uint32_t u[16];
      tmem_ld16(taddr + 16 * h, u);
      tmem_ld_wait(u);
#pragma unroll
      for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * a[16 * h + j]);
      tmem_st16(taddr + 16 * h, u);
      tmem_st_wait();
    }
  }
}

}  // namespace va
