// Score shaping shared by the attention kernels and the accumulated-weight
// pass: a tanh cap on the scores, a bias that falls with distance (a slope
// per query head), a sliding window and a per-sequence document start.
//
//   s = scale q.k;  s = c tanh(s / c) if c > 0;  s = s - slope_h |d|,
//   d = pos_q - pos_k,
//   visible: d < window, and for a prefix slot j: j >= key_start_b.
//
// A prefix key's position is its slot; draft token t's is token_pos[b][t] (or
// L_b + t).  Positions are used relative to L_b: offsets below 2^23 in
// magnitude and prefix slots within 2^24 of L_b are exact in fp32, and farther
// ones (which a window below 2^23 always hides) are off by 2^-24 of the
// distance, the rounding of the bias itself.
//
// Scores leave here in base-2 units (times log2 e), so that the softmaxes'
// exponent is 2^(s - m) with no further factor.
#pragma once

#include "va_common.cuh"
#include "va_kernels.h"

namespace va {

constexpr int kModMaxOff = 1 << 23;

// ---------------------------------------------------------------------------
// tanh
// ---------------------------------------------------------------------------
// tanh(y) = y P(y^2) / Q(y^2), a rational approximation fitted to the relative
// error on |y| <= 9.02 (reweighted least squares): 5.8e-8 with the coefficients
// below, 3.7e-7 with every step rounded to fp32 and the reciprocal too, whose
// approximation may add 6e-8.  Past 9.02, tanh rounds to 1 in fp32.  The hardware's one-instruction
// tanh is off by 2^-11, which a cap of 50 would turn into 0.02 of a score;
// 1 - 2 / (1 + e^2y) loses the small scores' digits the same way.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// y cut to where the approximation holds; NaN stays NaN.
__device__ __forceinline__ float cut_tanh_arg(float y) {
  float d;
  asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\tmin.NaN.f32 %0, t, %3;\n\t}"
      : "=f"(d) : "f"(y), "f"(-9.02f), "f"(9.02f));
  return d;
}

// cap2 * tanh of a pair; cap2 multiplies the numerators before the division.
__device__ __forceinline__ float2 capped_tanh2(float2 y, float cap2) {
  y.x = cut_tanh_arg(y.x);
  y.y = cut_tanh_arg(y.y);
  auto two = [](float c) { return make_float2(c, c); };
  const float2 z = mul2(y, y);
  float2 p = fma2(two(1.33188971e-08f), z, two(2.05833530e-05f));
  p = fma2(p, z, two(3.49402661e-03f));
  p = fma2(p, z, two(1.33797109e-01f));
  p = fma2(p, z, two(1.0f));
  float2 q = fma2(two(7.76194668e-07f), z, two(3.28308001e-04f));
  q = fma2(q, z, two(2.58710440e-02f));
  q = fma2(q, z, two(4.67130274e-01f));
  q = fma2(q, z, two(1.0f));
  return mul2(mul2(mul2(y, two(cap2)), p), make_float2(rcp_approx(q.x), rcp_approx(q.y)));
}
__device__ __forceinline__ float capped_tanh(float y, float cap2) {
  y = cut_tanh_arg(y);
  const float z = y * y;
  float p = fmaf(1.33188971e-08f, z, 2.05833530e-05f);
  p = fmaf(p, z, 3.49402661e-03f);
  p = fmaf(p, z, 1.33797109e-01f);
  p = fmaf(p, z, 1.0f);
  float q = fmaf(7.76194668e-07f, z, 3.28308001e-04f);
  q = fmaf(q, z, 2.58710440e-02f);
  q = fmaf(q, z, 4.67130274e-01f);
  q = fmaf(q, z, 1.0f);
  return (cap2 * y) * p * rcp_approx(q);
}

// raw * (sum of c[k] raw^2k) of N products in place.
template <int N, int K>
__device__ __forceinline__ void cap_small(const float *c, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 r = make_float2(x[i], x[i + 1]);
    const float2 z = mul2(r, r);
    float2 q = make_float2(c[K - 1], c[K - 1]);
#pragma unroll
    for (int k = K - 2; k >= 0; --k) q = fma2(q, z, make_float2(c[k], c[k]));
    q = mul2(q, r);
    x[i] = q.x;
    x[i + 1] = q.y;
  }
}

// Caps N raw products of a thread in place.  A cap well above the usual scores
// leaves small |y|, where tanh is an odd polynomial, with the scale and the cap
// folded into its coefficients and no division: where every product of the warp has
// |y| <= 0.45, of degree 7, and (kMid) up to 0.75 of degree 11 (fitted like the
// above: 2.5e-7 and 2.9e-8 relative; 3.3e-7 and 1.6e-7 in fp32).  A packed
// instruction keeps the FMA pipe for two cycles, and on 256 rows each one of a pair
// costs 8 us of a tree over 128K keys: five or seven against nineteen.
// The weights take one more term (kFine: |y| <= 0.55, degree 9, 3.2e-8; 1.4e-7 in
// fp32): exp(s - lse) shows a score's last digits, and with four terms the weights of a
// chain were off by 3.8e-6, twice what fp32 tanh leaves.
// Code costs as well: warps at different places of more code than the instruction
// caches hold wait for it.  With 64 scores a thread the 256-row tree took 537 us
// where a tile's warps went different ways and 212 where they did not (32 scores:
// 222 and 198), and the keys-on-lanes kernel loses more by the second polynomial
// than it gains (64 rows, scores past 0.45: 335 us with it, 314 without; the
// weights of 256 rows 164 and 200, and 167 with the term more).
// The form decides the last bits, so it may depend on nothing that no row sees: a
// thread whose key is hidden from every row (`hidden`) has no say, and where a thread
// has keys of both kinds (`mixed`) the general form is taken without asking.
template <int N, bool kMid, bool kFine>
__device__ __forceinline__ void cap_scores(const ModParams &m, float (&x)[N], bool hidden, bool mixed) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2) top = max3f(top, fabsf(x[i]), fabsf(x[i + 1]));
  if (hidden) top = 0.f;
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // (none is negative)
  if (mixed) top = INFINITY;
  if (top <= m.small_lim[0]) {
    cap_small<N, kFine ? 5 : 4>(m.small_c, x);
  } else if (kMid && top <= m.small_lim[1]) {
    cap_small<N, 6>(m.small_c6, x);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 y = capped_tanh2(mul2(make_float2(x[i], x[i + 1]), make_float2(m.in_mul, m.in_mul)), m.out_mul);
      x[i] = y.x;
      x[i + 1] = y.y;
    }
  }
}

// ---------------------------------------------------------------------------
// positions and visibility
// ---------------------------------------------------------------------------
// Whether a row's sum of weights holds a key.  NaN scores (a NaN in q) count, so that
// such a row's out and lse come out as NaN.
__device__ __forceinline__ bool mod_row_seen(float l) { return l != 0.f; }

// Position of draft token t of sequence b relative to L_b (clamped).
__device__ __forceinline__ int mod_off(const ModParams &m, int T, int b, int t, int L) {
  if (m.token_pos == nullptr) return t;
  const long long o = (long long)__ldg(m.token_pos + (size_t)b * T + t) - L;
  return (int)max(-(long long)kModMaxOff, min((long long)kModMaxOff, o));
}

// First slot of the prefix that a row at offset `off` sees, in [0, L].
__device__ __forceinline__ int mod_first_slot(const ModParams &m, int b, int off, int L) {
  int lo = m.key_start != nullptr ? __ldg(m.key_start + b) : 0;
  if (m.window > 0) lo = max(lo, L + off - m.window + 1);
  return max(0, min(lo, L));
}

// First slot that any row of sequence b sees (lo) and the first that every row
// sees (hi).  An offset out of range is recorded.
__device__ __forceinline__ void mod_range(const ModParams &m, int T, int b, int L, int *status, int &lo, int &hi) {
  int omin = 0, omax = T - 1;
  if (m.token_pos != nullptr && (m.window > 0 || status != nullptr)) {
    omin = kModMaxOff;
    omax = -kModMaxOff;
#pragma unroll 8
    for (int t = 0; t < T; ++t) {
      const int o = mod_off(m, T, b, t, L);
      omin = min(omin, o);
      omax = max(omax, o);
    }
    if (status != nullptr && (omin <= -kModMaxOff || omax >= kModMaxOff)) record_status(status, VA_ERR_DEVICE_BOUNDS);
  }
  lo = mod_first_slot(m, b, omin, L);
  hi = mod_first_slot(m, b, omax, L);
}

// Draft token t's visibility row with the keys cleared that its window hides.
__device__ __forceinline__ uint64_t mod_window_row(const ModParams &m, int T, int b, int t, int L, uint64_t row) {
  if (m.window <= 0) return row;
  const int o = mod_off(m, T, b, t, L);
  for (int j = 0; j < T; ++j)
    if (o - mod_off(m, T, b, j, L) >= m.window) row &= ~(1ull << j);
  return row;
}

// Bias slope of query head hq in base-2 units, negated (0 without slopes).
__device__ __forceinline__ float mod_slope(const ModParams &m, int hq) {
  return m.slopes != nullptr ? -kModLog2e * __ldg(m.slopes + hq) : 0.f;
}

// A raw product q.k as a score: the cap, then the bias of a key at distance d
// (fp32) for a head of (negated) slope ns.
__device__ __forceinline__ float mod_score(const ModParams &m, float raw, float ns, float d) {
  float s = m.softcap > 0.f ? capped_tanh(raw * m.in_mul, m.out_mul) : raw * m.out_mul;
  if (m.slopes != nullptr) s = fmaf(ns, fabsf(d), s);
  return s;
}

}  // namespace va
