// What the interval-mask attention kernels share: the score transforms and
// the look-up of a CTA's table entry.
#pragma once
#include "mc_layer_internal.h"
#include "ptx.cuh"

namespace mc {

constexpr float kOptLog2e = 1.4426950408889634f;
constexpr float kOptLn2 = 0.6931471805599453f;

template <bool B>
struct BoolC {
  static constexpr bool value = B;
};

template <int N>
struct IntC {
  static constexpr int value = N;
};

// 1 / x (one ulp; 1 / infinity = 0), x >= 1 here.
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Scores are kept in log2 units: y = z log2(e) with z = q k / sqrt(d), so
// that P = exp2(y - lse log2(e)).  With a cap c,
//   c tanh(z / c) = c - 2 c / (1 + exp(2 z / c)):
// for a large |z| the quotient is 0 or 1 and nothing overflows; for a small
// one the difference of the two terms has an absolute error of about
// 2 c 2^-24, which is what counts in an exponent.
struct ScoreConst {
  float mul;     // no cap: log2(e) / sqrt(d); cap: 2 log2(e) / (sqrt(d) c)
  float arg;     // cap: 1 / (sqrt(d) c), the tanh's argument per raw score
  float cap2;    // c log2(e)
  float slope2;  // slope log2(e)
};

// For |t| <= kCapSmall, tanh(t) = t p(t^2) with the degree-4 polynomial p of
// least largest error in tanh: 5.0e-08 (fitted on a Chebyshev grid by
// reweighted least squares; 1.2e-7 with 32-bit arithmetic, as the quotient
// form's).  It takes no special-function operations, of which the quotient
// form needs two per score beside the exponential: those run at 32 results per
// clock and SM.  Scores mostly are that far below their cap; a warp with one
// that is not takes the quotient form.
constexpr float kCapSmall = 0.65625f;

// p(t^2), times `scale`: c = scale * coefficients.
struct CapPoly {
  float k0, k1, k2, k3, k4;
};
__device__ __forceinline__ CapPoly cap_poly(float scale) {
  return {0.9999991655349731f * scale, -0.33329296112060547f * scale, 0.13278807699680328f * scale,
          -0.05090659484267235f * scale, 0.013971595093607903f * scale};
}
__device__ __forceinline__ float2 cap_small(float2 t, const CapPoly& c) {
  const float2 u = __fmul2_rn(t, t);
  float2 p = __ffma2_rn(make_float2(c.k4, c.k4), u, make_float2(c.k3, c.k3));
  p = __ffma2_rn(p, u, make_float2(c.k2, c.k2));
  p = __ffma2_rn(p, u, make_float2(c.k1, c.k1));
  return __ffma2_rn(p, u, make_float2(c.k0, c.k0));
}

template <bool CAP, bool BIAS>
__device__ __forceinline__ ScoreConst score_const(float rsqrt_d, float softcap, float slope) {
  ScoreConst c;
  c.mul = rsqrt_d * kOptLog2e;
  c.arg = 0.f;
  c.cap2 = 0.f;
  c.slope2 = 0.f;
  if constexpr (CAP) {
    c.arg = rsqrt_d / softcap;
    c.mul = 2.f * kOptLog2e * c.arg;
    c.cap2 = softcap * kOptLog2e;
  }
  if constexpr (BIAS) c.slope2 = slope * kOptLog2e;
  return c;
}

// r = 1 / (1 + exp(2 z / c)) of two raw scores: tanh(z / c) = 1 - 2 r and
// 1 - tanh^2 = 4 r (1 - r).
__device__ __forceinline__ float2 cap_r(float2 x, float mul) {
  const float2 t = __fmul2_rn(x, make_float2(mul, mul));
  const float2 e = __fadd2_rn(make_float2(fast_exp2(t.x), fast_exp2(t.y)), make_float2(1.f, 1.f));
  return make_float2(fast_rcp(e.x), fast_rcp(e.y));
}

// The table entry of this CTA (in dispatch order) and its head: `tables` has
// n entries, heads fastest when `head_major`.  False (after recording an
// error) when the entry is not one of this shape.
__device__ __forceinline__ bool opt_entry(const int32_t* tables, bool head_major, int b, int nb,
                                          int4& entry, int& hh, int* status) {
  const int rank = static_cast<int>(head_major ? blockIdx.y : blockIdx.x);
  hh = static_cast<int>(head_major ? blockIdx.x : blockIdx.y);
  entry = *reinterpret_cast<const int4*>(tables + 4 * static_cast<int64_t>(rank));
  const bool ok = entry.x >= 0 && entry.x < b && entry.y >= 0 && entry.y < nb;
  if (!ok && threadIdx.x == 0) record_error(status, MC_ERR_DEVICE_BOUNDS, kSiteAttention);
  return ok;
}

// Items of a persistent kernel, (table entry, head) pairs: the longest entries
// of all heads come first, and the grid's CTAs are dealt them in a snake, so
// that their shares are even.  (Groups of 1 to 7 heads at a time, whose K and V
// stay in L2, cost more by their uneven shares than they saved: 742 to 839 us
// against 734 us over 16,384 tokens and 16 heads.)
// Item r of this CTA: its table rank and head; false when its share is done.
// (b ceil(s / 128) H < 2^31 by the entry points' limits.)
__device__ __forceinline__ bool opt_item(int r, int n, int H, int& rank, int& hh) {
  const unsigned G = gridDim.x, c = blockIdx.x;
  const unsigned k = static_cast<unsigned>(r) * G + ((r & 1) ? G - 1 - c : c);
  if (k >= static_cast<unsigned>(n) * static_cast<unsigned>(H)) return false;
  rank = static_cast<int>(k / static_cast<unsigned>(H));
  hh = static_cast<int>(k % static_cast<unsigned>(H));
  return true;
}

// A table entry that is not one of this shape is reported and taken as an
// empty one of block 0.
__device__ __forceinline__ int4 opt_checked(int4 e, int b, int nb, int* status) {
  if (e.x >= 0 && e.x < b && e.y >= 0 && e.y < nb) return e;
  record_error(status, MC_ERR_DEVICE_BOUNDS, kSiteAttention);
  return make_int4(0, 0, 0, 0);
}

}  // namespace mc
