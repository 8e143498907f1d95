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
  float cap2;    // c log2(e)
  float slope2;  // slope log2(e)
};

template <bool CAP, bool BIAS>
__device__ __forceinline__ ScoreConst score_const(float rsqrt_d, float softcap, const float* slopes,
                                                  int head) {
  ScoreConst c;
  c.mul = rsqrt_d * kOptLog2e;
  c.cap2 = 0.f;
  c.slope2 = 0.f;
  if constexpr (CAP) {
    c.mul = 2.f * rsqrt_d * kOptLog2e / softcap;
    c.cap2 = softcap * kOptLog2e;
  }
  if constexpr (BIAS) c.slope2 = slopes[head] * kOptLog2e;
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

}  // namespace mc
