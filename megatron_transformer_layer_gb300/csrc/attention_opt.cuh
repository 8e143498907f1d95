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
__device__ __forceinline__ ScoreConst score_const(float rsqrt_d, float softcap, float slope) {
  ScoreConst c;
  c.mul = rsqrt_d * kOptLog2e;
  c.cap2 = 0.f;
  c.slope2 = 0.f;
  if constexpr (CAP) {
    c.mul = 2.f * rsqrt_d * kOptLog2e / softcap;
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

// Items of a persistent kernel, (table entry, head) pairs: heads are taken in
// groups of `group`, within a group the longest entries of all its heads come
// first, and the grid's CTAs are dealt them in a snake, so that their shares
// are even.  A group's K and V are what the CTAs running together read again
// and again: the group is as large as fits in L2 beside everything else.
inline int opt_head_group(int b, int s, int H, int d) {
  const int64_t head_bytes = static_cast<int64_t>(b) * s * d * 4;  // K and V of one head
  const int64_t fit = (64ll << 20) / head_bytes;
  return static_cast<int>(fit < 1 ? 1 : fit < H ? fit : H);
}

// Item r of this CTA: its table rank and head; false when its share is done.
// (b ceil(s / 128) H < 2^31 by the entry points' limits.)
__device__ __forceinline__ bool opt_item(int r, int n, int H, int group, int& rank, int& hh) {
  const unsigned G = gridDim.x, c = blockIdx.x;
  const unsigned k = static_cast<unsigned>(r) * G + ((r & 1) ? G - 1 - c : c);
  if (k >= static_cast<unsigned>(n) * static_cast<unsigned>(H)) return false;
  const unsigned per_group = static_cast<unsigned>(n) * static_cast<unsigned>(group);
  const unsigned g0 = k / per_group * static_cast<unsigned>(group);  // the group's first head
  const unsigned heads = min(static_cast<unsigned>(group), static_cast<unsigned>(H) - g0);
  const unsigned in = k - g0 * static_cast<unsigned>(n);
  rank = static_cast<int>(in / heads);
  hh = static_cast<int>(g0 + in % heads);
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
