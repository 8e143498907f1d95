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
  float slope;   // the bias per distance: slope sqrt(d) for raw scores, with a cap slope log2(e)
};

// For |t| <= kCapSmall, tanh(t) = t p(t^2) with the cubic p of least largest
// error in tanh: 7.4e-08 (fitted on a Chebyshev grid by reweighted least squares;
// 1.2e-7 with 32-bit arithmetic, as the quotient form's).  It takes no
// special-function operations, of which the quotient form needs two per score
// beside the exponential (an exponential 4 clocks per warp and quarter SM, a
// reciprocal 8, a packed multiply-add of two scores 2).  Scores mostly are
// that far below their cap; a warp with one that is not takes the quotient form.
constexpr float kCapSmall = 0.46875f;

// scale * tanh(arg x) = x (k0 + k1 x^2 + k2 x^4 + k3 x^6) for raw scores x: the
// powers of `arg` are in the coefficients.
struct CapPoly {
  float k0, k1, k2, k3;
};
__device__ __forceinline__ CapPoly cap_poly(float scale, float arg) {
  const float a2 = arg * arg;
  const float a1 = scale * arg, a3 = a1 * a2, a5 = a3 * a2;
  return {0.9999985694885254f * a1, -0.3332448899745941f * a3, 0.13184478878974915f * a5,
          -0.04449363797903061f * (a5 * a2)};
}
// The factor of x, from u = x^2.
__device__ __forceinline__ float2 cap_small(float2 u, const CapPoly& c) {
  float2 p = __ffma2_rn(make_float2(c.k3, c.k3), u, make_float2(c.k2, c.k2));
  p = __ffma2_rn(p, u, make_float2(c.k1, c.k1));
  return __ffma2_rn(p, u, make_float2(c.k0, c.k0));
}
// Raw scores up to this size (absolute) are small.  Caps are 2^-16 .. 2^16
// (checked at the entry points): 1 / (sqrt(d) c) is 1.3e-6 .. 8192, so that the
// coefficients, log2(e) / sqrt(d) times up to its sixth power, are normal.
__device__ __forceinline__ float cap_small_limit(float arg) { return kCapSmall / arg; }

template <bool CAP, bool BIAS>
__device__ __forceinline__ ScoreConst score_const(float rsqrt_d, float softcap, float slope) {
  ScoreConst c;
  c.mul = rsqrt_d * kOptLog2e;
  c.arg = 0.f;
  c.cap2 = 0.f;
  c.slope = 0.f;
  if constexpr (CAP) {
    c.arg = rsqrt_d / softcap;
    c.mul = 2.f * kOptLog2e * c.arg;
    c.cap2 = softcap * kOptLog2e;
  }
  if constexpr (BIAS) c.slope = CAP ? slope * kOptLog2e : slope / rsqrt_d;
  return c;
}

// r = 1 / (1 + exp(2 z / c)) of two raw scores: tanh(z / c) = 1 - 2 r and
// 1 - tanh^2 = 4 r (1 - r).
__device__ __forceinline__ float2 cap_r(float2 x, float mul) {
  const float2 t = __fmul2_rn(x, make_float2(mul, mul));
  const float2 e = __fadd2_rn(make_float2(fast_exp2(t.x), fast_exp2(t.y)), make_float2(1.f, 1.f));
  return make_float2(fast_rcp(e.x), fast_rcp(e.y));
}

// x[i] <- x[i] - slope |d0 + i|, i < N, for either sign of the slope.  The
// distance is exact (below 2^24), so the bias has one rounding of its own size;
// |slope i + slope d0|, the second product formed once, is off by a rounding of
// 127 slopes next to the query itself (1e-5 of a log-sum-exp for a slope of 2)
// and was no faster: a causal forward over 16,384 tokens and 16 heads 884 us
// against 867 us, 4 x 1037 tokens the same.  Products with an absolute value
// taken off them, one branch per sign, took 987 us, packed 1006 us.
template <int N>
__device__ __forceinline__ void bias_scores(float* x, float slope, float d0) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = fmaf(-slope, fabsf(d0 + static_cast<float>(i)), x[i]);
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

// Items of a persistent kernel: (table entry, head) pairs.  Up to four waves of
// them are dealt to one CTA per SM in a snake, the longest entries of all heads
// first.  More are one CTA each, of which as many start as fit and steal the
// others' indices as they finish (clc_request: a request takes one to two
// microseconds, which a short grid shows: 27 us against 24 us for a backward of
// 192 items, 36.7 against 35.8 us for a forward of 576; but 2048 items dealt
// take 98 us where stolen ones take 89).  Those take heads in groups whose K and V (or Q and dO), read
// again and again by the CTAs running together, stay in L2, each group's
// longest entries first: 64 MB against 32 or 96 MB at a time took 722, 751 and
// 743 us for a causal forward over 16,384 tokens and 16 heads.
struct OptGrid {
  int ctas;
  int steal;
  int head_group;
};
inline OptGrid opt_grid(int b, int s, int H, int d) {
  const int64_t items = static_cast<int64_t>(b) * ((s + 127) / 128) * H;
  if (items <= 4ll * num_sms())
    return {static_cast<int>(items < num_sms() ? items : num_sms()), 0, H};
  const int64_t head_bytes = static_cast<int64_t>(b) * s * d * 4;
  const int64_t fit = (64ll << 20) / head_bytes;
  // equal groups: a small last one would leave its long items for the end
  const int groups = fit < 1 ? H : fit < H ? static_cast<int>(H / fit) : 1;
  return {static_cast<int>(items), 1, (H + groups - 1) / groups};
}

// Item k of the grid: its table rank and head.
// (n = b ceil(s / 128) entries; n H < 2^31 by the entry points' limits.)
__device__ __forceinline__ void opt_item(int k, int n, int H, int group, int& rank, int& hh) {
  const unsigned per_group = static_cast<unsigned>(n) * static_cast<unsigned>(group);
  const unsigned g0 = static_cast<unsigned>(k) / per_group * static_cast<unsigned>(group);
  const unsigned heads = min(static_cast<unsigned>(group), static_cast<unsigned>(H) - g0);
  const unsigned in = static_cast<unsigned>(k) - g0 * static_cast<unsigned>(n);
  rank = static_cast<int>(in / heads);
  hh = static_cast<int>(g0 + in % heads);
}

// This CTA's items, for one thread: its own, then its share of the snake, or
// stolen ones, each requested one ahead.  `response` is 16 aligned bytes of
// shared memory, `bar` an mbarrier of one arrival.
struct OptItems {
  void* response;
  uint64_t* bar;
  int total;    // items of the grid
  int steal;
  int k;        // the item at hand
  int n;        // items taken before it
  bool more;    // `k` is valid
  bool asked;   // a request is under way
  __device__ __forceinline__ OptItems(void* r, uint64_t* b, int items, int steal_)
      : response(r), bar(b), total(items), steal(steal_), k(static_cast<int>(blockIdx.x)), n(0),
        more(true), asked(false) {
    ask();
  }
  __device__ __forceinline__ void ask() {
    if (!steal) return;
    clc_request(response, bar);
    asked = true;
  }
  // The next item into k; asks for the one after it.  False on a timeout.
  __device__ __forceinline__ bool next(int* status) {
    if (!steal) {
      ++n;
      const unsigned G = gridDim.x, c = blockIdx.x;
      const unsigned at = static_cast<unsigned>(n) * G + ((n & 1) ? G - 1 - c : c);
      more = at < static_cast<unsigned>(total);
      k = static_cast<int>(at);
      return true;
    }
    if (!mbar_wait(bar, n & 1, status, kSiteAttention)) return false;
    asked = false;
    ++n;
    more = clc_response(response, k);
    if (more) {
      fence_proxy_async_smem();  // the response has been read before it is overwritten
      ask();
    }
    return true;
  }
  // A response still under way must land before the CTA exits.
  __device__ __forceinline__ void finish(int* status) {
    if (asked) mbar_wait(bar, n & 1, status, kSiteAttention, 200000000ull, false);
  }
};

// Bits [first, end) of a word.
__device__ __forceinline__ uint32_t bit_range(int first, int end) {
  first = min(max(first, 0), 32);
  end = min(max(end, 0), 32);
  const uint32_t below_end = end == 32 ? 0xFFFFFFFFu : (1u << end) - 1u;
  const uint32_t below_first = first == 32 ? 0xFFFFFFFFu : (1u << first) - 1u;
  return below_end & ~below_first;
}

// A table entry that is not one of this shape is reported and taken as an
// empty one of block 0.
__device__ __forceinline__ int4 opt_checked(int4 e, int b, int nb, int* status) {
  if (e.x >= 0 && e.x < b && e.y >= 0 && e.y < nb) return e;
  record_error(status, MC_ERR_DEVICE_BOUNDS, kSiteAttention);
  return make_int4(0, 0, 0, 0);
}

}  // namespace mc
