// What the kernels that turn heads by their positions share: vectors of 16 bytes
// and less, divisions by a launch's constants, and a position's angle.
//
// The angle of a far position needs more than 32 bits: inv_freq / 2 pi is
// formed in integer arithmetic as turns in 64-bit fixed point (the float's 24
// bits times 1 / 2 pi to 128 bits), and whole turns drop out of the product
// with the position by the wrap of 64-bit integers.  A position of 2^31 leaves
// an error of 2^-33 turns for frequencies up to 2^64 (above, the 128 bits of
// 1 / 2 pi run out).  What is left of the turn goes to sincospif as a 32-bit
// float of half turns, below 1 and so off by at most 2^-25: 9.4e-8 radians, as
// much as the cosine's own rounding.  (The same in 64-bit floats is exact enough
// too, but they run at 1/64 of the 32-bit rate here.)
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace mc {

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC > 16 ? 16 : sizeof(T) * VEC) RotVec {
  T e[VEC];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// n / d for n d < 2^32, with m = 2^32 / d rounded up (m d - 2^32 < d, so the
// quotient is off by less than n / 2^32 < 1 / d); d = 1 has m = 0 (2^32).
__device__ __forceinline__ int fast_div(int n, uint32_t m) {
  return m == 0 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), m));
}

// 1 / 2 pi = 0.28BE60DB 9391054A 7F09D5F4 7D4D3770 (hexadecimal), in words of
// 32 bits from the least significant one.
__device__ constexpr uint32_t kInvTwoPi[4] = {0x7D4D3770u, 0x7F09D5F4u, 0x9391054Au, 0x28BE60DBu};

// f / 2 pi modulo 1 as 64-bit fixed point, rounded down.
__device__ __forceinline__ uint64_t turns_fixed(float f) {
  const uint32_t bits = __float_as_uint(f);
  const int e = static_cast<int>((bits >> 23) & 255u);
  const uint32_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  // f = m 2^(max(e, 1) - 150); the product m * kInvTwoPi has 5 words and 128
  // bits behind its point
  uint32_t w[6];
  uint64_t carry = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    carry += static_cast<uint64_t>(m) * kInvTwoPi[i];
    w[i] = static_cast<uint32_t>(carry);
    carry >>= 32;
  }
  w[4] = static_cast<uint32_t>(carry);
  w[5] = 0;
  // the 64 bits from bit `at` up
  const int at = 128 - 64 - ((e ? e : 1) - 150);
  uint64_t r = 0;
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    const int sh = 32 * i - at;  // where word i lands
    const uint64_t v = w[i];
    if (sh >= 0 && sh < 64) r |= v << sh;
    if (sh < 0 && sh > -32) r |= v >> -sh;
  }
  return bits >> 31 ? 0 - r : r;
}

// sin and cos of a position times `turns` (turns_fixed of its frequency): the
// nearest 2^-32 of a turn, in half turns (24 bits of it as a float).
__device__ __forceinline__ void turn_sincos(int64_t pos, uint64_t turns, float* s, float* c) {
  const uint64_t w = static_cast<uint64_t>(pos) * turns;
  const int32_t x = static_cast<int32_t>(static_cast<uint32_t>((w + 0x80000000ull) >> 32));
  sincospif(static_cast<float>(x) * 4.656612873077393e-10f, s, c);
}

// 2^32 / d rounded up, for fast_div.
inline uint32_t fast_div_magic(int d) {
  return d == 1 ? 0u : static_cast<uint32_t>((0x100000000ull + d - 1) / d);
}

}  // namespace mc
