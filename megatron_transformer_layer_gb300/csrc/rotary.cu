// Rotary positions with several axes: pair p of every head of token t turns by
// the angle  w = positions[axis(p)][t] * inv_freq[p],
//   (u, v) -> (u cos w - v sin w, u sin w + v cos w),
// and the gradient goes back by the opposite angle (the rotation is
// orthogonal).  Bound by HBM: every element is read and written once, and an
// angle is formed once per (token, pair) and shared by all heads.
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
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mc_layer_internal.h"
#include "ptx.cuh"

namespace mc {
namespace {

// 4096 tokens of 128 heads of 128 (bf16): 51.2 us, 5.2 TB/s; with 8 warps a
// block 55.4, with items of 4 turns 54.9, of 16 50.4 (but 28.2 against 27.8 for
// the rows of rotary_plan).
constexpr int kRotWarps = 4;
constexpr int kRotTurns = 8;    // turns of an item
constexpr int kRotTable = 512;  // (token, pair) entries of a warp's cos / sin table (4 KB)

struct RotaryArgs {
  int64_t tokens, ld_in, ld_out;
  int64_t items;    // (token group, unit range) pairs, one warp each
  int heads, head_dim, pairs;
  int units;        // work units per token: the rotating ones of all heads, then the copied
  int rot_units;    // rotating units of a head
  int copy_units;   // copying units of a head
  // from a unit's first vector to its second, 0: it has one (rot_second: where
  // a vector holds whole pairs)
  int rot_second, copy_second;
  int tok_item;     // tokens of an item
  int unit_item;    // units of each of them
  int ranges;       // unit ranges per token
  int inverse;
  uint32_t div_unit_item, div_rot, div_copy, div_pairs;  // 2^32 / d rounded up (fast_div)
  uint8_t axis[kRotaryMaxPairs];
};

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

// A unit is two vectors: of VEC pairs' halves, of VEC / 2 adjacent pairs each
// (VEC > 1), or copied ones; one where a head's do not pair up. A warp takes
// items of unit_item units of each of tok_item tokens, one per lane and turn.
// The first turn's loads are issued before the item's cos / sin table is formed,
// so one DRAM round trip covers both; the turns per position of every pair are
// formed once per block. What keeps the loads coming is the number of warps: two
// units per lane and turn, or the next turn's loads ahead of this one's work,
// cost registers and were slower (60 and 64 us against 52), as was holding the
// kernel to the registers of 8 blocks per SM (54.6).
template <typename T, int VEC, bool ADJACENT>
__global__ void __launch_bounds__(kRotWarps * 32)
    rotary_kernel(const T* in, T* out, const int32_t* __restrict__ positions,
                  const float* __restrict__ inv_freq, const __grid_constant__ RotaryArgs A,
                  int* status) {
  using V = RotVec<T, VEC>;
  using F = RotVec<float, (ADJACENT && VEC > 1) ? VEC / 2 : VEC>;
  __shared__ uint64_t turns[kRotaryMaxPairs];
  __shared__ __align__(16) float table[kRotWarps][2][kRotTable];
  pdl_wait();  // the previous kernel on the stream has completed
  pdl_launch();
  for (int p = threadIdx.x; p < A.pairs; p += kRotWarps * 32) turns[p] = turns_fixed(inv_freq[p]);
  __syncthreads();
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  float* const t_cos = table[warp][0];
  float* const t_sin = table[warp][1];
  constexpr bool kSplit = !ADJACENT || VEC == 1;  // a pair's halves are in two vectors
  constexpr int kPairs = kSplit ? VEC : VEC / 2;  // pairs from a unit's first vector on
  // from a rotating unit's first vector to its second
  const int second = kSplit ? (ADJACENT ? 1 : A.pairs) : A.rot_second;
  const int rotating = A.heads * A.rot_units;     // units before the copying ones

  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kRotWarps + warp; item < A.items;
       item += static_cast<int64_t>(gridDim.x) * kRotWarps) {
    const int64_t group = item / A.ranges;
    const int64_t t0 = group * A.tok_item;
    const int ntok = static_cast<int>(min(static_cast<int64_t>(A.tok_item), A.tokens - t0));
    const int u0 = static_cast<int>(item - group * A.ranges) * A.unit_item;
    const int nu = min(A.unit_item, A.units - u0);
    const int total = ntok * nu;
    const T* const in0 = in + t0 * A.ld_in;
    T* const out0 = out + t0 * A.ld_out;
    struct Unit {
      V a, b;
      int tok, off, at;  // off < 0: nothing; at < 0: a copied vector
    };
    auto load = [&](int e) {
      Unit x;
      x.off = x.at = -1;
      x.tok = 0;
      if (e < total) {
        const int tk = nu == A.unit_item ? fast_div(e, A.div_unit_item) : e / nu;
        const int u = u0 + (e - tk * nu);
        x.tok = tk;
        const T* row = in0 + tk * A.ld_in;
        if (u < rotating) {
          const int h = fast_div(u, A.div_rot);
          const int p = (u - h * A.rot_units) * kPairs;
          x.at = tk * A.pairs + p;
          x.off = h * A.head_dim + (ADJACENT ? 2 * p : p);
          x.a = *reinterpret_cast<const V*>(row + x.off);
          if (kSplit || second) x.b = *reinterpret_cast<const V*>(row + x.off + second);
        } else {
          const int h = fast_div(u - rotating, A.div_copy);
          x.off = h * A.head_dim + 2 * A.pairs + (u - rotating - h * A.copy_units) * VEC;
          x.a = *reinterpret_cast<const V*>(row + x.off);
          if (A.copy_second) x.b = *reinterpret_cast<const V*>(row + x.off + A.copy_second);
        }
      }
      return x;
    };
    Unit cur = load(lane);
    __syncwarp();  // the table of the item before has been read
    for (int i = lane; i < ntok * A.pairs; i += 32) {
      const int tk = fast_div(i, A.div_pairs), p = i - tk * A.pairs;
      const int64_t pos = positions[A.axis[p] * A.tokens + t0 + tk];
      const uint64_t w = static_cast<uint64_t>(A.inverse ? -pos : pos) * turns[p];
      // the nearest 2^-32 of a turn, in half turns (24 bits of it as a float)
      const int32_t x = static_cast<int32_t>(static_cast<uint32_t>((w + 0x80000000ull) >> 32));
      float s, c;
      sincospif(static_cast<float>(x) * 4.656612873077393e-10f, &s, &c);
      t_cos[i] = c;
      t_sin[i] = s;
    }
    __syncwarp();
    int held = -1;  // the table place whose entries are in cs / sn
    F cs, sn;
    [[maybe_unused]] F cs2, sn2;  // of the second vector's pairs, if it has its own
    for (int e = lane; e - lane < total; e += 32) {
      T* row = out0 + cur.tok * A.ld_out;
      if (cur.off >= 0 &&
          MC_DCHECK(t0 + cur.tok < A.tokens &&
                        cur.off + (cur.at < 0 ? A.copy_second : second) + VEC <=
                            A.heads * A.head_dim,
                    status, kSiteRotary)) {
        if (cur.at >= 0) {
          if (cur.at != held) {
            held = cur.at;
            cs = *reinterpret_cast<const F*>(t_cos + held);
            sn = *reinterpret_cast<const F*>(t_sin + held);
            if (!kSplit && second) {
              cs2 = *reinterpret_cast<const F*>(t_cos + held + second / 2);
              sn2 = *reinterpret_cast<const F*>(t_sin + held + second / 2);
            }
          }
          if constexpr (kSplit) {
            V ya, yb;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
              const float u = to_f32(cur.a.e[j]), v = to_f32(cur.b.e[j]);
              ya.e[j] = from_f32<T>(u * cs.e[j] - v * sn.e[j]);
              yb.e[j] = from_f32<T>(u * sn.e[j] + v * cs.e[j]);
            }
            *reinterpret_cast<V*>(row + cur.off) = ya;
            *reinterpret_cast<V*>(row + cur.off + second) = yb;
          } else {
            auto turn = [&](const V& x, const F& c, const F& n) {
              V y;
#pragma unroll
              for (int j = 0; j < kPairs; ++j) {
                const float u = to_f32(x.e[2 * j]), v = to_f32(x.e[2 * j + 1]);
                y.e[2 * j] = from_f32<T>(u * c.e[j] - v * n.e[j]);
                y.e[2 * j + 1] = from_f32<T>(u * n.e[j] + v * c.e[j]);
              }
              return y;
            };
            *reinterpret_cast<V*>(row + cur.off) = turn(cur.a, cs, sn);
            if (second) *reinterpret_cast<V*>(row + cur.off + second) = turn(cur.b, cs2, sn2);
          }
        } else {
          *reinterpret_cast<V*>(row + cur.off) = cur.a;
          if (A.copy_second) *reinterpret_cast<V*>(row + cur.off + A.copy_second) = cur.b;
        }
      }
      cur = load(e + 32);
    }
  }
}

template <typename T, int VEC, bool ADJACENT>
int rotary_launch(const T* in, T* out, const int32_t* positions, const float* inv_freq,
                  const RotaryArgs& A, int* status, cudaStream_t st) {
  auto kern = rotary_kernel<T, VEC, ADJACENT>;
  // at most as many blocks as are resident at once
  static PerDeviceInit init;
  long long resident = 0;
  const cudaError_t e = once_per_device(init, [&](long long* value) {
    int per_sm = 0;
    const cudaError_t r =
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kRotWarps * 32, 0);
    *value = static_cast<long long>(per_sm < 1 ? 1 : per_sm) * num_sms();
    return r;
  }, &resident);
  if (e != cudaSuccess) return MC_ERR_CUDA;
  const int64_t blocks = (A.items + kRotWarps - 1) / kRotWarps;
  launch_kernel(kern, dim3(static_cast<unsigned>(blocks < resident ? blocks : resident)),
                dim3(kRotWarps * 32), 0, st, 1, in, out, positions, inv_freq, A, status);
  return cudaGetLastError() == cudaSuccess ? MC_OK : MC_ERR_CUDA;
}

template <typename T, int VEC, bool ADJACENT>
int rotary_plan(const T* in, T* out, const int32_t* positions, const float* inv_freq, RotaryArgs A,
                int* status, cudaStream_t st) {
  A.rot_units = ADJACENT && VEC > 1 ? 2 * A.pairs / VEC : A.pairs / VEC;
  A.copy_units = in != out ? (A.head_dim - 2 * A.pairs) / VEC : 0;
  // Two vectors a unit where they pair up (one each: 8191 tokens of 32 heads of
  // 128, half of it turned, adjacent pairs, 32.4 us against 27.8).
  A.rot_second = A.copy_second = 0;
  if (ADJACENT && VEC > 1 && A.rot_units % 2 == 0) {
    A.rot_units /= 2;
    A.rot_second = A.rot_units * VEC;
  }
  if (A.copy_units % 2 == 0) {
    A.copy_units /= 2;
    A.copy_second = A.copy_units * VEC;
  }
  const int64_t units =
      static_cast<int64_t>(A.heads) * (A.rot_units + A.copy_units);  // <= 2^22
  A.units = static_cast<int>(units);
  // Units of an item: enough that forming its table does not show, or one turn
  // where the call is too short to fill the SMs otherwise.
  const bool small = units * A.tokens <= 1024ll * num_sms();
  const int item_units = small ? 32 : 32 * kRotTurns;
  A.unit_item = A.units < item_units ? A.units : item_units;
  int tk = item_units / A.unit_item;
  if (tk > kRotTable / A.pairs) tk = kRotTable / A.pairs;
  if (tk > A.tokens) tk = static_cast<int>(A.tokens);
  A.tok_item = tk;
  A.ranges = (A.units + A.unit_item - 1) / A.unit_item;
  A.items = (A.tokens + tk - 1) / tk * A.ranges;
  auto magic = [](int d) { return d == 1 ? 0u : static_cast<uint32_t>((0x100000000ull + d - 1) / d); };
  A.div_unit_item = magic(A.unit_item);
  A.div_rot = magic(A.rot_units);
  A.div_copy = magic(A.copy_units > 0 ? A.copy_units : 1);
  A.div_pairs = magic(A.pairs);
  return rotary_launch<T, VEC, ADJACENT>(in, out, positions, inv_freq, A, status, st);
}

template <typename T>
int rotary_typed(const void* in_, void* out_, const int32_t* positions, const float* inv_freq,
                 const RotaryArgs& A, bool adjacent, int* status, cudaStream_t st) {
  const T* in = static_cast<const T*>(in_);
  T* out = static_cast<T*>(out_);
  constexpr int kFull = 16 / sizeof(T);
  // The widest vector that pairs, copied dimensions, heads, rows and both
  // addresses are whole multiples of.
  auto fits = [&](int vec) {
    const uintptr_t bytes = sizeof(T) * static_cast<uintptr_t>(vec);
    return (adjacent ? 2 * A.pairs : A.pairs) % vec == 0 && A.head_dim % vec == 0 && A.ld_in % vec == 0 &&
           A.ld_out % vec == 0 && reinterpret_cast<uintptr_t>(in) % bytes == 0 &&
           reinterpret_cast<uintptr_t>(out) % bytes == 0;
  };
  const int vec = fits(kFull) ? kFull : (fits(2) ? 2 : 1);
  if (vec == kFull)
    return adjacent ? rotary_plan<T, kFull, true>(in, out, positions, inv_freq, A, status, st)
                    : rotary_plan<T, kFull, false>(in, out, positions, inv_freq, A, status, st);
  if (vec == 2)
    return adjacent ? rotary_plan<T, 2, true>(in, out, positions, inv_freq, A, status, st)
                    : rotary_plan<T, 2, false>(in, out, positions, inv_freq, A, status, st);
  return adjacent ? rotary_plan<T, 1, true>(in, out, positions, inv_freq, A, status, st)
                  : rotary_plan<T, 1, false>(in, out, positions, inv_freq, A, status, st);
}

}  // namespace

int check_rotary_spec(const mc_rotary_spec* spec, int head_dim) {
  if (!spec) return MC_ERR_NULLPTR;
  if (head_dim < 2 || spec->rot_dim < 2 || spec->rot_dim % 2 || spec->rot_dim > head_dim)
    return MC_ERR_SHAPE;
  if (spec->axes < 1 || spec->axes > MC_ROTARY_MAX_AXES) return MC_ERR_ARGUMENT;
  if (spec->flags & ~(MC_ROTARY_ADJACENT_PAIRS | MC_ROTARY_DEAL_AXES)) return MC_ERR_ARGUMENT;
  if (spec->rot_dim / 2 > kRotaryMaxPairs) return MC_ERR_UNSUPPORTED;
  int64_t sum = 0;
  for (int x = 0; x < spec->axes; ++x) {
    if (spec->sections[x] < 0) return MC_ERR_SHAPE;
    sum += spec->sections[x];
  }
  return sum == spec->rot_dim / 2 ? MC_OK : MC_ERR_SHAPE;
}

int launch_rotary(const void* in, void* out, bool bf16, int64_t tokens, int heads, int head_dim,
                  int64_t ld_in, int64_t ld_out, const int32_t* positions, const float* inv_freq,
                  const mc_rotary_spec* spec, bool inverse, int* status, cudaStream_t st) {
  const int rc = check_rotary_spec(spec, head_dim);
  if (rc != MC_OK) return rc;
  if (tokens < 1 || heads < 1) return MC_ERR_SHAPE;
  const int64_t width = static_cast<int64_t>(heads) * head_dim;
  // fast_div: fewer than 2^22 units, at most 2^10 of them of one head
  if (width > (1 << 22) || head_dim > 1024) return MC_ERR_UNSUPPORTED;
  if (ld_in < width || ld_out < width) return MC_ERR_SHAPE;
  if (!in || !out || !positions || !inv_freq) return MC_ERR_NULLPTR;
  const uintptr_t size = bf16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(in) % size || reinterpret_cast<uintptr_t>(out) % size ||
      reinterpret_cast<uintptr_t>(positions) % 4 || reinterpret_cast<uintptr_t>(inv_freq) % 4)
    return MC_ERR_ALIGN;
  if (in == out && ld_in != ld_out) return MC_ERR_ARGUMENT;
  RotaryArgs A = {};
  A.tokens = tokens;
  A.ld_in = ld_in;
  A.ld_out = ld_out;
  A.heads = heads;
  A.head_dim = head_dim;
  A.pairs = spec->rot_dim / 2;
  A.inverse = inverse ? 1 : 0;
  rotary_axes(spec, A.axis);
  const bool adjacent = (spec->flags & MC_ROTARY_ADJACENT_PAIRS) != 0;
  return bf16 ? rotary_typed<__nv_bfloat16>(in, out, positions, inv_freq, A, adjacent, status, st)
              : rotary_typed<float>(in, out, positions, inv_freq, A, adjacent, status, st);
}

// The axis of each pair: section after section, or (MC_ROTARY_DEAL_AXES) dealt
// in turn, an axis leaving the round when its section is used up.
void rotary_axes(const mc_rotary_spec* spec, uint8_t* axis) {
  int left[MC_ROTARY_MAX_AXES] = {};
  for (int x = 0; x < spec->axes; ++x) left[x] = spec->sections[x];
  const int pairs = spec->rot_dim / 2;
  int p = 0;
  if (spec->flags & MC_ROTARY_DEAL_AXES) {
    while (p < pairs)
      for (int x = 0; x < spec->axes && p < pairs; ++x)
        if (left[x] > 0) {
          axis[p++] = static_cast<uint8_t>(x);
          --left[x];
        }
  } else {
    for (int x = 0; x < spec->axes; ++x)
      for (int i = 0; i < left[x] && p < pairs; ++i) axis[p++] = static_cast<uint8_t>(x);
  }
}

}  // namespace mc

extern "C" {

int mc_rotary_forward(const void* in, void* out, int32_t is_bf16, int64_t tokens, int32_t heads,
                      int32_t head_dim, int64_t ld_in, int64_t ld_out, const int32_t* positions,
                      const float* inv_freq, const mc_rotary_spec* spec, int* status,
                      void* stream) {
  return mc::launch_rotary(in, out, is_bf16 != 0, tokens, heads, head_dim, ld_in, ld_out,
                           positions, inv_freq, spec, false, status,
                           static_cast<cudaStream_t>(stream));
}

int mc_rotary_backward(const void* dout, void* din, int32_t is_bf16, int64_t tokens,
                       int32_t heads, int32_t head_dim, int64_t ld_out, int64_t ld_in,
                       const int32_t* positions, const float* inv_freq,
                       const mc_rotary_spec* spec, int* status, void* stream) {
  return mc::launch_rotary(dout, din, is_bf16 != 0, tokens, heads, head_dim, ld_out, ld_in,
                           positions, inv_freq, spec, true, status,
                           static_cast<cudaStream_t>(stream));
}

}  // extern "C"
