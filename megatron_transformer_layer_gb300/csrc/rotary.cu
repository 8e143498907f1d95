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
// an error of 2^-33 turns; sincospif gets 32 bits of the turn.  (The same in
// 64-bit floats is exact enough too, but they run at 1/64 of the 32-bit rate
// here.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mc_layer_internal.h"
#include "ptx.cuh"

namespace mc {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotMaxTable = 4096;  // (token, pair) entries of a block's cos / sin table (32 KB)
constexpr int kRotMaxTokens = 32;   // tokens of a block

struct RotaryArgs {
  int64_t tokens, ld_in, ld_out;
  int heads, head_dim, pairs;
  uint32_t div_nu, div_units_head, div_pairs;  // 2^32 / d rounded up, for divisions (fast_div)
  int units;        // work units per token: heads * units_head
  int units_head;   // pairs / VEC rotating units, then the vectors that are copied
  int tok_block;    // tokens per block
  int unit_block;   // units of each of them per block
  int inverse;
  int copy_rest;    // out of place: the unrotated dimensions are copied
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

// A unit is VEC pairs of one head (two vectors of VEC elements: the halves of
// the pairs, or 2 VEC adjacent elements) or one copied vector.  A block takes
// unit_block units of each of tok_block tokens, up to UPT per thread; their
// loads are issued before the cos / sin table is formed, so one DRAM round
// trip covers both.
template <typename T, int VEC, bool ADJACENT, int UPT>
__global__ void __launch_bounds__(kRotThreads, UPT > 1 ? 3 : 4)
    rotary_kernel(const T* in, T* out, const int32_t* __restrict__ positions,
                  const float* __restrict__ inv_freq, const __grid_constant__ RotaryArgs A,
                  int* status) {
  using V = RotVec<T, VEC>;
  // cos and sin, [tok_block][pairs] each
  extern __shared__ __align__(16) float table[];
  float* const t_cos = table;
  float* const t_sin = table + A.tok_block * A.pairs;
  pdl_wait();  // the previous kernel on the stream has completed
  pdl_launch();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * A.tok_block;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(A.tok_block), A.tokens - t0));
  const int u0 = static_cast<int>(blockIdx.y) * A.unit_block;
  const int nu = min(A.unit_block, A.units - u0);
  const int total = ntok * nu;
  const int rot_units = A.pairs / VEC;

  V a[UPT], b[UPT];
  int tok[UPT], pair[UPT];  // pair < 0: nothing, or a copied vector
  int off[UPT];             // of the unit's first vector within its row
#pragma unroll
  for (int k = 0; k < UPT; ++k) {
    const int e = static_cast<int>(threadIdx.x) + k * kRotThreads;
    pair[k] = -1;
    off[k] = -1;
    tok[k] = 0;
    if (e < total) {
      const int tk = nu == A.unit_block ? fast_div(e, A.div_nu) : e / nu;
      const int u = u0 + (e - tk * nu);
      const int h = fast_div(u, A.div_units_head);
      const int w = u - h * A.units_head;
      tok[k] = tk;
      const T* row = in + (t0 + tk) * A.ld_in;
      const int base = h * A.head_dim;
      if (w < rot_units) {
        pair[k] = w * VEC;
        off[k] = base + (ADJACENT ? 2 * w * VEC : w * VEC);
        a[k] = *reinterpret_cast<const V*>(row + off[k]);
        b[k] = *reinterpret_cast<const V*>(row + off[k] + (ADJACENT ? VEC : A.pairs));
      } else if (A.copy_rest) {
        off[k] = base + 2 * A.pairs + (w - rot_units) * VEC;
        a[k] = *reinterpret_cast<const V*>(row + off[k]);
      }
    }
  }

  for (int i = threadIdx.x; i < ntok * A.pairs; i += kRotThreads) {
    const int tk = fast_div(i, A.div_pairs), p = i - tk * A.pairs;
    const uint64_t f = turns_fixed(inv_freq[p]);
    const int64_t pos = positions[A.axis[p] * A.tokens + t0 + tk];
    const uint64_t w = static_cast<uint64_t>(A.inverse ? -pos : pos) * f;
    const float x = static_cast<float>(static_cast<int32_t>(static_cast<uint32_t>((w + 0x80000000ull) >> 32)));
    float s, c;
    sincospif(x * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    t_cos[i] = c;
    t_sin[i] = s;
  }
  __syncthreads();

  int held = -1;  // the table place whose VEC entries are in cs / sn
  RotVec<float, VEC> cs, sn;
#pragma unroll
  for (int k = 0; k < UPT; ++k) {
    if (off[k] < 0) continue;
    T* row = out + (t0 + tok[k]) * A.ld_out;
    const int rest = pair[k] >= 0 ? (ADJACENT ? VEC : A.pairs) : 0;
    if (!MC_DCHECK(t0 + tok[k] < A.tokens &&
                       off[k] + rest + VEC <= A.heads * A.head_dim,
                   status, kSiteRotary))
      continue;
    if (pair[k] >= 0) {
      const int at = tok[k] * A.pairs + pair[k];
      if (at != held) {
        held = at;
        cs = *reinterpret_cast<const RotVec<float, VEC>*>(t_cos + at);
        sn = *reinterpret_cast<const RotVec<float, VEC>*>(t_sin + at);
      }
      V ya, yb;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float2 r = make_float2(cs.e[j], sn.e[j]);
        float u, v;
        if constexpr (ADJACENT) {  // pair j: elements 2j, 2j + 1 of a | b
          u = to_f32(2 * j < VEC ? a[k].e[(2 * j) % VEC] : b[k].e[(2 * j) % VEC]);
          v = to_f32(2 * j + 1 < VEC ? a[k].e[(2 * j + 1) % VEC] : b[k].e[(2 * j + 1) % VEC]);
        } else {
          u = to_f32(a[k].e[j]);
          v = to_f32(b[k].e[j]);
        }
        const T nu_ = from_f32<T>(u * r.x - v * r.y), nv_ = from_f32<T>(u * r.y + v * r.x);
        if constexpr (ADJACENT) {
          if (2 * j < VEC) ya.e[(2 * j) % VEC] = nu_; else yb.e[(2 * j) % VEC] = nu_;
          if (2 * j + 1 < VEC) ya.e[(2 * j + 1) % VEC] = nv_; else yb.e[(2 * j + 1) % VEC] = nv_;
        } else {
          ya.e[j] = nu_;
          yb.e[j] = nv_;
        }
      }
      *reinterpret_cast<V*>(row + off[k]) = ya;
      *reinterpret_cast<V*>(row + off[k] + rest) = yb;
    } else {
      *reinterpret_cast<V*>(row + off[k]) = a[k];
    }
  }
}

template <typename T, int VEC, bool ADJACENT, int UPT>
int rotary_launch(const T* in, T* out, const int32_t* positions, const float* inv_freq,
                  const RotaryArgs& A, int64_t gx, int64_t gy, int* status, cudaStream_t st) {
  launch_kernel(rotary_kernel<T, VEC, ADJACENT, UPT>,
                dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), dim3(kRotThreads),
                2 * sizeof(float) * A.tok_block * A.pairs, st, 1, in, out, positions, inv_freq, A,
                status);
  return cudaGetLastError() == cudaSuccess ? MC_OK : MC_ERR_CUDA;
}

template <typename T, int VEC, bool ADJACENT>
int rotary_plan(const T* in, T* out, const int32_t* positions, const float* inv_freq, RotaryArgs A,
                int* status, cudaStream_t st) {
  const int rest = A.copy_rest ? (A.head_dim - 2 * A.pairs) / VEC : 0;
  A.units_head = A.pairs / VEC + rest;
  const int64_t units = static_cast<int64_t>(A.heads) * A.units_head;  // <= 2^22
  A.units = static_cast<int>(units);
  // Four units per thread keep enough loads in flight; few units in all take
  // one per thread, so that more SMs share the call.
  const bool small = units * A.tokens <= 4ll * kRotThreads * num_sms();
  const int block_units = small ? kRotThreads : 4 * kRotThreads;
  A.unit_block = A.units < block_units ? A.units : block_units;
  int tb = block_units / A.unit_block;
  if (tb > kRotMaxTokens) tb = kRotMaxTokens;
  if (tb > kRotMaxTable / A.pairs) tb = kRotMaxTable / A.pairs;
  if (tb > A.tokens) tb = static_cast<int>(A.tokens);
  A.tok_block = tb;
  auto magic = [](int d) { return d == 1 ? 0u : static_cast<uint32_t>((0x100000000ull + d - 1) / d); };
  A.div_nu = magic(A.unit_block);
  A.div_units_head = magic(A.units_head);
  A.div_pairs = magic(A.pairs);
  const int64_t gx = (A.tokens + tb - 1) / tb;
  const int64_t gy = (A.units + A.unit_block - 1) / A.unit_block;
  if (gx > 0x7fffffff) return MC_ERR_UNSUPPORTED;
  return small ? rotary_launch<T, VEC, ADJACENT, 1>(in, out, positions, inv_freq, A, gx, gy, status, st)
               : rotary_launch<T, VEC, ADJACENT, 4>(in, out, positions, inv_freq, A, gx, gy, status, st);
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
    return A.pairs % vec == 0 && A.head_dim % vec == 0 && A.ld_in % vec == 0 &&
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
  // (2^22 units of at most 512 per head: within fast_div)
  if (width > (1 << 22)) return MC_ERR_UNSUPPORTED;
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
  A.copy_rest = in != out ? 1 : 0;
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
