// Norms of queries and keys, head by head, with the rotary positions in the
// same pass.  A head x of d elements, with its gain g and shift c:
//   m = mean(x) (centred) or 0,  r = 1 / sqrt(mean((x - m)^2) + eps),
//   n = (x - m) r,  out = R(w) (n g + c)
// and back, with t = R(-w) dout and u = t g:
//   dx = r (u - n mean(u n) - mean(u)) (the last mean only if centred),
//   dg = sum of t n and dc = sum of t over tokens and heads.
// Bound by HBM: forward every element is read and written once, backward x and
// dout are read and dx is written; n is formed from x again, so that nothing
// is kept between the passes.  All sums are 32-bit, results are rounded once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "mc_layer_internal.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace mc {
namespace {

constexpr int kNormTable = 224;  // (token, pair) entries of a warp's cos / sin table
constexpr int kNormMaxDim = 256;
constexpr int kNormWords = kNormMaxDim / 2 + 8;  // of gains or shifts, two elements each
constexpr int kNormMaxBlocks = 512;  // of the backward pass: rows of partial sums
// A chunk of a warp's work is this many turns of its lanes, 1 KB of each input a
// turn, and so many chunks are on their way.
constexpr int kNormTurnBytes = 1024;
template <bool BACK>
struct NormCfg {
  // (the backward pass takes 168 registers a thread: 12 warps per SM)
  static constexpr int kWarps = BACK ? 12 : 8, kBlocks = BACK ? 1 : 2;
  // (4 turns, forward: 8191 tokens of 40 heads of 128 take 54 us against 50, one 58)
  static constexpr int kTurns = 2;
  static constexpr int kInputs = BACK ? 2 : 1;
  static constexpr int kStages = 3;
  static constexpr int kStage = kTurns * kInputs * kNormTurnBytes;
  static constexpr int kWarp = kStages * kStage + 2 * kNormTable * 4;
  static constexpr int kSmem = kWarps * (kWarp + kStages * 8) + kNormMaxDim / 2 * 8 +
                               2 * kNormWords * 4 + kNormMaxDim / 2;
  static_assert(kBlocks * (kSmem + 1024) <= 228 * 1024, "blocks per SM");
  static_assert(kStages * kStage >= 2 * kNormMaxDim * 4, "a warp's sums go through its ring");
  static_assert(kWarps * kStages % 2 == 0, "the gains behind the barriers are read 16 bytes at a time");
};

// Queries (0) and keys (1) are walked apart, each by blocks of its own, so that
// a lane's gains, shifts and gradient sums stay in registers.
struct NormType {
  const uint16_t* gain;   // bf16 [d], or NULL: ones
  const uint16_t* shift;  // or NULL: zeros
  float* dgain;           // or NULL
  float* dshift;
  int64_t chunks;      // (token group, head range) pairs, shared out to the warps in runs:
  int64_t per_warp, more;  // so many each, the first `more` of them one more
  int head0, heads;    // of the row's heads
  int tok_chunk, head_chunk, ranges;  // a chunk: tokens, heads of each; ranges per token group
  int block0, blocks;
  uint32_t div_head_chunk;
};

struct NormArgs {
  NormType type[2];
  int64_t tokens, ld_in, ld_dout, ld_out;
  int d, pairs, axes;
  int lanes, log_lanes, units;  // lanes of a head (a power of two) and its units
  int centred, inverse, accumulate;
  float eps;
  uint32_t div_pairs;
  float* partials;  // backward: [block][2][d]
  uint8_t axis[kRotaryMaxPairs];
};

// Elements in 32 bits, two at a time where a vector has an even number of them.
template <int VEC>
struct Two {
  using P = float2;
};
template <>
struct Two<1> {
  using P = float;
};
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float sum(float2 a) { return a.x + a.y; }
__device__ __forceinline__ float2 swap(float2 a) { return make_float2(a.y, a.x); }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float sum(float a) { return a; }
__device__ __forceinline__ float swap(float a) { return a; }
template <typename P>
__device__ __forceinline__ P both(float x);
template <>
__device__ __forceinline__ float2 both<float2>(float x) { return make_float2(x, x); }
template <>
__device__ __forceinline__ float both<float>(float x) { return x; }
__device__ __forceinline__ float& at(float2& p, int i) { return i ? p.y : p.x; }
__device__ __forceinline__ float& at(float& p, int) { return p; }

template <typename T, int VEC, typename P>
__device__ __forceinline__ void unpack(const RotVec<T, VEC>& v, P* f) {
  if constexpr (VEC == 1) {
    f[0] = to_f32(v.e[0]);
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) f[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) f[i] = make_float2(v.e[2 * i], v.e[2 * i + 1]);
  }
}
template <typename T, int VEC, typename P>
__device__ __forceinline__ RotVec<T, VEC> pack(const P* f) {
  RotVec<T, VEC> v;
  if constexpr (VEC == 1) {
    v.e[0] = from_f32<T>(f[0]);
  } else if constexpr (sizeof(T) == 2) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) w[i] = pack_bf16x2(f[i].x, f[i].y);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) v.e[2 * i] = f[i].x, v.e[2 * i + 1] = f[i].y;
  }
  return v;
}

// A unit is two vectors: the halves of VEC pairs, or of adjacent pairs and of
// what does not turn two neighbouring ones (the second may be missing).  `lanes`
// lanes hold a head, one unit (or N, for narrow vectors) each, and a lane has
// the same unit of every head it meets: its gains are loaded once, its cosines
// once per token.  Of a warp's turn the lanes hold 32 / lanes heads, of the same
// token or of the next ones.
//
// A warp's chunks are one run of the rows.  With vectors of 16 bytes they come
// by bulk copies into a ring of its own, so that the loads on their way do not
// depend on registers; with narrower ones (odd sizes or addresses) the lanes
// load them.
//
// Measured (bf16): 4096 tokens of 128 heads of 128, 46.7 us = 5.7 TB/s, 0.85 of a copy's
// rate, at 240 instructions a turn of a warp; 8191 tokens of 40 such heads, centred, half
// of a head turned in adjacent pairs, 50.4 us = 3.3 TB/s at 330: a warp has some 35 turns
// there, each a chain of two sums over the lanes, four warps to a scheduler, which
// issues 42% of the time.  Two turns side by side in a warp were slower (57 against 53 us:
// more registers), more warps of fewer registers too (60).  Backward 86 us = 4.7 TB/s for
// the first shape; 18 us for 2036 tokens of 24 heads of 64, of which the sums of the
// gradients over blocks take 7.  fp32, the first shape: 99 us = 5.4 TB/s, backward 137 =
// 5.9.  Vectors of two elements or one (no ring, each load waited for): bf16 164 and 241
// us, fp32 172 and 249, backward bf16 340 and 388.
template <typename T, int VEC, bool ADJACENT, bool BACK, bool SHIFT>
__global__ void __launch_bounds__(NormCfg<BACK>::kWarps * 32, NormCfg<BACK>::kBlocks)
    qk_norm_kernel(const T* in, const T* dout, T* out, const int32_t* __restrict__ positions,
                   const float* __restrict__ inv_freq, const __grid_constant__ NormArgs A,
                   int* status) {
  using V = RotVec<T, VEC>;
  using P = typename Two<VEC>::P;
  using C = NormCfg<BACK>;
  constexpr int W = VEC > 1 ? VEC / 2 : 1, E = VEC > 1 ? 2 : 1;  // VEC = W E
  constexpr bool kBulk = VEC * sizeof(T) == 16;
  constexpr bool kSplit = !ADJACENT || VEC == 1;  // a pair's halves are in two vectors
  constexpr int N = kBulk ? 1 : (VEC == 2 ? 2 : 4);
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  uint8_t* const ring = smem + warp * C::kWarp;
  float* const t_cos = reinterpret_cast<float*>(ring + C::kStages * C::kStage);
  float* const t_sin = t_cos + kNormTable;
  uint64_t* const turns = reinterpret_cast<uint64_t*>(smem + C::kWarps * C::kWarp);
  uint64_t* const full = turns + kNormMaxDim / 2 + warp * C::kStages;
  if (kBulk && lane == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  pdl_wait();  // the previous kernel on the stream has completed
  pdl_launch();
  const NormType& Y = A.type[static_cast<int>(blockIdx.x) >= A.type[1].block0 ? 1 : 0];
  const int d = A.d, L = A.lanes;
  const int seg = lane >> A.log_lanes, per_turn = 32 >> A.log_lanes;
  const float inv_d = 1.f / static_cast<float>(d);

  // this warp's run of chunks
  const int me = (static_cast<int>(blockIdx.x) - Y.block0) * C::kWarps + warp;
  const int64_t c_begin = me * Y.per_warp + min(static_cast<int64_t>(me), Y.more);
  const int64_t c_end = c_begin + Y.per_warp + (me < Y.more ? 1 : 0);
  struct Chunk {
    int64_t t0;
    int h0, ntok, nh;
  };
  auto bound = [&](Chunk& x) {
    x.ntok = static_cast<int>(min(static_cast<int64_t>(Y.tok_chunk), A.tokens - x.t0));
    x.nh = min(Y.head_chunk, Y.heads - x.h0);
  };
  auto advance = [&](Chunk& x) {
    x.h0 += Y.head_chunk;
    if (x.h0 >= Y.heads) x.h0 = 0, x.t0 += Y.tok_chunk;
    bound(x);
  };
  Chunk x;
  int64_t group;
  if (c_begin >> 31 == 0)  // (a 64-bit division takes half a microsecond)
    group = static_cast<uint32_t>(c_begin) / static_cast<uint32_t>(Y.ranges);
  else
    group = c_begin / Y.ranges;
  x.t0 = group * Y.tok_chunk;
  x.h0 = static_cast<int>(c_begin - group * Y.ranges) * Y.head_chunk;
  bound(x);
  [[maybe_unused]] Chunk ahead = x;  // the next one to load
  // A row's heads of the next chunk into stage st, a copy per token and input.
  auto issue = [&](int st) {
    const uint32_t bytes = static_cast<uint32_t>(ahead.nh * d * static_cast<int>(sizeof(T)));
    if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes * ahead.ntok * C::kInputs);
    __syncwarp();
    for (int tk = lane; tk < ahead.ntok; tk += 32) {
      uint8_t* dst = ring + st * C::kStage + tk * bytes;
      const int64_t col = static_cast<int64_t>(Y.head0 + ahead.h0) * d;
      bulk_load(dst, in + (ahead.t0 + tk) * A.ld_in + col, bytes, &full[st]);
      if constexpr (BACK)
        bulk_load(dst + C::kTurns * kNormTurnBytes, dout + (ahead.t0 + tk) * A.ld_dout + col, bytes,
                  &full[st]);
    }
    advance(ahead);
  };
  if constexpr (kBulk) {
    __syncwarp();
    for (int i = 0; i < C::kStages; ++i)
      if (c_begin + i < c_end) issue(i);
  }
  // The positions of a group's tokens (axis by axis, 32 at most: a lane each) are
  // loaded a group ahead.
  const int my_axis = lane / Y.tok_chunk, my_tok = lane - my_axis * Y.tok_chunk;
  auto positions_of = [&](int64_t t0) -> int32_t {
    return A.pairs > 0 && my_axis < A.axes && t0 + my_tok < A.tokens
               ? positions[my_axis * A.tokens + t0 + my_tok]
               : 0;
  };
  int32_t pos_next = c_begin < c_end ? positions_of(x.t0) : 0;
  uint32_t* const words = reinterpret_cast<uint32_t*>(turns + kNormMaxDim / 2 + C::kWarps * C::kStages);
  uint8_t* const axis = reinterpret_cast<uint8_t*>(words + 2 * kNormWords);
  for (int p = threadIdx.x; p < A.pairs; p += C::kWarps * 32) {
    turns[p] = turns_fixed(inv_freq[p]);
    axis[p] = A.axis[p];
  }

  // this lane's units: first dimensions of the two vectors (-1: none) and the
  // first pair of each (of both, where the vectors are halves; -1: does not turn)
  int oa[N], ob[N], pa[N], pb[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int u = (lane & (L - 1)) + j * L;
    oa[j] = ob[j] = pa[j] = pb[j] = -1;
    if (u < A.units) {
      if (kSplit && u * VEC < A.pairs) {
        oa[j] = ADJACENT ? 2 * u : u * VEC;
        ob[j] = ADJACENT ? 2 * u + 1 : A.pairs + u * VEC;
        pa[j] = u * VEC;
      } else {
        oa[j] = kSplit ? 2 * A.pairs + 2 * (u * VEC - A.pairs) : 2 * u * VEC;
        ob[j] = oa[j] + VEC < d ? oa[j] + VEC : -1;
        if (!kSplit) {
          if (oa[j] < 2 * A.pairs) pa[j] = oa[j] / 2;
          if (ob[j] >= 0 && ob[j] < 2 * A.pairs) pb[j] = ob[j] / 2;
        }
      }
    }
  }
  // Gains and shifts, bf16, unit by unit in shared memory: the first vector's
  // element in the low half of a word, the second's above.  (Forward, they are
  // read once per token, into its factors.)
  if (warp == C::kWarps - 1 && seg == 0) {
    const uint32_t one = 0x3F80u;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int w = (lane + j * L) * VEC + i;
        if (oa[j] < 0) continue;
        const uint32_t lo = Y.gain ? Y.gain[oa[j] + i] : one;
        const uint32_t hi = Y.gain && ob[j] >= 0 ? Y.gain[ob[j] + i] : one;
        words[w] = lo | (hi << 16);
        const uint32_t slo = !BACK && Y.shift ? Y.shift[oa[j] + i] : 0u;
        const uint32_t shi = !BACK && Y.shift && ob[j] >= 0 ? Y.shift[ob[j] + i] : 0u;
        words[kNormWords + w] = slo | (shi << 16);
      }
  }
  __syncthreads();  // `turns`, `axis` and `words`
  using Words = RotVec<uint32_t, VEC>;
  auto load_words = [&](int part, int j) -> Words {
    Words w = {};
    if (oa[j] >= 0)
      w = *reinterpret_cast<const Words*>(words + part * kNormWords + ((lane & (L - 1)) + j * L) * VEC);
    return w;
  };
  // (the backward pass needs the gains at every head)
  uint32_t gain[BACK ? N : 1][VEC];
  if constexpr (BACK) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const Words w = load_words(0, j);
#pragma unroll
      for (int i = 0; i < VEC; ++i) gain[j][i] = w.e[i];
    }
  }
  // backward: this lane's sums of t n and t
  P sga[BACK ? N : 1][W] = {}, sgb[BACK ? N : 1][W] = {};
  P sca[BACK && SHIFT ? N : 1][W] = {}, scb[BACK && SHIFT ? N : 1][W] = {};
  // What a token's angles make of a head, by element: own factor, partner's
  // factor, and a constant:  y = r (x f + partner(x) h) + k, gains and shifts in
  // them (forward), t = dout f + partner(dout) h (backward).
  P fa[N][W], fb[N][W], ha[N][W], hb[N][W];
  P ka[!BACK && SHIFT ? N : 1][W], kb[!BACK && SHIFT ? N : 1][W];
  auto factors = [&](int j, const float (&cs)[VEC], const float (&sn)[VEC]) {
    [[maybe_unused]] Words wg, wc;
    if constexpr (!BACK) wg = load_words(0, j);
    if constexpr (!BACK && SHIFT) wc = load_words(1, j);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      // the angle of element i of a and of b, and its place in the pair
      const int ia = kSplit ? i : i / 2, ib = kSplit ? i : VEC / 2 + i / 2;
      const float sa = kSplit || i % 2 == 0 ? -sn[ia] : sn[ia];
      const float sb = kSplit || i % 2 == 1 ? sn[ib] : -sn[ib];
      float &f0 = at(fa[j][i / E], i % E), &f1 = at(fb[j][i / E], i % E);
      float &h0 = at(ha[j][i / E], i % E), &h1 = at(hb[j][i / E], i % E);
      if constexpr (BACK) {
        f0 = cs[ia], h0 = sa, f1 = cs[ib], h1 = sb;
      } else {
        // the partners' gains and shifts
        const int o = kSplit || VEC == 1 ? i : i ^ 1;
        const uint32_t g = wg.e[i], go = wg.e[o];
        f0 = bf16_lo(g) * cs[ia];
        h0 = (kSplit ? bf16_hi(g) : bf16_lo(go)) * sa;
        f1 = bf16_hi(g) * cs[ib];
        h1 = (kSplit ? bf16_lo(g) : bf16_hi(go)) * sb;
        if constexpr (SHIFT) {
          const uint32_t c = wc.e[i], co = wc.e[o];
          at(ka[j][i / E], i % E) = bf16_lo(c) * cs[ia] + (kSplit ? bf16_hi(c) : bf16_lo(co)) * sa;
          at(kb[j][i / E], i % E) = bf16_hi(c) * cs[ib] + (kSplit ? bf16_lo(c) : bf16_hi(co)) * sb;
        }
      }
    }
  };
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float cs[VEC], sn[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) cs[i] = 1.f, sn[i] = 0.f;
    factors(j, cs, sn);
  }

  // sums over the lanes of a head
  auto over_lanes = [&](auto&& step) {
    switch (A.log_lanes) {  // (the usual sizes without a loop)
      case 2: step(2), step(1); break;
      case 3: step(4), step(2), step(1); break;
      case 4: step(8), step(4), step(2), step(1); break;
      default:
        for (int o = L >> 1; o > 0; o >>= 1) step(o);
    }
  };
  auto head_sum = [&](float& a) {
    over_lanes([&](int o) { a += __shfl_xor_sync(0xffffffffu, a, o); });
  };
  auto head_sum2 = [&](float& a, float& b) {
    over_lanes([&](int o) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    });
  };
  // x f + partner(x) h of both vectors
  auto turn = [&](int j, P (&a)[W], P (&b)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const P u = a[i], v = b[i];
      a[i] = fma(u, fa[j][i], mul(kSplit ? v : swap(u), ha[j][i]));
      b[i] = fma(v, fb[j][i], mul(kSplit ? u : swap(v), hb[j][i]));
    }
  };

  int64_t tabled = -1;  // the token group whose angles are in the table
  int held = -1;        // and the token of it in cs, sn
  int n = 0;            // chunks done
  for (int64_t c = c_begin; c < c_end; ++c, ++n, advance(x)) {
    const int st = n % C::kStages;
    if (A.pairs > 0 && x.t0 != tabled) {
      tabled = x.t0;
      held = -1;
      const int32_t pos_now = pos_next;
      pos_next = positions_of(x.t0 + Y.tok_chunk);
      __syncwarp();  // the table of the group before has been read
      for (int i0 = 0; i0 < x.ntok * A.pairs; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < x.ntok * A.pairs;
        const int tk = in ? fast_div(i, A.div_pairs) : 0, p = in ? i - tk * A.pairs : 0;
        const int64_t pos = __shfl_sync(0xffffffffu, pos_now, axis[p] * Y.tok_chunk + tk);
        if (in) turn_sincos(A.inverse ? -pos : pos, turns[p], t_sin + i, t_cos + i);
      }
      __syncwarp();
    }
    if constexpr (kBulk) {
      if (!mbar_wait_warp(&full[st], (n / C::kStages) & 1, status, kSiteQkNorm)) break;
    }
    const int total = x.ntok * x.nh;
#pragma unroll 1
    for (int e0 = 0; e0 < total; e0 += per_turn) {
      // (token, head) e of the chunk: this lane's, or none
      const bool live = e0 + seg < total;
      const int e = live ? e0 + seg : 0;
      int tok = 0, head = e;
      if (x.ntok > 1) {
        tok = x.nh == Y.head_chunk ? fast_div(e, Y.div_head_chunk) : e / x.nh;
        head = e - tok * x.nh;
      }
      // (Lanes without a vector or a head load some other one: what they make of it
      // enters no sum and is not stored.)
      const int64_t col = static_cast<int64_t>(Y.head0 + x.h0 + head) * d;
      const T* row;
      [[maybe_unused]] const T* drow = nullptr;
      if constexpr (kBulk) {
        row = reinterpret_cast<const T*>(ring + st * C::kStage) + e * d;
        if constexpr (BACK) drow = row + C::kTurns * kNormTurnBytes / static_cast<int>(sizeof(T));
      } else {
        row = in + (x.t0 + tok) * A.ld_in + col;
        if constexpr (BACK) drow = dout + (x.t0 + tok) * A.ld_dout + col;
      }
      P a[N][W], b[N][W];
      [[maybe_unused]] P ta[N][W], tb[N][W];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int la = max(oa[j], 0), lb = max(ob[j], 0);
        unpack<T, VEC>(*reinterpret_cast<const V*>(row + la), a[j]);
        unpack<T, VEC>(*reinterpret_cast<const V*>(row + lb), b[j]);
        if constexpr (BACK) {
          unpack<T, VEC>(*reinterpret_cast<const V*>(drow + la), ta[j]);
          unpack<T, VEC>(*reinterpret_cast<const V*>(drow + lb), tb[j]);
        }
      }
      if (A.pairs > 0 && live && tok != held) {
        held = tok;
        const float* c0 = t_cos + held * A.pairs;
        const float* s0 = t_sin + held * A.pairs;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float cs[VEC], sn[VEC];
          // (the first pair's cosines, or those of either vector, one after another)
          constexpr int kRun = kSplit ? VEC : VEC / 2;
#pragma unroll
          for (int i = 0; i < VEC; i += kRun) {
            const int p = i == 0 ? pa[j] : pb[j];
            RotVec<float, kRun> co, si;
#pragma unroll
            for (int k = 0; k < kRun; ++k) co.e[k] = 1.f, si.e[k] = 0.f;
            if (p >= 0) {
              if constexpr (kBulk) {  // (runs are aligned)
                co = *reinterpret_cast<const RotVec<float, kRun>*>(c0 + p);
                si = *reinterpret_cast<const RotVec<float, kRun>*>(s0 + p);
              } else {
#pragma unroll
                for (int k = 0; k < kRun; ++k) co.e[k] = c0[p + k], si.e[k] = s0[p + k];
              }
            }
#pragma unroll
            for (int k = 0; k < kRun; ++k) cs[i + k] = co.e[k], sn[i + k] = si.e[k];
          }
          factors(j, cs, sn);
        }
      }
      // u = t g
      [[maybe_unused]] P ua[BACK ? N : 1][W], ub[BACK ? N : 1][W];
      if constexpr (BACK) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          turn(j, ta[j], tb[j]);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            at(ua[j][i / E], i % E) = at(ta[j][i / E], i % E) * bf16_lo(gain[j][i]);
            at(ub[j][i / E], i % E) = at(tb[j][i / E], i % E) * bf16_hi(gain[j][i]);
          }
        }
      }
      float um = 0.f;  // mean(u), if it counts
      if (A.centred) {
        float s1 = 0.f, us1 = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          P sa = a[j][0], sb = b[j][0], va, vb;
          if constexpr (BACK) va = ua[j][0], vb = ub[j][0];
#pragma unroll
          for (int i = 1; i < W; ++i) {
            sa = add(sa, a[j][i]);
            sb = add(sb, b[j][i]);
            if constexpr (BACK) va = add(va, ua[j][i]), vb = add(vb, ub[j][i]);
          }
          s1 += (oa[j] >= 0 ? sum(sa) : 0.f) + (ob[j] >= 0 ? sum(sb) : 0.f);
          if constexpr (BACK) us1 += (oa[j] >= 0 ? sum(va) : 0.f) + (ob[j] >= 0 ? sum(vb) : 0.f);
        }
        if constexpr (BACK)
          head_sum2(s1, us1);
        else
          head_sum(s1);
        um = us1 * inv_d;
        const P ma = both<P>(-s1 * inv_d);
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int i = 0; i < W; ++i) {
            a[j][i] = add(a[j][i], ma);
            b[j][i] = add(b[j][i], ma);
          }
      }
      float sq = 0.f, ux = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        P qa = mul(a[j][0], a[j][0]), qb = mul(b[j][0], b[j][0]), xa, xb;
        if constexpr (BACK) xa = mul(a[j][0], ua[j][0]), xb = mul(b[j][0], ub[j][0]);
#pragma unroll
        for (int i = 1; i < W; ++i) {
          qa = fma(a[j][i], a[j][i], qa);
          qb = fma(b[j][i], b[j][i], qb);
          if constexpr (BACK) {
            xa = fma(a[j][i], ua[j][i], xa);
            xb = fma(b[j][i], ub[j][i], xb);
          }
        }
        sq += (oa[j] >= 0 ? sum(qa) : 0.f) + (ob[j] >= 0 ? sum(qb) : 0.f);
        if constexpr (BACK) ux += (oa[j] >= 0 ? sum(xa) : 0.f) + (ob[j] >= 0 ? sum(xb) : 0.f);
      }
      if constexpr (BACK)
        head_sum2(sq, ux);
      else
        head_sum(sq);
      const float r = rsqrtf(fmaf(sq, inv_d, A.eps));
      T* to = out + (x.t0 + tok) * A.ld_out + col;
      const bool put = live && MC_DCHECK(x.t0 + tok < A.tokens && x.h0 + head < Y.heads, status,
                                         kSiteQkNorm);
      // backward: r (u - n mean(u n) - mean(u)) = r u + x k1 + k0
      [[maybe_unused]] const P k1 = both<P>(-r * r * (ux * r * inv_d)), k0 = both<P>(-r * um);
      const P rr = both<P>(r);
      [[maybe_unused]] const P r_live = both<P>(live ? r : 0.f), one = both<P>(live ? 1.f : 0.f);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if constexpr (BACK) {
#pragma unroll
          for (int i = 0; i < W; ++i) {
            sga[j][i] = fma(mul(ta[j][i], r_live), a[j][i], sga[j][i]);
            sgb[j][i] = fma(mul(tb[j][i], r_live), b[j][i], sgb[j][i]);
            if constexpr (SHIFT) {
              sca[j][i] = fma(ta[j][i], one, sca[j][i]);
              scb[j][i] = fma(tb[j][i], one, scb[j][i]);
            }
            a[j][i] = fma(ua[j][i], rr, fma(a[j][i], k1, k0));
            b[j][i] = fma(ub[j][i], rr, fma(b[j][i], k1, k0));
          }
        } else {
          turn(j, a[j], b[j]);
#pragma unroll
          for (int i = 0; i < W; ++i) {
            if constexpr (SHIFT) {
              a[j][i] = fma(a[j][i], rr, ka[j][i]);
              b[j][i] = fma(b[j][i], rr, kb[j][i]);
            } else {
              a[j][i] = mul(a[j][i], rr);
              b[j][i] = mul(b[j][i], rr);
            }
          }
        }
        if (put && oa[j] >= 0) *reinterpret_cast<V*>(to + oa[j]) = pack<T, VEC>(a[j]);
        if (put && ob[j] >= 0) *reinterpret_cast<V*>(to + ob[j]) = pack<T, VEC>(b[j]);
      }
    }
    if constexpr (kBulk) {
      __syncwarp();  // the stage has been read
      if (c + C::kStages < c_end) issue(st);
    }
  }
  if constexpr (kBulk) {
    // (only after a wait that ran out: what is on its way must land)
    for (int i = n; i < n + C::kStages && c_begin + i < c_end; ++i)
      mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1, status, kSiteQkNorm, 200000000ull, false);
  }

  if constexpr (BACK) {
    if (!Y.dgain && !Y.dshift) return;
    // Sums over the heads of a warp's turn, then over the warps, in this order
    // whatever ran when: repeated calls give the same bits.
    float* const mine = reinterpret_cast<float*>(ring);
    __syncwarp();
    auto over_turn = [&](float v) {
      for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    };
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float g0 = over_turn(at(sga[j][i / E], i % E)), g1 = over_turn(at(sgb[j][i / E], i % E));
        float c0 = 0.f, c1 = 0.f;
        if constexpr (SHIFT) c0 = over_turn(at(sca[j][i / E], i % E)), c1 = over_turn(at(scb[j][i / E], i % E));
        if (seg == 0) {
          if (oa[j] >= 0) mine[oa[j] + i] = g0, mine[d + oa[j] + i] = c0;
          if (ob[j] >= 0) mine[ob[j] + i] = g1, mine[d + ob[j] + i] = c1;
        }
      }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * d; k += C::kWarps * 32) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) v += reinterpret_cast<float*>(smem + w * C::kWarp)[k];
      A.partials[static_cast<int64_t>(blockIdx.x) * 2 * d + k] = v;
    }
  }
}

// Sums the blocks' partial sums, in a fixed order: 32 dimensions of one gradient
// a block, its rows dealt to 16 warps.
constexpr int kNormSumWarps = 16;
__global__ void __launch_bounds__(kNormSumWarps * 32)
    qk_norm_sum_kernel(const __grid_constant__ NormArgs A) {
  __shared__ float red[kNormSumWarps][33];
  pdl_wait();  // the partial sums are complete
  pdl_launch();
  const NormType& Y = A.type[blockIdx.z];
  float* out = blockIdx.y == 0 ? Y.dgain : Y.dshift;
  if (!out) return;
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const int k = static_cast<int>(blockIdx.x) * 32 + lane;
  float v = 0.f;
  if (k < A.d) {
    const float* p = A.partials + static_cast<int64_t>(Y.block0) * 2 * A.d +
                     static_cast<int>(blockIdx.y) * A.d + k;
#pragma unroll 8
    for (int row = warp; row < Y.blocks; row += kNormSumWarps) v += p[static_cast<int64_t>(row) * 2 * A.d];
  }
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && k < A.d) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kNormSumWarps; ++w) s += red[w][lane];
    out[k] = A.accumulate ? out[k] + s : s;
  }
}

struct NormCall {
  const void *in, *dout;
  void* out;
  const int32_t* positions;
  const float* inv_freq;
  int* status;
  cudaStream_t st;
};

template <typename T, int VEC, bool ADJACENT, bool BACK, bool SHIFT>
int norm_launch(const NormCall& c, NormArgs A) {
  auto kern = qk_norm_kernel<T, VEC, ADJACENT, BACK, SHIFT>;
  using C = NormCfg<BACK>;
  // at most as many blocks as are resident at once
  static PerDeviceInit init;
  long long resident = 0;
  const cudaError_t e = once_per_device(init, [&](long long* value) {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (r != cudaSuccess) return r;
    int per_sm = 0;
    r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, C::kWarps * 32, C::kSmem);
    *value = static_cast<long long>(per_sm < 1 ? 1 : per_sm) * num_sms();
    return r;
  }, &resident);
  if (e != cudaSuccess) return MC_ERR_CUDA;
  // units of a head
  const int vecs = A.d / VEC;
  A.units = ADJACENT && VEC > 1 ? (vecs + 1) / 2
                                : A.pairs / VEC + ((A.d - 2 * A.pairs) / VEC + 1) / 2;
  A.log_lanes = 0;
  while ((1 << A.log_lanes) < A.units && A.log_lanes < 5) ++A.log_lanes;
  A.lanes = 1 << A.log_lanes;
  const int per_turn = 32 / A.lanes;
  A.div_pairs = fast_div_magic(A.pairs > 0 ? A.pairs : 1);
  // Turns of a chunk: one where the call is too short to fill the SMs otherwise.
  int64_t blocks[2] = {0, 0}, all = 0;
  double cost[2] = {0.0, 0.0};
  const int64_t all_turns =
      A.tokens * (A.type[0].heads + A.type[1].heads) / per_turn;
  const int turns = all_turns < 4 * C::kTurns * resident * C::kWarps ? 1 : C::kTurns;
  for (int t = 0; t < 2; ++t) {
    NormType& Y = A.type[t];
    Y.chunks = 0;
    Y.head_chunk = Y.tok_chunk = Y.ranges = 1;
    if (Y.heads > 0) {
      const int slots = per_turn * turns;
      Y.head_chunk = Y.heads < slots ? Y.heads : slots;
      int tk = slots / Y.head_chunk;
      if (A.pairs > 0 && tk > kNormTable / A.pairs) tk = kNormTable / A.pairs;
      if (A.pairs > 0 && tk > 32 / A.axes) tk = 32 / A.axes;
      if (tk > A.tokens) tk = static_cast<int>(A.tokens);
      Y.tok_chunk = tk;
      Y.ranges = (Y.heads + Y.head_chunk - 1) / Y.head_chunk;
      Y.chunks = (A.tokens + tk - 1) / tk * Y.ranges;
    }
    Y.div_head_chunk = fast_div_magic(Y.head_chunk);
    blocks[t] = (Y.chunks + C::kWarps - 1) / C::kWarps;
    all += blocks[t];
    // a token's angles and factors take a warp as long as a turn and a half
    cost[t] = static_cast<double>(Y.chunks) *
              (turns + (A.pairs > 0 ? 1.5 * Y.tok_chunk / Y.ranges : 0.0));
  }
  const int64_t most = BACK && resident > kNormMaxBlocks ? kNormMaxBlocks : resident;
  if (all > most) {
    // shared out by the work, one block at least where there is any
    const int64_t q = static_cast<int64_t>(cost[0] / (cost[0] + cost[1]) * most + 0.5);
    if (blocks[0] > 0 && blocks[1] > 0) {
      blocks[0] = q < 1 ? 1 : q > most - 1 ? most - 1 : q;
      blocks[1] = most - blocks[0];
    } else {
      (blocks[0] > 0 ? blocks[0] : blocks[1]) = most;
    }
  }
  A.type[0].block0 = 0;
  A.type[0].blocks = static_cast<int>(blocks[0]);
  A.type[1].block0 = A.type[0].blocks;
  A.type[1].blocks = static_cast<int>(blocks[1]);
  for (int t = 0; t < 2; ++t) {
    NormType& Y = A.type[t];
    const int64_t warps = static_cast<int64_t>(Y.blocks) * C::kWarps;
    Y.per_warp = warps > 0 ? Y.chunks / warps : 0;
    Y.more = Y.chunks - Y.per_warp * warps;
  }
  launch_kernel(kern, dim3(static_cast<unsigned>(blocks[0] + blocks[1])), dim3(C::kWarps * 32),
                C::kSmem, c.st, 1, static_cast<const T*>(c.in), static_cast<const T*>(c.dout),
                static_cast<T*>(c.out), c.positions, c.inv_freq, A, c.status);
  if (cudaGetLastError() != cudaSuccess) return MC_ERR_CUDA;
  if constexpr (BACK) {
    bool any = false;
    for (int t = 0; t < 2; ++t) {
      if (A.type[t].heads == 0) A.type[t].dgain = A.type[t].dshift = nullptr;
      any = any || A.type[t].dgain || A.type[t].dshift;
    }
    if (any) {
      launch_kernel(qk_norm_sum_kernel, dim3(static_cast<unsigned>((A.d + 31) / 32), 2, 2),
                    dim3(kNormSumWarps * 32), 0, c.st, 1, A);
      if (cudaGetLastError() != cudaSuccess) return MC_ERR_CUDA;
    }
  }
  return MC_OK;
}

template <typename T, int VEC>
int norm_vec(const NormCall& c, const NormArgs& A, bool adjacent, bool back) {
  const bool shift = back ? A.type[0].dshift || A.type[1].dshift
                          : A.type[0].shift || A.type[1].shift;
  if (!back && shift)
    return adjacent ? norm_launch<T, VEC, true, false, true>(c, A)
                    : norm_launch<T, VEC, false, false, true>(c, A);
  if (!back)
    return adjacent ? norm_launch<T, VEC, true, false, false>(c, A)
                    : norm_launch<T, VEC, false, false, false>(c, A);
  if (shift)
    return adjacent ? norm_launch<T, VEC, true, true, true>(c, A)
                    : norm_launch<T, VEC, false, true, true>(c, A);
  return adjacent ? norm_launch<T, VEC, true, true, false>(c, A)
                  : norm_launch<T, VEC, false, true, false>(c, A);
}

template <typename T>
int norm_typed(const NormCall& c, const NormArgs& A, bool adjacent, bool back) {
  constexpr int kFull = 16 / sizeof(T);
  // The widest vector that pairs, heads, rows and all addresses are whole
  // multiples of.
  auto fits = [&](int vec) {
    const uintptr_t bytes = sizeof(T) * static_cast<uintptr_t>(vec);
    auto at = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    return (adjacent ? 2 * A.pairs : A.pairs) % vec == 0 && A.d % vec == 0 && A.ld_in % vec == 0 &&
           A.ld_out % vec == 0 && (!back || A.ld_dout % vec == 0) && at(c.in) && at(c.out) &&
           (!back || at(c.dout));
  };
  if (fits(kFull)) return norm_vec<T, kFull>(c, A, adjacent, back);
  if (fits(2)) return norm_vec<T, 2>(c, A, adjacent, back);
  return norm_vec<T, 1>(c, A, adjacent, back);
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

int check_qk_norm(const mc_qk_norm* norm) {
  if (!norm) return MC_ERR_NULLPTR;
  if (norm->flags & ~MC_QK_NORM_CENTRED) return MC_ERR_ARGUMENT;
  if (!(norm->eps >= 1e-12f && norm->eps <= 1.f)) return MC_ERR_ARGUMENT;
  if (!aligned(norm->q_gain, 2) || !aligned(norm->q_shift, 2) || !aligned(norm->k_gain, 2) ||
      !aligned(norm->k_shift, 2))
    return MC_ERR_ALIGN;
  return MC_OK;
}

size_t qk_norm_scratch_floats(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim) {
  if (tokens < 1 || q_heads < 0 || k_heads < 0 || q_heads + k_heads < 1 || head_dim < 1 ||
      head_dim > kNormMaxDim)
    return 0;
  // a row of two sums per dimension for every block; a block has a (token, head)
  // pair at least, of queries or of keys
  const double pairs = static_cast<double>(tokens) * static_cast<double>(q_heads + k_heads);
  const int64_t rows = pairs < kNormMaxBlocks ? static_cast<int64_t>(pairs) : kNormMaxBlocks;
  return static_cast<size_t>(rows * 2 * head_dim);
}

int launch_qk_norm(const QkNormCall& q, cudaStream_t st) {
  int rc = check_qk_norm(q.norm);
  if (rc != MC_OK) return rc;
  const bool back = q.dout != nullptr || q.backward;
  if (q.head_dim < 1) return MC_ERR_SHAPE;
  if (q.spec) {
    rc = check_rotary_spec(q.spec, q.head_dim);
    if (rc != MC_OK) return rc;
  }
  if (q.tokens < 1 || q.q_heads < 0 || q.k_heads < 0) return MC_ERR_SHAPE;
  const int64_t heads = static_cast<int64_t>(q.q_heads) + q.k_heads;
  if (heads < 1) return MC_ERR_SHAPE;
  const int64_t width = heads * q.head_dim;
  if (q.head_dim > kNormMaxDim || width > (1 << 22)) return MC_ERR_UNSUPPORTED;
  if (q.ld_in < width || q.ld_out < width || (back && q.ld_dout < width)) return MC_ERR_SHAPE;
  if (!q.in || !q.out || (back && !q.dout)) return MC_ERR_NULLPTR;
  if (q.spec && (!q.positions || !q.inv_freq)) return MC_ERR_NULLPTR;
  const uintptr_t size = q.bf16 ? 2 : 4;
  if (!aligned(q.in, size) || !aligned(q.out, size) || !aligned(q.dout, size)) return MC_ERR_ALIGN;
  if (q.spec && (!aligned(q.positions, 4) || !aligned(q.inv_freq, 4))) return MC_ERR_ALIGN;
  // in place: the same rows
  if ((q.in == q.out && q.ld_in != q.ld_out) || (back && q.dout == q.out && q.ld_dout != q.ld_out))
    return MC_ERR_ARGUMENT;
  NormArgs A = {};
  A.type[0].gain = q.norm->q_gain;
  A.type[0].shift = q.norm->q_shift;
  A.type[1].gain = q.norm->k_gain;
  A.type[1].shift = q.norm->k_shift;
  if (back && q.grads) {
    const mc_qk_norm_grads& g = *q.grads;
    if (!aligned(g.q_gain, 4) || !aligned(g.q_shift, 4) || !aligned(g.k_gain, 4) ||
        !aligned(g.k_shift, 4) || !aligned(q.scratch, 4))
      return MC_ERR_ALIGN;
    if ((g.q_gain || g.q_shift || g.k_gain || g.k_shift) && !q.scratch) return MC_ERR_NULLPTR;
    A.type[0].dgain = g.q_gain;
    A.type[0].dshift = g.q_shift;
    A.type[1].dgain = g.k_gain;
    A.type[1].dshift = g.k_shift;
  }
  A.type[0].heads = q.q_heads;
  A.type[1].head0 = q.q_heads;
  A.type[1].heads = q.k_heads;
  A.tokens = q.tokens;
  A.ld_in = q.ld_in;
  A.ld_dout = q.ld_dout;
  A.ld_out = q.ld_out;
  A.d = q.head_dim;
  A.pairs = q.spec ? q.spec->rot_dim / 2 : 0;
  A.axes = q.spec ? q.spec->axes : 1;
  A.centred = (q.norm->flags & MC_QK_NORM_CENTRED) ? 1 : 0;
  A.inverse = back ? 1 : 0;
  A.accumulate = q.accumulate;
  A.eps = q.norm->eps;
  A.partials = q.scratch;
  if (q.spec) rotary_axes(q.spec, A.axis);
  const bool adjacent = q.spec && (q.spec->flags & MC_ROTARY_ADJACENT_PAIRS);
  const NormCall c = {q.in, q.dout, q.out, q.positions, q.inv_freq, q.status, st};
  return q.bf16 ? norm_typed<__nv_bfloat16>(c, A, adjacent, back)
                : norm_typed<float>(c, A, adjacent, back);
}

}  // namespace mc

extern "C" {

int mc_qk_norm_forward(const void* in, void* out, int32_t is_bf16, int64_t tokens,
                       int32_t q_heads, int32_t k_heads, int32_t head_dim, int64_t ld_in,
                       int64_t ld_out, const mc_qk_norm* norm, const int32_t* positions,
                       const float* inv_freq, const mc_rotary_spec* spec, int* status,
                       void* stream) {
  mc::QkNormCall q = {};
  q.in = in;
  q.out = out;
  q.bf16 = is_bf16 != 0;
  q.tokens = tokens;
  q.q_heads = q_heads;
  q.k_heads = k_heads;
  q.head_dim = head_dim;
  q.ld_in = ld_in;
  q.ld_out = ld_out;
  q.norm = norm;
  q.positions = positions;
  q.inv_freq = inv_freq;
  q.spec = spec;
  q.status = status;
  return mc::launch_qk_norm(q, static_cast<cudaStream_t>(stream));
}

size_t mc_qk_norm_scratch_floats(int64_t tokens, int32_t q_heads, int32_t k_heads,
                                 int32_t head_dim) {
  return mc::qk_norm_scratch_floats(tokens, q_heads, k_heads, head_dim);
}

int mc_qk_norm_backward(const void* in, const void* dout, void* din, int32_t is_bf16,
                        int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                        int64_t ld_in, int64_t ld_dout, int64_t ld_din, const mc_qk_norm* norm,
                        const int32_t* positions, const float* inv_freq,
                        const mc_rotary_spec* spec, const mc_qk_norm_grads* grads,
                        int32_t accumulate, float* scratch, int* status, void* stream) {
  mc::QkNormCall q = {};
  q.in = in;
  q.dout = dout;
  q.out = din;
  q.backward = true;
  q.bf16 = is_bf16 != 0;
  q.tokens = tokens;
  q.q_heads = q_heads;
  q.k_heads = k_heads;
  q.head_dim = head_dim;
  q.ld_in = ld_in;
  q.ld_dout = ld_dout;
  q.ld_out = ld_din;
  q.norm = norm;
  q.positions = positions;
  q.inv_freq = inv_freq;
  q.spec = spec;
  q.grads = grads;
  q.accumulate = accumulate;
  q.scratch = scratch;
  q.status = status;
  return mc::launch_qk_norm(q, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
