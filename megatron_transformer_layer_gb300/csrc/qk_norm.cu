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

constexpr int kNormWarps = 4;
constexpr int kNormTurns = 8;    // turns of an item, at most
constexpr int kNormTable = 512;  // (token, pair) entries of a warp's cos / sin table (4 KB)
constexpr int kNormMaxDim = 256;
constexpr int kNormMaxBlocks = 1024;  // of the backward pass: rows of partial sums

// Queries (0) and keys (1) are walked apart, each by blocks of its own, so that
// a lane's gains, shifts and gradient sums stay in registers.
struct NormType {
  const uint16_t* gain;   // bf16 [d], or NULL: ones
  const uint16_t* shift;  // or NULL: zeros
  float* dgain;           // or NULL
  float* dshift;
  int64_t items;       // (token group, head range) pairs, one warp each
  int head0, heads;    // of the row's heads
  int tok_item, head_item, ranges;  // an item: tokens, heads of each; ranges per token
  int block0, blocks;
  uint32_t div_head_item;
};

struct NormArgs {
  NormType type[2];
  int64_t tokens, ld_in, ld_dout, ld_out;
  int d, pairs;
  int lanes, units;  // lanes of a head (a power of two) and its units
  int centred, inverse, accumulate;
  float eps;
  uint32_t div_pairs;
  float* partials;  // backward: [block][2][d]
  uint8_t axis[kRotaryMaxPairs];
};

// A unit is two vectors: the halves of VEC pairs, or of adjacent pairs and of
// what does not turn two neighbouring ones (the second may be missing).  `lanes`
// lanes hold a head, one unit (or N, for narrow vectors) each, and a lane has
// the same unit of every head it meets: its gains are loaded once, its cosines
// once per token.  Of a warp's turn the lanes hold 32 / lanes heads, of the same
// token or of the next ones.
template <typename T, int VEC, bool ADJACENT, bool BACK, bool SHIFT>
__global__ void __launch_bounds__(kNormWarps * 32)
    qk_norm_kernel(const T* in, const T* dout, T* out, const int32_t* __restrict__ positions,
                   const float* __restrict__ inv_freq, const __grid_constant__ NormArgs A,
                   int* status) {
  using V = RotVec<T, VEC>;
  constexpr bool kSplit = !ADJACENT || VEC == 1;  // a pair's halves are in two vectors
  constexpr int N = VEC * sizeof(T) == 16 ? 1 : (VEC == 2 ? 2 : 4);
  __shared__ uint64_t turns[kNormMaxDim / 2];
  __shared__ __align__(16) float table[kNormWarps][2][kNormTable];
  pdl_wait();  // the previous kernel on the stream has completed
  pdl_launch();
  for (int p = threadIdx.x; p < A.pairs; p += kNormWarps * 32) turns[p] = turns_fixed(inv_freq[p]);
  __syncthreads();
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  float* const t_cos = table[warp][0];
  float* const t_sin = table[warp][1];
  const NormType& Y = A.type[static_cast<int>(blockIdx.x) >= A.type[1].block0 ? 1 : 0];
  const int d = A.d, L = A.lanes;
  const int seg = lane / L, per_turn = 32 / L;
  const float inv_d = 1.f / static_cast<float>(d);

  // this lane's units: first dimensions of the two vectors (-1: none) and the
  // first pair of each (of both, where the vectors are halves; -1: does not turn)
  int oa[N], ob[N], pa[N], pb[N];
  float ga[N][VEC], gb[N][VEC], ca[N][VEC], cb[N][VEC];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int u = lane % L + j * L;
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
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      ga[j][i] = gb[j][i] = 1.f;
      ca[j][i] = cb[j][i] = 0.f;
      if (Y.gain && oa[j] >= 0) ga[j][i] = bf16_lo(Y.gain[oa[j] + i]);
      if (Y.gain && ob[j] >= 0) gb[j][i] = bf16_lo(Y.gain[ob[j] + i]);
      if constexpr (!BACK) {
        if (Y.shift && oa[j] >= 0) ca[j][i] = bf16_lo(Y.shift[oa[j] + i]);
        if (Y.shift && ob[j] >= 0) cb[j][i] = bf16_lo(Y.shift[ob[j] + i]);
      }
    }
  }
  // backward: this lane's sums of t n and t
  float sga[BACK ? N : 1][VEC] = {}, sgb[BACK ? N : 1][VEC] = {};
  float sca[BACK && SHIFT ? N : 1][VEC] = {}, scb[BACK && SHIFT ? N : 1][VEC] = {};
  float cs[N][VEC], sn[N][VEC];  // of the token `held` (adjacent: half for each vector)
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) cs[j][i] = 1.f, sn[j][i] = 0.f;

  // sums over the lanes of a head
  auto head_sum2 = [&](float& a, float& b) {
    for (int o = L >> 1; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
  };

  struct Raw {
    V a[N], b[N];
    [[maybe_unused]] V da[N], db[N];
    int tok, head;  // tok < 0: nothing
  };
  const int64_t warps = static_cast<int64_t>(Y.blocks) * kNormWarps;
  for (int64_t item = static_cast<int64_t>(static_cast<int>(blockIdx.x) - Y.block0) * kNormWarps + warp;
       item < Y.items; item += warps) {
    const int64_t group = item / Y.ranges;
    const int64_t t0 = group * Y.tok_item;
    const int ntok = static_cast<int>(min(static_cast<int64_t>(Y.tok_item), A.tokens - t0));
    const int h0 = static_cast<int>(item - group * Y.ranges) * Y.head_item;
    const int nh = min(Y.head_item, Y.heads - h0);
    const int total = ntok * nh;
    auto load = [&](int e) {
      Raw x;
      x.tok = -1;
      x.head = 0;
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          x.a[j].e[i] = x.b[j].e[i] = from_f32<T>(0.f);
          if constexpr (BACK) x.da[j].e[i] = x.db[j].e[i] = from_f32<T>(0.f);
        }
      if (e < total) {
        x.tok = nh == Y.head_item ? fast_div(e, Y.div_head_item) : e / nh;
        x.head = Y.head0 + h0 + (e - x.tok * nh);
        const T* row = in + (t0 + x.tok) * A.ld_in + static_cast<int64_t>(x.head) * d;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (oa[j] >= 0) x.a[j] = *reinterpret_cast<const V*>(row + oa[j]);
          if (ob[j] >= 0) x.b[j] = *reinterpret_cast<const V*>(row + ob[j]);
        }
        if constexpr (BACK) {
          const T* drow = dout + (t0 + x.tok) * A.ld_dout + static_cast<int64_t>(x.head) * d;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            if (oa[j] >= 0) x.da[j] = *reinterpret_cast<const V*>(drow + oa[j]);
            if (ob[j] >= 0) x.db[j] = *reinterpret_cast<const V*>(drow + ob[j]);
          }
        }
      }
      return x;
    };
    Raw cur = load(seg);
    int held = -1;
    if (A.pairs > 0) {
      __syncwarp();  // the table of the item before has been read
      for (int i = lane; i < ntok * A.pairs; i += 32) {
        const int tk = fast_div(i, A.div_pairs), p = i - tk * A.pairs;
        const int64_t pos = positions[A.axis[p] * A.tokens + t0 + tk];
        float s, c;
        turn_sincos(A.inverse ? -pos : pos, turns[p], &s, &c);
        t_cos[i] = c;
        t_sin[i] = s;
      }
      __syncwarp();
    }
    for (int e0 = 0; e0 < total; e0 += per_turn) {
      if (A.pairs > 0 && cur.tok >= 0 && cur.tok != held) {
        held = cur.tok;
        const float* c0 = t_cos + held * A.pairs;
        const float* s0 = t_sin + held * A.pairs;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const int p = kSplit ? pa[j] : (i < VEC / 2 ? pa[j] : pb[j]);
            const int at = kSplit || i < VEC / 2 ? i : i - VEC / 2;
            if (p >= 0) cs[j][i] = c0[p + at], sn[j][i] = s0[p + at];
          }
      }
      // pairs turn by the angle whose cosine and sine are cs, sn
      auto turn = [&](int j, float (&a)[VEC], float (&b)[VEC]) {
        if constexpr (kSplit) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float u = a[i], v = b[i];
            a[i] = u * cs[j][i] - v * sn[j][i];
            b[i] = u * sn[j][i] + v * cs[j][i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            const float u = a[2 * i], v = a[2 * i + 1], x = b[2 * i], y = b[2 * i + 1];
            a[2 * i] = u * cs[j][i] - v * sn[j][i];
            a[2 * i + 1] = u * sn[j][i] + v * cs[j][i];
            b[2 * i] = x * cs[j][VEC / 2 + i] - y * sn[j][VEC / 2 + i];
            b[2 * i + 1] = x * sn[j][VEC / 2 + i] + y * cs[j][VEC / 2 + i];
          }
        }
      };
      float a[N][VEC], b[N][VEC];
      [[maybe_unused]] float ta[N][VEC], tb[N][VEC];
      float sum = 0.f, usum = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          a[j][i] = to_f32(cur.a[j].e[i]);
          b[j][i] = to_f32(cur.b[j].e[i]);
          sum += a[j][i] + b[j][i];
          if constexpr (BACK) {
            ta[j][i] = to_f32(cur.da[j].e[i]);
            tb[j][i] = to_f32(cur.db[j].e[i]);
          }
        }
        if constexpr (BACK) {
          turn(j, ta[j], tb[j]);
#pragma unroll
          for (int i = 0; i < VEC; ++i) usum += ta[j][i] * ga[j][i] + tb[j][i] * gb[j][i];
        }
      }
      if (A.centred) {
        head_sum2(sum, usum);
        const float m = sum * inv_d;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            if (oa[j] >= 0) a[j][i] -= m;
            if (ob[j] >= 0) b[j][i] -= m;
          }
      }
      float sq = 0.f, ux = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          sq += a[j][i] * a[j][i] + b[j][i] * b[j][i];
          if constexpr (BACK)
            ux += ta[j][i] * ga[j][i] * a[j][i] + tb[j][i] * gb[j][i] * b[j][i];
        }
      head_sum2(sq, ux);
      const float r = rsqrtf(fmaf(sq, inv_d, A.eps));
      const float un = ux * r * inv_d, um = A.centred ? usum * inv_d : 0.f;  // mean(u n), mean(u)
      T* row = out + (t0 + max(cur.tok, 0)) * A.ld_out + static_cast<int64_t>(cur.head) * d;
      const bool put = cur.tok >= 0 &&
                       MC_DCHECK(t0 + cur.tok < A.tokens && cur.head < Y.head0 + Y.heads, status,
                                 kSiteQkNorm);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        V ya, yb;
        if constexpr (BACK) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float na = a[j][i] * r, nb = b[j][i] * r;
            ya.e[i] = from_f32<T>(r * (ta[j][i] * ga[j][i] - na * un - um));
            yb.e[i] = from_f32<T>(r * (tb[j][i] * gb[j][i] - nb * un - um));
            sga[j][i] += ta[j][i] * na;
            sgb[j][i] += tb[j][i] * nb;
            if constexpr (SHIFT) {
              sca[j][i] += ta[j][i];
              scb[j][i] += tb[j][i];
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            a[j][i] = fmaf(a[j][i] * r, ga[j][i], ca[j][i]);
            b[j][i] = fmaf(b[j][i] * r, gb[j][i], cb[j][i]);
          }
          turn(j, a[j], b[j]);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            ya.e[i] = from_f32<T>(a[j][i]);
            yb.e[i] = from_f32<T>(b[j][i]);
          }
        }
        if (put && oa[j] >= 0) *reinterpret_cast<V*>(row + oa[j]) = ya;
        if (put && ob[j] >= 0) *reinterpret_cast<V*>(row + ob[j]) = yb;
      }
      cur = load(e0 + per_turn + seg);
    }
  }

  if constexpr (BACK) {
    if (!Y.dgain && !Y.dshift) return;
    // Sums over the heads of a warp's turn, then over the warps, in this order
    // whatever ran when: repeated calls give the same bits.  (`table` is free:
    // 2 x 256 floats of each warp.)
    __syncthreads();
    auto over_turn = [&](float v) {
      for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    };
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float g0 = over_turn(sga[j][i]), g1 = over_turn(sgb[j][i]);
        float c0 = 0.f, c1 = 0.f;
        if constexpr (SHIFT) c0 = over_turn(sca[j][i]), c1 = over_turn(scb[j][i]);
        if (seg == 0) {
          if (oa[j] >= 0) t_cos[oa[j] + i] = g0, t_sin[oa[j] + i] = c0;
          if (ob[j] >= 0) t_cos[ob[j] + i] = g1, t_sin[ob[j] + i] = c1;
        }
      }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * d; k += kNormWarps * 32) {
      const int part = k >= d, at = k - part * d;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kNormWarps; ++w) v += table[w][part][at];
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
  // at most as many blocks as are resident at once
  static PerDeviceInit init;
  long long resident = 0;
  const cudaError_t e = once_per_device(init, [&](long long* value) {
    int per_sm = 0;
    const cudaError_t r =
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kNormWarps * 32, 0);
    *value = static_cast<long long>(per_sm < 1 ? 1 : per_sm) * num_sms();
    return r;
  }, &resident);
  if (e != cudaSuccess) return MC_ERR_CUDA;
  // units of a head
  const int vecs = A.d / VEC;
  A.units = ADJACENT && VEC > 1 ? (vecs + 1) / 2
                                : A.pairs / VEC + ((A.d - 2 * A.pairs) / VEC + 1) / 2;
  A.lanes = 1;
  while (A.lanes < A.units && A.lanes < 32) A.lanes *= 2;
  const int per_turn = 32 / A.lanes;
  A.div_pairs = fast_div_magic(A.pairs > 0 ? A.pairs : 1);
  // Turns of an item: enough that forming its table does not show, fewer where
  // the call is too short to fill the SMs otherwise.
  int64_t blocks[2] = {0, 0}, all = 0;
  const int64_t all_turns =
      A.tokens * (A.type[0].heads + A.type[1].heads) / per_turn;
  const int64_t fill = all_turns / (32ll * num_sms());
  const int turns = fill < 1 ? 1 : fill > kNormTurns ? kNormTurns : static_cast<int>(fill);
  for (int t = 0; t < 2; ++t) {
    NormType& Y = A.type[t];
    Y.items = 0;
    Y.head_item = Y.tok_item = Y.ranges = 1;
    if (Y.heads > 0) {
      const int slots = per_turn * turns;
      Y.head_item = Y.heads < slots ? Y.heads : slots;
      int tk = slots / Y.head_item;
      if (A.pairs > 0 && tk > kNormTable / A.pairs) tk = kNormTable / A.pairs;
      if (tk > A.tokens) tk = static_cast<int>(A.tokens);
      Y.tok_item = tk;
      Y.ranges = (Y.heads + Y.head_item - 1) / Y.head_item;
      Y.items = (A.tokens + tk - 1) / tk * Y.ranges;
    }
    Y.div_head_item = fast_div_magic(Y.head_item);
    blocks[t] = (Y.items + kNormWarps - 1) / kNormWarps;
    all += blocks[t];
  }
  const int64_t most = BACK && resident > kNormMaxBlocks ? kNormMaxBlocks : resident;
  if (all > most) {
    // shared out by the items, one block at least where there are any
    const int64_t q = (blocks[0] * most + all / 2) / all;
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
  launch_kernel(kern, dim3(static_cast<unsigned>(blocks[0] + blocks[1])), dim3(kNormWarps * 32), 0,
                c.st, 1, static_cast<const T*>(c.in), static_cast<const T*>(c.dout),
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
  const bool shift = A.type[0].dshift || A.type[1].dshift;
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
