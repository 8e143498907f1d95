// Attention forward over interval masks (sm_103a, tcgen05), scores optionally
// capped by a tanh and biased by the distance:
//   O_i = sum_j P_ij V_j over the keys j in [lo_i, hi_i), P the softmax.
//
// One CTA per (128-query block, head), longest key ranges first (the mask's
// tables), walks the 128-key blocks between its rows' lowest and highest key
// with one running maximum and sum per row.  192 threads:
//   warp 0      TMA: Q once, K and V blocks
//   warp 1      TMEM and the MMA thread: S = Q K^T, O += P V
//   warps 2..5  softmax: thread = row, the row's 128 scores in registers
// Two CTAs share an SM (256 TMEM columns and at most 113 KB of shared memory
// each): while one is in its softmax, or fetches its first blocks or writes
// its O, the other's products keep the tensor cores busy.  That is why S has
// no second buffer (P_j takes S_j's columns, S_{j+1} follows O += P_j V_j),
// and it suits packed documents, whose CTAs have one to a few key blocks.
// TMEM: S [0, 128) with P (bf16 pairs) over [0, 64), O [128, 128 + D).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attention_opt.cuh"

namespace mc {
namespace {

constexpr int kOptFwdThreads = 192;
// O is rescaled only when a row's maximum grows by more than this (log2
// units): P stays below 2^8 and the final division by the sum, taken against
// the same maximum, cancels the difference.
constexpr float kOptRescale = 8.0f;

template <int D>
struct OptFwdCfg {
  static constexpr int kChunks = D / 64;        // 128-byte boxes per row
  static constexpr int kTile = 128 * D * 2;     // 128 rows of Q, K or V
  static constexpr int kStages = D == 64 ? 2 : 1;
  static constexpr int kBars = 16 * 8;
  static constexpr int kUsed = kTile + 2 * kStages * kTile + kBars;
  static constexpr int kSmem = kUsed + 1024;    // + alignment slack
  static_assert(kSmem <= 113 * 1024, "two CTAs per SM");
  static constexpr uint32_t kTmemCols = 256;
  static constexpr uint32_t kColS = 0, kColO = 128;
};

struct OptFwdArgs {
  uint16_t* out;
  float* lse;
  const int32_t* key_lo;
  const int32_t* key_hi;
  const int32_t* tables;
  const float* slopes;
  float softcap;
  int b, s, H;
  int head_major;
  int* status;
};

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kOptFwdThreads, 2)
    attn_opt_fwd_kernel(const __grid_constant__ CUtensorMap tm,
                        const __grid_constant__ OptFwdArgs A) {
  using C = OptFwdCfg<D>;
  constexpr int KS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::kTile;
  uint8_t* sV = sK + KS * C::kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + KS * C::kTile);
  uint64_t* q_full = bars + 0;
  uint64_t* k_full = bars + 1;    // [KS]
  uint64_t* k_empty = bars + 3;   // [KS]  after S_j
  uint64_t* v_full = bars + 5;    // [KS]
  uint64_t* v_empty = bars + 7;   // [KS]  after O += P_j V_j
  uint64_t* s_full = bars + 9;    // S_j in TMEM
  uint64_t* p_full = bars + 10;   // P_j in TMEM (128 threads)
  uint64_t* pv_done = bars + 11;  // O += P_j V_j complete
  uint64_t* drain = bars + 12;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 13);
  int* status = A.status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = A.s, a = A.H * D;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < KS; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(p_full, 128);
    mbar_init(pv_done, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // the previous kernel on the stream has completed
  const uint32_t tS = tmem + C::kColS, tO = tmem + C::kColO;

  int4 entry;  // sequence, query block, lowest and highest visible key
  int hh;
  const bool ok_entry =
      opt_entry(A.tables, A.head_major != 0, A.b, (s + 127) / 128, entry, hh, status);
  const int bi = entry.x;
  const int q0 = entry.y * 128;
  const int k_lo = max(entry.z, 0), k_hi = min(entry.w, s);
  const int n_kb = ok_entry && k_hi > k_lo ? (k_hi - k_lo + 127) / 128 : 0;

  if (warp == 0) {
    if (lane == 0 && n_kb > 0) {
      // -------------------------------------------------------- producer
      mbar_arrive_expect_tx(q_full, C::kTile);
      for (int c = 0; c < C::kChunks; ++c)
        tma_load_3d(sQ + c * 16384, &tm, q_full, hh * D + c * 64, q0, bi);
      int k_issued = 0, v_issued = 0;
      for (int j = 0; j < n_kb; ++j) {
        const int st = j % KS;
        const uint32_t ph = ((j / KS) & 1) ^ 1u;
        if (!mbar_wait(&k_empty[st], ph, status, kSiteAttention)) break;
        mbar_arrive_expect_tx(&k_full[st], C::kTile);
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_3d(sK + st * C::kTile + c * 16384, &tm, &k_full[st], a + hh * D + c * 64,
                      k_lo + j * 128, bi);
        ++k_issued;
        if (!mbar_wait(&v_empty[st], ph, status, kSiteAttention)) break;
        mbar_arrive_expect_tx(&v_full[st], C::kTile);
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_3d(sV + st * C::kTile + c * 16384, &tm, &v_full[st], 2 * a + hh * D + c * 64,
                      k_lo + j * 128, bi);
        ++v_issued;
      }
      pdl_launch();  // every load of this CTA is issued
      // Copies still in flight must land before the CTA exits.
      mbar_wait(q_full, 0, status, kSiteAttention, 200000000ull, false);
      for (int j = k_issued - 1; j >= 0 && j >= k_issued - KS; --j)
        mbar_wait(&k_full[j % KS], (j / KS) & 1, status, kSiteAttention, 200000000ull, false);
      for (int j = v_issued - 1; j >= 0 && j >= v_issued - KS; --j)
        mbar_wait(&v_full[j % KS], (j / KS) & 1, status, kSiteAttention, 200000000ull, false);
    }
  } else if (warp == 1) {
    if (lane == 0 && n_kb > 0) {
      // -------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, false, true);
      const uint32_t qb = smem_u32(sQ);
      auto issue_s = [&](int j) -> bool {
        const int st = j % KS;
        if (!mbar_wait(&k_full[st], (j / KS) & 1, status, kSiteAttention)) return false;
        tc_fence_after();
        const uint32_t kbase = smem_u32(sK + st * C::kTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          umma_bf16(tS, smem_desc_sw128(qb + off, 16, 1024), smem_desc_sw128(kbase + off, 16, 1024),
                    kIdescQK, kk > 0 ? 1u : 0u);
        }
        umma_commit(s_full);
        umma_commit(&k_empty[st]);
        return true;
      };
      bool ok = mbar_wait(q_full, 0, status, kSiteAttention) && issue_s(0);
      for (int j = 0; ok && j < n_kb; ++j) {
        const int st = j % KS;
        if (!mbar_wait(p_full, j & 1, status, kSiteAttention)) break;
        if (!mbar_wait(&v_full[st], (j / KS) & 1, status, kSiteAttention)) break;
        tc_fence_after();
        const uint32_t vb = smem_u32(sV + st * C::kTile);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          // P: 16 keys = 8 packed columns; V (MN-major): 16 key rows of
          // 128 B, 64-wide d chunks 16 KB apart
          umma_bf16_ts(tO, tS + kk * 8, smem_desc_sw128(vb + kk * 2048, 16384, 1024), kIdescPV,
                       (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&v_empty[st]);
        umma_commit(pv_done);
        if (j + 1 < n_kb) {
          // S_{j+1} overwrites the P_j that the products above read
          if (!mbar_wait(pv_done, j & 1, status, kSiteAttention)) break;
          ok = issue_s(j + 1);
        }
      }
      umma_commit(drain);
      mbar_wait(drain, 0, status, kSiteAttention, 200000000ull, false);
    }
  } else {
    // ---------------------------------------------------------- softmax
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int q = q0 + row;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    // Rows past the sequence (zeros from the TMA, never stored) see everything,
    // so that they do not make a block an edge.
    int lo = 0, hi = 0x7fffffff;
    if (ok_entry && q < s) {
      lo = A.key_lo[static_cast<int64_t>(bi) * s + q];
      hi = min(A.key_hi[static_cast<int64_t>(bi) * s + q], s);
    }
    const ScoreConst sc =
        score_const<CAP, BIAS>(rsqrtf(static_cast<float>(D)), A.softcap, A.slopes, hh);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_kb; ++j) {
      // S_j in TMEM also means that O += P_{j-1} V_{j-1} is complete
      if (!mbar_wait_warp(s_full, j & 1, status, kSiteAttention)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float x[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32_nowait(tS + lane_off + 32 * c, x + 32 * c);
      tmem_ld_wait();
      const int key0 = k_lo + j * 128;
      // ---- scores in log2 units (without cap and bias the scale is folded
      //      into the exponent's argument below)
      if constexpr (CAP || BIAS) {
        float2 add = make_float2(sc.cap2, sc.cap2);
        const float base = static_cast<float>(key0 - q);
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          float2 y = make_float2(x[2 * i], x[2 * i + 1]);
          if constexpr (BIAS) {
            add.x = fmaf(-sc.slope2, fabsf(base + (2 * i)), sc.cap2);
            add.y = fmaf(-sc.slope2, fabsf(base + (2 * i + 1)), sc.cap2);
          }
          if constexpr (CAP)
            y = __ffma2_rn(cap_r(y, sc.mul), make_float2(-2.f * sc.cap2, -2.f * sc.cap2), add);
          else
            y = __ffma2_rn(y, make_float2(sc.mul, sc.mul), add);
          x[2 * i] = y.x;
          x[2 * i + 1] = y.y;
        }
      }
      // ---- keys [lo, hi) are visible
      if (__any_sync(0xffffffffu, lo > key0 || hi < key0 + 128)) {
        const int first = lo - key0, end = hi - key0;
#pragma unroll
        for (int i = 0; i < 128; ++i) x[i] = (i >= first && i < end) ? x[i] : -INFINITY;
      }
      // ---- running maximum: four chains of three-input maxima, then a tree
      float mc[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int p = 0; p < 62; ++p) mc[p & 3] = fmax3f(mc[p & 3], x[4 + 2 * p], x[5 + 2 * p]);
      float mx = fmaxf(fmax3f(mc[0], mc[1], mc[2]), mc[3]);
      const float mul = CAP || BIAS ? 1.f : sc.mul;
      mx *= mul;  // > 0
      const float m_new = fmaxf(m, mx);
      // a row that has seen nothing yet (m = -infinity) has l = 0 and O = 0
      const bool need = j > 0 && m_new > m + kOptRescale;
      float alpha = 1.f;
      if (j == 0) m = m_new;
      if (need) {
        alpha = fast_exp2(m - m_new);
        l *= alpha;
        m = m_new;
      }
      const float m_use = m == -INFINITY ? 0.f : m;
      // ---- P, its row sum in 32 bits, and P as bf16 for the product
      uint32_t pk[64];
      float2 sm2[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
      const float2 mul2 = make_float2(mul, mul), negm2 = make_float2(-m_use, -m_use);
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        const float2 xi = make_float2(x[2 * i], x[2 * i + 1]);
        const float2 y = CAP || BIAS ? __fadd2_rn(xi, negm2) : __ffma2_rn(xi, mul2, negm2);
        const float2 pv = make_float2(fast_exp2(y.x), fast_exp2(y.y));
        sm2[i & 3] = __fadd2_rn(sm2[i & 3], pv);
        pk[i] = pack_bf16x2(pv.x, pv.y);
      }
      const float2 s01 = __fadd2_rn(__fadd2_rn(sm2[0], sm2[1]), __fadd2_rn(sm2[2], sm2[3]));
      l += s01.x + s01.y;
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          float v[16];
          tmem_ld_32x32b_x16(tO + lane_off + c * 16, v);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i] * alpha);
          tmem_st_32x32b_x16(tO + lane_off + c * 16, w);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = pk[c * 32 + i];
        tmem_st_32x32b_x32(tS + lane_off + c * 32, w);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(p_full);
    }
    if (n_kb > 0 && ok)
      ok = mbar_wait_warp(pv_done, (n_kb - 1) & 1, status, kSiteAttention);
    if (ok && ok_entry) {
      tc_fence_after();
      // a row that sees nothing: O = 0, log-sum-exp = -infinity
      const bool empty = l == 0.f;
      const float inv = empty ? 0.f : 1.f / l;
      uint16_t* orow = A.out + (static_cast<int64_t>(bi) * s + q) * a + hh * D;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float v[32];
        if (n_kb > 0) {
          tmem_ld_32x32b_x32(tO + lane_off + c * 32, v);
        }
        if (q < s && MC_DCHECK(q >= 0 && hh * D + c * 32 + 32 <= a, status, kSiteAttention)) {
          uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 wv = make_uint4(0u, 0u, 0u, 0u);
            if (!empty) {
              wv.x = pack_bf16x2(v[8 * i + 0] * inv, v[8 * i + 1] * inv);
              wv.y = pack_bf16x2(v[8 * i + 2] * inv, v[8 * i + 3] * inv);
              wv.z = pack_bf16x2(v[8 * i + 4] * inv, v[8 * i + 5] * inv);
              wv.w = pack_bf16x2(v[8 * i + 6] * inv, v[8 * i + 7] * inv);
            }
            dst[i] = wv;
          }
        }
      }
      if (q < s)
        A.lse[(static_cast<int64_t>(bi) * A.H + hh) * s + q] =
            empty ? -INFINITY : (m + log2f(l)) * kOptLn2;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, bool CAP, bool BIAS>
int launch_fwd(const uint16_t* qkv, const OptFwdArgs& A, cudaStream_t st) {
  using C = OptFwdCfg<D>;
  const uint64_t a3 = 3ull * A.H * D;
  CUtensorMap tm;
  const uint64_t dims[3] = {a3, static_cast<uint64_t>(A.s), static_cast<uint64_t>(A.b)};
  const uint64_t strides[2] = {a3 * 2, a3 * 2 * static_cast<uint64_t>(A.s)};
  const uint32_t box[3] = {64, 128, 1};
  if (!make_tmap_bf16(&tm, qkv, 3, dims, strides, box)) return MC_ERR_CUDA;
  auto kern = attn_opt_fwd_kernel<D, CAP, BIAS>;
  static PerDeviceInit init;
  const cudaError_t attr = once_per_device(init, [&](long long*) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (attr != cudaSuccess) return MC_ERR_CUDA;
  const unsigned n = static_cast<unsigned>(A.b) * static_cast<unsigned>((A.s + 127) / 128);
  const dim3 grid = A.head_major ? dim3(static_cast<unsigned>(A.H), n, 1u)
                                 : dim3(n, static_cast<unsigned>(A.H), 1u);
  launch_kernel(kern, grid, dim3(kOptFwdThreads), C::kSmem, st, 1, tm, A);
  return cudaGetLastError() == cudaSuccess ? MC_OK : MC_ERR_CUDA;
}

template <int D>
int launch_fwd_d(const uint16_t* qkv, const OptFwdArgs& A, cudaStream_t st) {
  const bool cap = A.softcap > 0.f, bias = A.slopes != nullptr;
  if (cap) return bias ? launch_fwd<D, true, true>(qkv, A, st) : launch_fwd<D, true, false>(qkv, A, st);
  return bias ? launch_fwd<D, false, true>(qkv, A, st) : launch_fwd<D, false, false>(qkv, A, st);
}

}  // namespace

int launch_attention_opt_fwd(const uint16_t* qkv, uint16_t* o, float* lse, int b, int s, int H,
                             int d, const mc_attention_options& opt, int* status,
                             cudaStream_t st) {
  OptFwdArgs A = {};
  A.out = o;
  A.lse = lse;
  A.key_lo = opt.key_lo;
  A.key_hi = opt.key_hi;
  A.tables = opt.tables;
  A.slopes = opt.slopes;
  A.softcap = opt.softcap;
  A.b = b;
  A.s = s;
  A.H = H;
  A.head_major = attention_head_major(static_cast<int64_t>(b) * ((s + 127) / 128), H, 1) ? 1 : 0;
  A.status = status;
  return d == 64 ? launch_fwd_d<64>(qkv, A, st) : launch_fwd_d<128>(qkv, A, st);
}

}  // namespace mc
