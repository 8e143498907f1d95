// Attention to keys of another length, forward, two CTAs per SM (sm_103a, tcgen05).
// The items and the mathematics are those of attention_cross_fwd.cu; what differs is
// what hides the time between an item's products: there one CTA keeps the next S
// ahead, here the other CTA of the SM works meanwhile, so that an item's start and
// end (its loads, the store of O) are hidden as well.
//
// A block is 128 keys; of a sequence's last one only as many as there are are
// multiplied (in 16s) and exponentiated (in 32s, D = 128).  256 threads:
//   warp 0      the items into shared memory, and TMA
//   warp 1      TMEM and the MMA thread: S = Q K^T, O += P V
//   warps 4..7  softmax and the store of O: a thread has a row
// TMEM, 256 columns a CTA: S [0, 128), O [128, 128 + D), P (bf16 pairs) in columns of
// its own where there are any (D = 64: [192, 256)), else over S, which it then holds
// until its product is complete.
//
// What bounds it: S, softmax and product of a block are a chain of some 3,000 clocks at
// D = 128, of which the two CTAs overlap two (4 x 1037 queries of 64 heads, the same
// inputs again: 128 keys 36 us, 256 51 us, 512 81 us; two threads to a row, which then
// exchange maxima: 19% slower).  At D = 64, where S runs ahead, no unit is full: 4096
// queries to 8192 keys, 16 heads, issue 46% of the slots, the tensor pipe is active 39%
// of the time, the exponentials' pipe 39%, multiply-adds 23%; what is left are waits
// between a row's softmax and the products (64 heads: 552-568 us, floor 282; a part of
// the exponentials as polynomials, an eighth of them, was 10% slower).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attention_cross.cuh"

namespace mc {
namespace {

constexpr int kPairThreads = 256;
// 128 x 48 + 128 x 208 of the launch's 256 x 128 registers (a row's scores are 128).
constexpr int kPairRegsIo = 48, kPairRegsSoftmax = 208;
constexpr int kPairRing = 4;  // items in shared memory
constexpr float kPairRescale = 8.0f;  // as in attention_cross_fwd.cu

// What every role needs to know of an item.
struct alignas(16) PairItem {
  int q0, real, slot;  // its first query row; queries of the block that are real, that have rows
  int blocks;          // of keys (-1: no more items)
  int k0, keys;        // first key row, and how many
  int hk;              // key head
  int pad;
};

template <int D>
struct PairCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = 128 * D * 2;    // Q [128][D] bf16
  static constexpr int kNQ = D == 64 ? 2 : 1;  // tiles of Q
  // Tiles of 128 rows of K and V come through one ring, in the order of their use.
  // (Five of the half size at D = 128, replaced as they are used: 10% slower.)
  static constexpr int kSlots = D == 64 ? 5 : 2;
  // The dynamic shared memory starts 1024-byte aligned (checked at run time).
  static constexpr int kSmem = (kNQ + kSlots) * kTile +
                               kPairRing * static_cast<int>(sizeof(PairItem)) + 32 * 8 + kCrossSorted;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
  static constexpr uint32_t kTmemCols = 256;
  static constexpr bool kOwnP = D == 64;
  static constexpr uint32_t kColO = 128, kColP = kOwnP ? 192 : 0;
};

struct PairArgs {
  CrossArgs c;
  uint16_t* out;
  float* lse;
  int items, steal, sort;
};

template <int D>
__global__ void __launch_bounds__(kPairThreads, 2)
    cross_pair_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ PairArgs F) {
  using C = PairCfg<D>;
  constexpr int NQ = C::kNQ, NS = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  const CrossArgs& A = F.c;
  int* status = A.status;
  if (smem_u32(smem) & 1023u) {  // the 128-byte swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) record_error(status, MC_ERR_DEVICE_BOUNDS, kSiteCross);
    return;
  }
  uint8_t* sQ = smem;                  // [NQ]
  uint8_t* sR = smem + NQ * C::kTile;  // K and V
  PairItem* items = reinterpret_cast<PairItem*>(sR + NS * C::kTile);
  uint64_t* bars = reinterpret_cast<uint64_t*>(items + kPairRing);
  uint64_t* q_full = bars + 0;     // [NQ]
  uint64_t* q_empty = bars + 2;    // [NQ] the item's last S
  uint64_t* full = bars + 4;       // [NS]
  uint64_t* empty = bars + 9;      // [NS] after S (K), after O += P V (V)
  uint64_t* s_full = bars + 14;    // S in TMEM
  uint64_t* s_free = bars + 15;    // and in registers (4 warps)
  uint64_t* p_full = bars + 16;    // P in TMEM (4 warps)
  uint64_t* pv_done = bars + 17;   // O += P V complete
  uint64_t* drain = bars + 18;
  uint64_t* steal_bar = bars + 19;
  uint64_t* it_full = bars + 20;   // [kPairRing]
  uint64_t* it_empty = bars + 24;  // [kPairRing] read by the MMA thread and the softmax (5)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 28);
  void* response = bars + 30;  // 16 bytes, aligned as the items are
  int8_t* order = reinterpret_cast<int8_t*>(bars + 32);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, 4);
    mbar_init(p_full, 4);
    mbar_init(pv_done, 1);
    mbar_init(drain, 1);
    mbar_init(steal_bar, 1);
    for (int i = 0; i < kPairRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], 5);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // (rows of zeros: what is left in shared memory must not slow the softmax's
  // rescaling down, nothing reads those rows' results)
  for (int i = 0; i < NQ; ++i)
    cross_clear_rows<D>(sQ + i * C::kTile, A, threadIdx.x, kPairThreads);
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // the previous kernel on the stream has completed
  const uint32_t tS = tmem, tO = tmem + C::kColO, tP = tmem + C::kColP;

  if (F.sort) {
    if (warp == 3) cross_order(A, true, order, lane);
    __syncthreads();
  }

  if (warp < 4) {
    setmaxnreg_dec<kPairRegsIo>();
    if (warp == 0) {
      if (lane == 0) {
        // -------------------------------------------------------- producer
        int u = 0, q_n = 0;  // tiles of K and V, and of Q issued
        bool ok = true;
        const uint32_t q_bytes = static_cast<uint32_t>(A.G * A.pq * 128 * C::kChunks);
        OptItems steal(response, steal_bar, F.items, F.steal);
        struct Cur {
          int q0, blocks, k0, hk;
        };
        Cur cur, next;
        auto announce = [&](int r, Cur& c) -> bool {
          PairItem it = {};
          it.blocks = -1;
          if (steal.more) {
            const CrossItem which = cross_item(steal.k, A.KV, A.nqb);
            const int n = F.sort ? order[which.n] : which.n, at = which.block * A.pq;
            const CrossRows q = cross_queries(A, n), kv = cross_keys(A, n);
            it.hk = which.hk;
            it.q0 = q.first + at;
            it.real = min(max(q.real - at, 0), A.pq);
            it.slot = min(max(q.slot - at, 0), A.pq);
            it.k0 = kv.first;
            it.keys = it.real > 0 ? kv.real : 0;
            it.blocks = (it.keys + 127) / 128;
          }
          c = {it.q0, it.blocks, it.k0, it.hk};
          const int slot = r % kPairRing;
          if (!mbar_wait(&it_empty[slot], ((r / kPairRing) & 1) ^ 1u, status, kSiteCross))
            return false;
          items[slot] = it;
          mbar_arrive(&it_full[slot]);
          return true;
        };
        // (an item's first loads are issued before the next item is asked about)
        auto go_on = [&](int r) -> bool {
          if (steal.more && !steal.next(status)) return false;
          return announce(r + 1, next);
        };
        ok = announce(0, cur);
        for (int r = 0; ok && cur.blocks >= 0; ++r, cur = next) {
          if (cur.blocks == 0 && !(ok = go_on(r))) break;
          for (int j = 0; j < cur.blocks; ++j) {
            if (j == 0) {
              const int qb = q_n % NQ;
              if (!(ok = mbar_wait(&q_empty[qb], ((q_n / NQ) & 1) ^ 1u, status, kSiteCross))) break;
              mbar_arrive_expect_tx(&q_full[qb], q_bytes);
              for (int c = 0; c < C::kChunks; ++c)
                cross_load_q(sQ + qb * C::kTile + c * 16384, &tm_q, &q_full[qb], A, D, c, cur.hk,
                             cur.q0);
              ++q_n;
            }
            for (int n = 0; n < 2; ++n, ++u) {  // K, then V
              const int st = u % NS;
              if (!(ok = mbar_wait(&empty[st], ((u / NS) & 1) ^ 1u, status, kSiteCross))) break;
              mbar_arrive_expect_tx(&full[st], C::kTile);
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_2d(sR + st * C::kTile + c * 16384, n == 0 ? &tm_k : &tm_v, &full[st],
                            cur.hk * D + c * 64, cur.k0 + j * 128);
            }
            if (!ok || (j == 0 && !(ok = go_on(r)))) break;
          }
        }
        steal.finish(status);
        pdl_launch();  // every load of this CTA is issued
        // Copies still in flight must land before the CTA exits.
        for (int i = q_n - 1; i >= 0 && i >= q_n - NQ; --i)
          mbar_wait(&q_full[i % NQ], (i / NQ) & 1, status, kSiteCross, 200000000ull, false);
        for (int i = u - 1; i >= 0 && i >= u - NS; --i)
          mbar_wait(&full[i % NS], (i / NS) & 1, status, kSiteCross, 200000000ull, false);
      }
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, false, true);
      const bool leader = elect_one();
      // K-major Q and K (1024 B per 8 rows), MN-major V (64-wide d chunks 16 KB apart)
      const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(smem_u32(sR), 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(smem_u32(sR), 16384, 1024);
      int g = 0, n_items = 0;  // blocks whose S is issued, items with blocks
      int p_keys = 0;          // of the block whose O += P V is still to be issued
      bool p_first = false;    // as the first one of its item
      bool ok = true;
      auto issue_pv = [&](int gp) -> bool {
        const int u = 2 * gp + 1, st = u % NS;
        if (!mbar_wait_warp(&full[st], (u / NS) & 1, status, kSiteCross)) return false;
        // steps of 16 keys; P is 0 for those behind the sequence, V may be anything there
        const int steps = (p_keys + 15) >> 4;
        if (p_keys < steps * 16)
          cross_clear_tail<D>(sR + st * C::kTile, p_keys, lane, steps * 16);
        if (!mbar_wait_warp(p_full, gp & 1, status, kSiteCross)) return false;
        tc_fence_after();
        const uint64_t vd = smem_desc_add(v_desc, st * C::kTile);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            if (kk < steps)
              umma_bf16_ts(tO, tP + kk * 8, smem_desc_add(vd, kk * 2048), kIdescPV,
                           kk > 0 || !p_first ? 1u : 0u);
          umma_commit(&empty[st]);
          umma_commit(pv_done);
        }
        __syncwarp();
        p_keys = 0;
        return true;
      };
      for (int r = 0; ok; ++r) {
        const int slot = r % kPairRing;
        if (!(ok = mbar_wait_warp(&it_full[slot], (r / kPairRing) & 1, status, kSiteCross))) break;
        const int blocks = __shfl_sync(0xffffffffu, items[slot].blocks, 0);
        const int keys = __shfl_sync(0xffffffffu, items[slot].keys, 0);
        __syncwarp();
        if (leader) mbar_arrive(&it_empty[slot]);
        if (blocks < 0) break;
        const int qb = n_items % NQ;
        for (int j = 0; j < blocks; ++j, ++g) {
          const int left = min(keys - j * 128, 128);
          const int u = 2 * g, st = u % NS;
          if (j == 0 &&
              !(ok = mbar_wait_warp(&q_full[qb], (n_items / NQ) & 1, status, kSiteCross)))
            break;
          if (!(ok = mbar_wait_warp(&full[st], (u / NS) & 1, status, kSiteCross))) break;
          // S is in registers; where P lies over it, the products have read P
          if (g > 0 && !(ok = C::kOwnP
                                  ? mbar_wait_warp(s_free, (g - 1) & 1, status, kSiteCross)
                                  : mbar_wait_warp(pv_done, (g - 1) & 1, status, kSiteCross)))
            break;
          tc_fence_after();
          // (as many columns as there are keys, in 16s)
          const uint32_t idesc = idesc_bf16_f32(128, (left + 15) & ~15, false, false);
          const uint64_t qd = smem_desc_add(q_desc, qb * C::kTile);
          const uint64_t kd = smem_desc_add(k_desc, st * C::kTile);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
              umma_bf16(tS, smem_desc_add(qd, off), smem_desc_add(kd, off), idesc, kk > 0 ? 1u : 0u);
            }
            umma_commit(s_full);
            umma_commit(&empty[st]);
            if (j == blocks - 1) umma_commit(&q_empty[qb]);
          }
          __syncwarp();
          if constexpr (C::kOwnP) {
            if (p_keys > 0 && !(ok = issue_pv(g - 1))) break;
          }
          p_keys = left;
          p_first = j == 0;
          if (!C::kOwnP || j == blocks - 1) {
            if (!(ok = issue_pv(g))) break;
          }
        }
        if (blocks > 0) ++n_items;
      }
      if (leader) {
        umma_commit(drain);
        mbar_wait(drain, 0, status, kSiteCross, 200000000ull, false);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- softmax
    setmaxnreg_inc<kPairRegsSoftmax>();
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int my_query = cross_query(A, row), my_head = row - my_query * A.G;
    const int warp_query = cross_query(A, quarter * 32);
    const float mul = A.scale * kOptLog2e;  // raw scores to log2 units
    bool ok = true;
    int g = 0;
    for (int r = 0; ok; ++r) {
      const int slot = r % kPairRing;
      if (!mbar_wait_warp(&it_full[slot], (r / kPairRing) & 1, status, kSiteCross)) break;
      const PairItem it = items[slot];
      mbar_arrive_warp(&it_empty[slot], lane);
      if (it.blocks < 0) break;
      const bool idle = warp_query >= it.real;  // a warp without a real row
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < it.blocks; ++j, ++g) {
        if (!(ok = mbar_wait_warp(s_full, g & 1, status, kSiteCross))) break;
        if (idle) {
          if constexpr (C::kOwnP) mbar_arrive_warp(s_free, lane);
          // (not before the products of block g - 1, whose P it would announce)
          if (g > 0 && !(ok = mbar_wait_warp(pv_done, (g - 1) & 1, status, kSiteCross))) break;
          mbar_arrive_warp(p_full, lane);
          continue;
        }
        tc_fence_after();
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_ld_32x32b_x32_nowait(tS + lane_off + 32 * c, x + 32 * c);
        tmem_ld_wait();
        tc_fence_before();
        if constexpr (C::kOwnP) mbar_arrive_warp(s_free, lane);
        const int end = it.keys - j * 128;
        // Where S is held until the product, a last block does no more than it has
        // keys for (333 keys, D = 128: 67 us against 71; at D = 64, where S is free
        // at once, the branch costs more than it saves: 8192 keys 6% more).
        float mx = -INFINITY;
        if (C::kOwnP || end >= 128) {
          if (C::kOwnP && end < 128) {
#pragma unroll
            for (int i = 0; i < 128; ++i) x[i] = i < end ? x[i] : -INFINITY;
          }
          // row maximum: four chains of three-input maxima, then a tree
          float mc[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int p = 0; p < 62; ++p) mc[p & 3] = fmax3f(mc[p & 3], x[4 + 2 * p], x[5 + 2 * p]);
          mx = fmaxf(fmax3f(mc[0], mc[1], mc[2]), mc[3]);
        } else {
          // (S holds nothing of use behind the keys)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (32 * c >= end) break;
            float* y = x + 32 * c;
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = 32 * c + i < end ? y[i] : -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx = fmax3f(mx, y[i], y[i + 1]);
          }
        }
        mx *= mul;
        const bool need = j > 0 && mx > m + kPairRescale;
        float alpha = 1.f;
        if (j == 0) m = mx;
        if (need) {
          alpha = fast_exp2(m - mx);
          l *= alpha;
          m = mx;
        }
        // ---- P and its row sum in 32 bits
        const float m_use = m == -INFINITY ? 0.f : m;
        float2 sm2[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
        const float2 mul2 = make_float2(mul, mul), negm2 = make_float2(-m_use, -m_use);
        // (in place: pair i of the bf16 P takes score i's register, which pair i / 2 was
        // the last to need)
        auto exp_pair = [&](int i) {
          const float2 y = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), mul2, negm2);
          const float2 pv = make_float2(fast_exp2(y.x), fast_exp2(y.y));
          sm2[i & 3] = __fadd2_rn(sm2[i & 3], pv);
          x[i] = __uint_as_float(pack_bf16x2(pv.x, pv.y));  // V's type (see attention_cross_fwd.cu)
        };
        auto put = [&](int c) {  // 32 keys' P
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(x[16 * c + i]);
          tmem_st_32x32b_x16(tP + lane_off + c * 16, w);
        };
        auto rescale = [&]() {
          tc_fence_after();
          if (!__any_sync(0xffffffffu, need)) return;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            float v[16];
            tmem_ld_32x32b_x16(tO + lane_off + c * 16, v);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i] * alpha);
            tmem_st_32x32b_x16(tO + lane_off + c * 16, w);
          }
        };
        if constexpr (C::kOwnP) {
#pragma unroll
          for (int i = 0; i < 64; ++i) exp_pair(i);
          // The products of block g - 1 have to be complete before O is rescaled or P
          // overwritten (where P lies over S they are).
          if (g > 0 && !(ok = mbar_wait_warp(pv_done, (g - 1) & 1, status, kSiteCross))) break;
          rescale();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(x[c * 32 + i]);
            tmem_st_32x32b_x32(tP + lane_off + c * 32, w);
          }
        } else {
          rescale();
          if (end >= 128) {
#pragma unroll
            for (int i = 0; i < 64; ++i) exp_pair(i);
#pragma unroll
            for (int c = 0; c < 4; ++c) put(c);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (32 * c >= end) break;
#pragma unroll
              for (int i = 0; i < 16; ++i) exp_pair(16 * c + i);
              put(c);
            }
          }
        }
        const float2 s01 = __fadd2_rn(__fadd2_rn(sm2[0], sm2[1]), __fadd2_rn(sm2[2], sm2[3]));
        l += s01.x + s01.y;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(p_full, lane);
      }
      if (!ok) break;
      // ---- the item's O
      if (it.blocks > 0 && !(ok = mbar_wait_warp(pv_done, (g - 1) & 1, status, kSiteCross))) break;
      if (warp_query >= it.slot) continue;
      tc_fence_after();
      if (my_query >= it.real) l = 0.f;
      // a row that sees nothing: O = 0, log-sum-exp = -infinity
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t head0 = static_cast<int64_t>(it.hk) * A.G;
      uint16_t* to[4];  // 4 lanes store 64 bytes of row k of their four
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r4 = quarter * 32 + (lane & ~3) + k;
        const int qi = cross_query(A, r4), hd = r4 - qi * A.G;
        const bool in = qi < it.slot && qi < A.pq &&
                        MC_DCHECK(it.q0 + qi < A.q_rows && head0 + hd < A.H, status, kSiteCross);
        to[k] = in ? F.out + (static_cast<int64_t>(it.q0) + qi) * A.ld_o + (head0 + hd) * D +
                         (lane & 3) * 8
                   : nullptr;
      }
#pragma unroll 1  // (unrolled, 128 keys take 2 us more: instructions missed)
      for (int c = 0; c < D / 32; ++c) {
        float v[32] = {};
        if (it.blocks > 0) tmem_ld_32x32b_x32(tO + lane_off + c * 32, v);
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = l == 0.f ? 0u : pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
        transpose_16b_x4(w, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (to[k])
            *reinterpret_cast<uint4*>(to[k] + c * 32) =
                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
      }
      tc_fence_before();  // (O is overwritten behind the next P)
      if (my_query < it.slot && my_query < A.pq)
        F.lse[(head0 + my_head) * A.q_rows + it.q0 + my_query] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * kOptLn2;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D>
int launch_pair(const uint16_t* q, const uint16_t* k, const uint16_t* v, PairArgs& F,
                cudaStream_t st) {
  using C = PairCfg<D>;
  const CrossArgs& A = F.c;
  CUtensorMap tq, tk, tv;
  if (!cross_q_map(&tq, q, D, A, A.ld_q) || !cross_kv_map(&tk, k, D, A) ||
      !cross_kv_map(&tv, v, D, A))
    return MC_ERR_CUDA;
  auto kern = cross_pair_kernel<D>;
  static PerDeviceInit init;
  const cudaError_t attr = once_per_device(init, [&](long long*) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (attr != cudaSuccess) return MC_ERR_CUDA;
  const int ctas = 2 * num_sms();
  F.sort = cross_sorts(A) && F.items > ctas ? 1 : 0;
  F.steal = F.items > 2 * ctas || F.sort ? 1 : 0;
  const int grid = F.steal || F.items < ctas ? F.items : ctas;
  const cudaError_t e = launch_kernel(kern, dim3(static_cast<unsigned>(grid)), dim3(kPairThreads),
                                      C::kSmem, st, 1u, tq, tk, tv, F);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MC_OK : MC_ERR_CUDA;
}

}  // namespace

int launch_attention_cross_pair(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                uint16_t* o, float* lse, const CrossArgs& c, int d,
                                cudaStream_t st) {
  PairArgs F = {};
  F.c = c;
  F.out = o;
  F.lse = lse;
  F.items = c.n * c.KV * c.nqb;
  return d == 64 ? launch_pair<64>(q, k, v, F, st) : launch_pair<128>(q, k, v, F, st);
}

}  // namespace mc
