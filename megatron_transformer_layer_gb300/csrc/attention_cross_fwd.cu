// Attention to keys of another length, forward (sm_103a, tcgen05):
//   O_i = sum_j P_ij V_j over all keys of the query's sequence, P the softmax.
//
// An item is a block of 128 rows (queries by the heads that share a key head,
// attention_cross.cuh) against the keys of its sequence, in blocks of 256 (the
// last one only half, where 128 keys or fewer are left) with one running
// maximum and sum per row.  384 threads:
//   warp 0       the items into shared memory, and TMA: Q once per item, K
//                blocks into a 2-deep ring, V as 128-key halves into a ring,
//                running on across items
//   warp 1       TMEM and the MMA thread: S = Q K^T, O += P V
//   warps 4..11  softmax, two warps per TMEM lane quarter: a thread takes 128
//                of its row's 256 scores; the two exchange maxima and sums.
//                Warps without a real row (a few new tokens) only signal.
// S_{g+1} is formed while the softmax of block g runs (P has TMEM columns of
// its own), across items too.
// TMEM: S [0, 256), O [256, 256 + D), P [384, 512) (bf16 pairs, 256 keys).
//
// Where items fill the SMs the kernel is persistent, one CTA per SM (D = 128 and many
// keys; for the others see kXPairKeys).  Where they do not (a few queries, many
// keys) a cluster of up to 8 CTAs takes an item, each a share of its keys; they leave
// maxima, sums and O in shared memory and each adds up its part of the rows, read
// from the others' shared memory in the order of their shares (SPLIT).
//
// P is rounded to bf16, by at most 2^-8 of itself: an operand of a tcgen05
// product has the type of the other one, here V's.  The row sums take P before
// that, sums and statistics are 32-bit, and O is rounded once more when stored.
//
// Bound by the tensor cores and by what their products wait for: 4096 queries to 8192
// keys, 64 heads of 128, 750 us on the same inputs again, 800 on others each time =
// 1.47 and 1.37 PFLOP/s, 3,400-3,600 clocks a block of which the products take 2,048;
// loading S, the exchange of maxima and the write of P stand between the softmax of one
// block and the next.  Not kept there: a maximum that lags a block behind (768 us), warps
// of their own for the store of O (784), K in three halves and two tiles of Q (790), two
// CTAs per SM (840), a part of the exponentials as polynomials on the multiply-add units
// (an eighth 768, three 849).  32 x 1 query to lengths up to 8192 (8 key heads, 4.2 MB an
// item): 5.9-6.1 TB/s; equal lengths 6.8, a copy's rate.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attention_cross.cuh"

namespace mc {
namespace {

constexpr int kXFwdThreads = 384;
// The launch gives every thread 168 registers (384 x 168 = 64,512); the softmax
// warpgroups, which hold a row's 128 scores, take what the producer's leaves:
// 128 x 72 + 256 x 216 = 64,512.
constexpr int kXRegsIo = 72, kXRegsSoftmax = 216;
constexpr int kXKeys = 256;  // keys per block
constexpr int kXRing = 4;    // items in shared memory
// Up to so many keys two CTAs per SM take the items (attention_cross_pair.cu).  At
// D = 128 (equal lengths, the same inputs again), 4 x 1037 queries of 64 heads: 128 keys
// 36 us against 80 of this kernel, 256 51 against 68, 333 68 against 95, 512 81 against
// 91, 900 135 against 145, 960 139 against 142, 1024 139 against 136.  (A block of 256
// keys that is not full is selected and exponentiated in full here, so that 128 keys
// take longer than 256.)  One query of each of 32 sequences, 64 heads on 8 key heads:
// 300 keys 12 against 17, 960 25 against 27, ragged lengths up to 8192 120 against 96.
// Where no heads share the keys or items are fewer than SMs one query is slower: 30
// sequences, 900 keys, 32 heads 84 against 74; 12 sequences, 8 heads 18 against 15.  At
// D = 64 always, where P has columns of its own there: 333 keys 52 against 86, 8192 keys
// 552 against 655, one query to 300 (300 sequences, 12 heads) 63 against 144.
constexpr int kXPairKeys = 960;
// O is rescaled only when a row's maximum grows by more than this (log2
// units): P stays below 2^8 and the final division by the sum, taken against
// the same maximum, cancels the difference.
constexpr float kXRescale = 8.0f;

// What every role needs to know of an item.
struct alignas(16) XItem {
  int q0, real, slot;  // its first query row; queries of the block that are real, that have rows
  int halves;          // 128-key halves to visit (-1: no more items)
  int k0, keys;        // first key row, and how many
  int hk;              // key head
  int pad;
};

template <int D>
struct XFwdCfg {
  static constexpr int kChunks = D / 64;         // 128-byte boxes per row
  static constexpr int kQTile = 128 * D * 2;     // Q [128][D] bf16
  static constexpr int kKTile = kXKeys * D * 2;  // K [256][D] bf16
  static constexpr int kChunkBytes = kXKeys * 128;  // one 64-wide d chunk of 256 rows
  static constexpr int kHalf = 128 * D * 2;      // 128 rows of K or V
  static constexpr int kVSlots = D == 64 ? 4 : 2;
  static constexpr int kXch = 2 * 2 * 128 * 4;   // [parity][half][row] floats
  static constexpr int kBars = 38 * 8;           // and 16 bytes of work stealing
  // The dynamic shared memory starts 1024-byte aligned (checked at run time),
  // so no alignment slack is reserved: at D = 128 it would not fit.
  static constexpr int kUsed = kQTile + 2 * kKTile + kVSlots * kHalf + kXch +
                               kXRing * static_cast<int>(sizeof(XItem)) + kBars + kCrossSorted;
  static constexpr int kSmem = kUsed > 116 * 1024 ? kUsed : 116 * 1024;
  static_assert(kUsed <= 227 * 1024, "forward shared memory");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0, kColO = 256, kColP = 384;
  // SPLIT: O of the share in 32 bits, over K's ring; rows padded to spread banks
  static constexpr int kPitch = D + 4;
  static_assert(128 * (kPitch * 4 + 8) <= 2 * kKTile, "a share's O fits into K's ring");
};

struct XFwdArgs {
  CrossArgs c;
  uint16_t* out;
  float* lse;
  int items, steal, sort;
  int shares;  // SPLIT: CTAs of a cluster
};

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kXFwdThreads, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ XFwdArgs F) {
  using C = XFwdCfg<D>;
  constexpr int VS = C::kVSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  const CrossArgs& A = F.c;
  int* status = A.status;
  if (smem_u32(smem) & 1023u) {  // the 128-byte swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) record_error(status, MC_ERR_DEVICE_BOUNDS, kSiteCross);
    return;  // (the same in every CTA of a cluster)
  }
  uint8_t* sQ = smem;
  uint8_t* sK[2] = {smem + C::kQTile, smem + C::kQTile + C::kKTile};
  uint8_t* sV0 = smem + C::kQTile + 2 * C::kKTile;
  float* xch = reinterpret_cast<float*>(sV0 + VS * C::kHalf);
  XItem* items = reinterpret_cast<XItem*>(reinterpret_cast<uint8_t*>(xch) + C::kXch);
  uint64_t* bars = reinterpret_cast<uint64_t*>(items + kXRing);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;    // the item's last S
  uint64_t* k_full = bars + 2;     // [2]
  uint64_t* k_empty = bars + 4;    // [2]  after S
  uint64_t* v_full = bars + 6;     // [4] per half-tile slot (VS used)
  uint64_t* v_empty = bars + 10;   // [4]  after the half's PV steps
  uint64_t* s_full = bars + 14;    // S in TMEM
  uint64_t* s_free = bars + 15;    // the softmax holds S in registers (256 threads)
  uint64_t* p_full = bars + 16;    // P in TMEM (256 threads)
  uint64_t* pv_done = bars + 17;   // O += P V complete
  uint64_t* o_free = bars + 18;    // the item's O is in registers (256 threads)
  uint64_t* drain = bars + 19;
  uint64_t* xbar = bars + 20;      // [4] per lane quarter: the halves' exchange (64 threads)
  uint64_t* it_full = bars + 24;   // [kXRing]
  uint64_t* it_empty = bars + 28;  // [kXRing] read by the MMA thread and the softmax (257)
  uint64_t* steal_bar = bars + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 33);
  void* response = bars + 34;  // 16 bytes, aligned as the items are
  int8_t* order = reinterpret_cast<int8_t*>(bars + 38);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, 256);
    mbar_init(p_full, 256);
    mbar_init(pv_done, 1);
    mbar_init(o_free, 256);
    mbar_init(drain, 1);
    mbar_init(steal_bar, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&xbar[i], 64);
    for (int i = 0; i < kXRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], 257);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // (rows of zeros: what is left in shared memory must not slow the softmax's
  // rescaling down, nothing reads those rows' results)
  cross_clear_rows<D>(sQ, A, threadIdx.x, kXFwdThreads);
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
  const uint32_t tS = tmem + C::kColS, tO = tmem + C::kColO, tP = tmem + C::kColP;

  if (!SPLIT && F.sort) {
    if (warp == 3) cross_order(A, true, order, lane);
    __syncthreads();
  }
  const int share = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  auto item_of = [&](int k) -> XItem {
    XItem it;
    const CrossItem which = cross_item(k, A.KV, A.nqb);
    const int n = !SPLIT && F.sort ? order[which.n] : which.n, at = which.block * A.pq;
    it.hk = which.hk;
    const CrossRows q = cross_queries(A, n), kv = cross_keys(A, n);
    it.q0 = q.first + at;
    it.real = min(max(q.real - at, 0), A.pq);
    it.slot = min(max(q.slot - at, 0), A.pq);
    it.k0 = kv.first;
    it.keys = it.real > 0 ? kv.real : 0;
    if constexpr (SPLIT) {
      const int blocks = (it.keys + kXKeys - 1) / kXKeys;
      const int b0 = blocks * share / F.shares, b1 = blocks * (share + 1) / F.shares;
      it.k0 += b0 * kXKeys;
      it.keys = min(it.keys, b1 * kXKeys) - b0 * kXKeys;
    }
    it.halves = (it.keys + 127) / 128;
    it.pad = 0;
    return it;
  };

  // Every role walks the same items (r) and blocks (g, across items).
  if (warp < 4) {
    setmaxnreg_dec<kXRegsIo>();
    if (warp == 0) {
      if (lane == 0) {
        // -------------------------------------------------------- producer
        int g = 0, u = 0, q_n = 0;  // K blocks, V halves and Q tiles issued
        bool ok = true;
        const uint32_t q_bytes = static_cast<uint32_t>(A.G * A.pq * 128 * C::kChunks);
        // V of a block is loaded after K of the next: what is left to load
        int v_keys = 0, v_row = 0, v_col = 0;
        auto load_v = [&]() {
          for (int h = 0; ok && h * 128 < v_keys; ++h) {
            const int slot = u % VS;
            if (!mbar_wait(&v_empty[slot], ((u / VS) & 1) ^ 1u, status, kSiteCross)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&v_full[slot], C::kHalf);
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_2d(sV0 + slot * C::kHalf + c * 16384, &tm_v, &v_full[slot], v_col + c * 64,
                          v_row + h * 128);
            ++u;
          }
          v_keys = 0;
        };
        // Items are announced one ahead, so that the MMA thread knows the next.
        OptItems steal(response, steal_bar, F.items, F.steal);
        if constexpr (SPLIT) steal.k = static_cast<int>(blockIdx.x) / F.shares;
        XItem cur, next;
        auto announce = [&](int r, XItem& it) -> bool {
          if (steal.more) {
            it = item_of(steal.k);
          } else {
            it = XItem{};
            it.halves = -1;
          }
          const int slot = r % kXRing;
          if (!mbar_wait(&it_empty[slot], ((r / kXRing) & 1) ^ 1u, status, kSiteCross))
            return false;
          items[slot] = it;
          mbar_arrive(&it_full[slot]);
          return true;
        };
        ok = announce(0, cur);
        // (an item's first loads are issued before the next item is asked about)
        auto go_on = [&](int r) -> bool {
          if constexpr (SPLIT) {
            steal.more = false;
          } else if (steal.more) {
            if (!steal.next(status)) return false;
          }
          return announce(r + 1, next);
        };
        for (int r = 0; ok && cur.halves >= 0; ++r, cur = next) {
          // Announcing waits for an earlier item's softmax, which waits for its
          // last V: with empty items in between that V is not left pending.
          if (cur.halves == 0) load_v();
          const bool early = r > 0 || cur.halves == 0;  // (the first item's loads go first)
          if (ok && early) ok = go_on(r);
          for (int j = 0; ok && 2 * j < cur.halves; ++j, ++g) {
            if (j == 0) {
              if (!(ok = mbar_wait(q_empty, (q_n & 1) ^ 1u, status, kSiteCross))) break;
              mbar_arrive_expect_tx(q_full, q_bytes);
              for (int c = 0; c < C::kChunks; ++c)
                cross_load_q(sQ + c * 16384, &tm_q, q_full, A, D, c, cur.hk, cur.q0);
              ++q_n;
            }
            const int ks = g & 1, left = cur.keys - j * kXKeys;
            const int nh = left > 128 ? 2 : 1;
            if (!(ok = mbar_wait(&k_empty[ks], ((g >> 1) & 1) ^ 1u, status, kSiteCross))) break;
            mbar_arrive_expect_tx(&k_full[ks], nh * C::kHalf);
            for (int c = 0; c < C::kChunks; ++c)
              for (int h = 0; h < nh; ++h)
                tma_load_2d(sK[ks] + c * C::kChunkBytes + h * 16384, &tm_k, &k_full[ks],
                            cur.hk * D + c * 64, cur.k0 + j * kXKeys + h * 128);
            if (j == 0 && !early && !(ok = go_on(r))) {
              ++g;
              break;
            }
            load_v();
            v_keys = min(left, kXKeys);
            v_row = cur.k0 + j * kXKeys;
            v_col = cur.hk * D;
          }
        }
        if (ok) load_v();
        if constexpr (!SPLIT) steal.finish(status);
        pdl_launch();  // every load of this CTA is issued
        // Copies still in flight must land before the CTA exits.
        if (q_n > 0) mbar_wait(q_full, (q_n - 1) & 1, status, kSiteCross, 200000000ull, false);
        for (int i = g - 1; i >= 0 && i >= g - 2; --i)
          mbar_wait(&k_full[i & 1], (i >> 1) & 1, status, kSiteCross, 200000000ull, false);
        for (int i = u - 1; i >= 0 && i >= u - VS; --i)
          mbar_wait(&v_full[i % VS], (i / VS) & 1, status, kSiteCross, 200000000ull, false);
      }
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      // The whole warp walks the loop, so that addresses and descriptors stay
      // in uniform registers; one lane issues.
      constexpr uint32_t kIdescQK1 = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t kIdescQK2 = idesc_bf16_f32(128, 256, false, false);
      constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, false, true);
      const bool leader = elect_one();
      // K-major Q and K (1024 B per 8 rows), MN-major V (64-wide d chunks 16 KB apart)
      const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(smem_u32(sK[0]), 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(smem_u32(sV0), 16384, 1024);
      int g = 0, u = 0, n_items = 0;  // blocks and V halves (of the products), items with blocks
      int p_halves = 0;               // the block whose O += P V is still to be issued,
      int p_tail = 128;               // the keys that its last half holds
      bool p_first = false, ok = true;
      auto issue_pv = [&](int gp) -> bool {
        if (!mbar_wait_warp(p_full, gp & 1, status, kSiteCross)) return false;
        // the previous item's O has been read
        if (p_first && n_items > 1 && !mbar_wait_warp(o_free, n_items & 1, status, kSiteCross))
          return false;
        for (int h = 0; h < p_halves; ++h, ++u) {
          const int slot = u % VS;
          if (!mbar_wait_warp(&v_full[slot], (u / VS) & 1, status, kSiteCross)) return false;
          if (h == p_halves - 1 && p_tail < 128)
            cross_clear_tail<D>(sV0 + slot * C::kHalf, p_tail, lane);
          tc_fence_after();
          const uint64_t vd = smem_desc_add(v_desc, slot * C::kHalf);
          const uint32_t acc = !p_first || h > 0 ? 1u : 0u;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              // 16 keys: 8 packed columns of P, 16 rows of 128 B of V
              umma_bf16_ts(tO, tP + (8 * h + kk) * 8, smem_desc_add(vd, kk * 2048), kIdescPV,
                           kk > 0 ? 1u : acc);
            umma_commit(&v_empty[slot]);
          }
        }
        if (leader) umma_commit(pv_done);
        __syncwarp();
        return true;
      };
      for (int r = 0; ok; ++r) {
        const int slot = r % kXRing;
        if (!(ok = mbar_wait_warp(&it_full[slot], (r / kXRing) & 1, status, kSiteCross))) break;
        const int halves = __shfl_sync(0xffffffffu, items[slot].halves, 0);
        const int keys = __shfl_sync(0xffffffffu, items[slot].keys, 0);
        __syncwarp();
        if (leader) mbar_arrive(&it_empty[slot]);
        if (halves < 0) break;
        if (halves == 0 && p_halves > 0) {
          // nothing to overlap with, and the items behind may wait for this one
          if (!(ok = issue_pv(g - 1))) break;
          p_halves = 0;
        }
        for (int j = 0; ok && 2 * j < halves; ++j, ++g) {
          const int ks = g & 1, nh = min(2, halves - 2 * j);
          // S_g before the products of block g - 1, unless those are ready
          // first (an item's first S waits for its Q).
          if (j == 0) {
            if (p_halves > 0) {
              const int first =
                  mbar_wait_first(q_full, n_items & 1, p_full, (g - 1) & 1, status, kSiteCross);
              if (__all_sync(0xffffffffu, first == 2)) {
                if (!(ok = issue_pv(g - 1))) break;
                p_halves = 0;
              }
            }
            if (!(ok = mbar_wait_warp(q_full, n_items & 1, status, kSiteCross))) break;
          }
          if (!(ok = mbar_wait_warp(&k_full[ks], (g >> 1) & 1, status, kSiteCross))) break;
          // S still holds block g - 1 until the softmax has it in registers.
          if (g > 0 && !(ok = mbar_wait_warp(s_free, (g - 1) & 1, status, kSiteCross))) break;
          tc_fence_after();
          const uint64_t kd = smem_desc_add(k_desc, ks * C::kKTile);
          const uint32_t idesc = nh == 2 ? kIdescQK2 : kIdescQK1;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_bf16(tS, smem_desc_add(q_desc, (kk >> 2) * 16384 + (kk & 3) * 32),
                        smem_desc_add(kd, (kk >> 2) * C::kChunkBytes + (kk & 3) * 32), idesc,
                        kk > 0 ? 1u : 0u);
            umma_commit(s_full);
            umma_commit(&k_empty[ks]);
            if (2 * (j + 1) >= halves) umma_commit(q_empty);
          }
          __syncwarp();
          if (p_halves > 0 && !(ok = issue_pv(g - 1))) break;
          p_halves = nh;
          p_tail = 2 * (j + 1) >= halves ? keys - (halves - 1) * 128 : 128;
          p_first = j == 0;
          if (j == 0) ++n_items;
        }
      }
      if (ok && p_halves > 0) issue_pv(g - 1);
      if (leader) {
        umma_commit(drain);
        mbar_wait(drain, 0, status, kSiteCross, 200000000ull, false);
      }
      __syncwarp();
    }
    if constexpr (SPLIT) {
      __syncwarp();
      cluster_sync();  // the shares are in shared memory
    }
  } else {
    // ---------------------------------------------------------- softmax
    setmaxnreg_inc<kXRegsSoftmax>();
    const int quarter = warp & 3;
    const int half = (warp - 4) >> 2;  // keys [128 half, 128 half + 128) of a block
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int my_query = cross_query(A, row), my_head = row - my_query * A.G;
    const float mul = A.scale * kOptLog2e;  // raw scores to log2 units
    bool ok = true;
    // Exchange with the other half of the row (bounded wait on the quarter's
    // barrier); slots alternate by phase so a fast peer never overwrites a
    // value the other has not read.
    int xphase = 0;
    auto offer = [&](float v) {
      xch[(xphase & 1) * 256 + half * 128 + row] = v;
      mbar_arrive(&xbar[quarter]);
    };
    auto take = [&]() -> float {
      if (!mbar_wait(&xbar[quarter], xphase & 1, status, kSiteCross)) ok = false;
      const float peer = xch[(xphase & 1) * 256 + (half ^ 1) * 128 + row];
      ++xphase;
      return peer;
    };
    // The item before, whose O is still in TMEM: its products run during this
    // item's first softmax, and it is stored once they are complete.
    bool pending = false;
    float p_l = 0.f, p_m = 0.f;
    int p_q0 = 0, p_slot = 0, p_hk = 0;
    auto store_item = [&](bool from_tmem) {
      // a row that sees nothing: O = 0, log-sum-exp = -infinity
      const float inv = p_l == 0.f ? 0.f : 1.f / p_l;
      const int64_t head0 = static_cast<int64_t>(p_hk) * A.G;
      // (a warp whose rows all lie behind the sequence only passes O on)
      const bool any = cross_query(A, quarter * 32) < p_slot;
      uint16_t* to[4];  // 4 lanes store 64 bytes of row k of their four
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r4 = quarter * 32 + (lane & ~3) + k;
        const int qi = cross_query(A, r4), hd = r4 - qi * A.G;
        const bool in = qi < p_slot && qi < A.pq &&
                        MC_DCHECK(p_q0 + qi < A.q_rows && head0 + hd < A.H, status, kSiteCross);
        to[k] = in ? F.out + (static_cast<int64_t>(p_q0) + qi) * A.ld_o + (head0 + hd) * D +
                         half * (D / 2) + (lane & 3) * 8
                   : nullptr;
      }
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {  // this thread's half of the row's O
        float v[32] = {};
        if (from_tmem) {
          if (any) tmem_ld_32x32b_x32(tO + lane_off + half * (D / 2) + c * 32, v);
          if (c == D / 64 - 1) {
            tc_fence_before();
            mbar_arrive(o_free);  // the next products may overwrite O
          }
        }
        if (!any) continue;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = p_l == 0.f ? 0u : pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
        transpose_16b_x4(w, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (to[k])
            *reinterpret_cast<uint4*>(to[k] + c * 32) =
                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
      }
      if (half == 0 && my_query < p_slot && my_query < A.pq)
        F.lse[(head0 + my_head) * A.q_rows + p_q0 + my_query] =
            p_l == 0.f ? -INFINITY : (p_m + log2f(p_l)) * kOptLn2;
    };
    int g = 0;
    for (int r = 0; ok; ++r) {
      if (!mbar_wait_warp(&it_full[r % kXRing], (r / kXRing) & 1, status, kSiteCross)) {
        ok = false;
        break;
      }
      const XItem it = items[r % kXRing];
      mbar_arrive(&it_empty[r % kXRing]);
      const int halves = it.halves;
      if (halves < 0) break;
      // a warp without a real row
      const bool idle = cross_query(A, quarter * 32) >= it.real;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; 2 * j < halves; ++j, ++g) {
        if (!ok || !mbar_wait_warp(s_full, g & 1, status, kSiteCross)) {
          ok = false;
          break;
        }
        if (idle) {
          mbar_arrive(s_free);
          // (not before the products of block g - 1, whose P it would announce)
          if (g > 0 && !mbar_wait_warp(pv_done, (g - 1) & 1, status, kSiteCross)) {
            ok = false;
            break;
          }
          if (pending) {
            tc_fence_after();
            store_item(true);
            pending = false;
          }
          mbar_arrive(p_full);
          continue;
        }
        tc_fence_after();
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_ld_32x32b_x32_nowait(tS + lane_off + half * 128 + 32 * c, x + 32 * c);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(s_free);
        // ---- the last block may end inside this half, or before it (S is then
        //      an older one there)
        const int end = it.keys - j * kXKeys - half * 128;
        if (end < 128) {
#pragma unroll
          for (int i = 0; i < 128; ++i) x[i] = i < end ? x[i] : -INFINITY;
        }
        // ---- row maximum: four chains of three-input maxima, then a tree
        float mc[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int p = 0; p < 62; ++p) mc[p & 3] = fmax3f(mc[p & 3], x[4 + 2 * p], x[5 + 2 * p]);
        float mx = fmaxf(fmax3f(mc[0], mc[1], mc[2]), mc[3]);
        offer(mx);
        mx = fmaxf(mx, take());
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        mx *= mul;
        const float m_new = fmaxf(m, mx);
        const bool need = j > 0 && m_new > m + kXRescale;
        float alpha = 1.f;
        if (j == 0) m = m_new;
        if (need) {
          alpha = fast_exp2(m - m_new);
          l *= alpha;
          m = m_new;
        }
        const float m_use = m == -INFINITY ? 0.f : m;
        // ---- P, its row sum in 32 bits, and P as bf16 in registers, while the
        //      products of the block before may still run (in place: pair i of
        //      the bf16 P takes score i's register, which pair i / 2 was the
        //      last to need)
        float2 sm2[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
        const float2 mul2 = make_float2(mul, mul), negm2 = make_float2(-m_use, -m_use);
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          const float2 y = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), mul2, negm2);
          const float2 pv = make_float2(fast_exp2(y.x), fast_exp2(y.y));
          sm2[i & 3] = __fadd2_rn(sm2[i & 3], pv);
          x[i] = __uint_as_float(pack_bf16x2(pv.x, pv.y));  // V's type (see the top)
        }
        const float2 s01 = __fadd2_rn(__fadd2_rn(sm2[0], sm2[1]), __fadd2_rn(sm2[2], sm2[3]));
        l += s01.x + s01.y;
        // The products of block g - 1 have to be complete before O is rescaled
        // or P overwritten.
        if (g > 0 && !mbar_wait_warp(pv_done, (g - 1) & 1, status, kSiteCross)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (pending) {
          store_item(true);
          pending = false;
        }
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll 1
          for (int c = half * (D / 32); c < (half + 1) * (D / 32); ++c) {
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
          for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(x[c * 32 + i]);
          tmem_st_32x32b_x32(tP + lane_off + half * 64 + c * 32, w);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full);
      }
      if (!ok) break;
      const float l0 = p_l, m0 = p_m;
      const int q0 = p_q0, s0 = p_slot, h0 = p_hk;
      if (halves > 0 && !idle) {
        offer(l);
        l += take();  // both halves' sums, taken against the same maximum
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
      }
      p_l = my_query < it.real ? l : 0.f;
      p_m = m;
      p_q0 = it.q0;
      p_slot = it.slot;
      p_hk = it.hk;
      if constexpr (!SPLIT) {
        if (halves > 0) {
          pending = true;
        } else {
          // nothing to see: stored at once (what is pending waits in its TMEM)
          store_item(false);
          p_l = l0, p_m = m0, p_q0 = q0, p_slot = s0, p_hk = h0;
        }
      }
    }
    if constexpr (!SPLIT) {
      if (ok && pending && mbar_wait_warp(pv_done, (g - 1) & 1, status, kSiteCross)) {
        tc_fence_after();
        store_item(true);
      }
    } else {
      // This share's maxima, sums and O (not divided) into shared memory, over K's
      // ring: every product that read it is complete.
      if (g > 0 && !mbar_wait_warp(pv_done, (g - 1) & 1, status, kSiteCross)) ok = false;
      tc_fence_after();
      float* so = reinterpret_cast<float*>(sK[0]);
      float2* ml = reinterpret_cast<float2*>(so + 128 * C::kPitch);
      const bool has = ok && g > 0 && cross_query(A, quarter * 32) < p_slot;
      if (half == 0) ml[row] = has && p_l != 0.f ? make_float2(p_m, p_l) : make_float2(-INFINITY, 0.f);
      if (has) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          float v[32];
          tmem_ld_32x32b_x32(tO + lane_off + half * (D / 2) + c * 32, v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(so + row * C::kPitch + half * (D / 2) + c * 32 + 4 * i) =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      __syncwarp();
      cluster_sync();  // (every thread of every CTA, whatever it met)
      // The rows of the item, dealt to the CTAs: four columns a thread, the shares
      // in their order.
      constexpr int kPer = D / 4;
      const int t = static_cast<int>(threadIdx.x) - 128, col = (t % kPer) * 4;
      for (int rr = share + (t / kPer) * F.shares; rr < p_slot * A.G;
           rr += (256 / kPer) * F.shares) {
        float mx = -INFINITY;
        for (int s = 0; s < F.shares; ++s) mx = fmaxf(mx, ld_cluster_v2(mapa_shared(ml + rr, s)).x);
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < F.shares; ++s) {
          const float2 w2 = ld_cluster_v2(mapa_shared(ml + rr, s));
          const float4 v = ld_cluster_v4(mapa_shared(so + rr * C::kPitch + col, s));
          if (w2.y != 0.f) {  // (a share without keys, or of padding, left nothing)
            const float w = fast_exp2(w2.x - mx);
            sum = fmaf(w, w2.y, sum);
            o.x = fmaf(w, v.x, o.x);
            o.y = fmaf(w, v.y, o.y);
            o.z = fmaf(w, v.z, o.z);
            o.w = fmaf(w, v.w, o.w);
          }
        }
        const float inv = sum != 0.f ? 1.f / sum : 0.f;
        const int qi = cross_query(A, rr), hd = p_hk * A.G + rr - qi * A.G;
        const int64_t q = static_cast<int64_t>(p_q0) + qi;
        if (MC_DCHECK(q < A.q_rows && hd < A.H, status, kSiteCross)) {
          *reinterpret_cast<uint2*>(F.out + q * A.ld_o + static_cast<int64_t>(hd) * D + col) =
              make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
          if (col == 0)
            F.lse[static_cast<int64_t>(hd) * A.q_rows + q] =
                sum != 0.f ? (mx + log2f(sum)) * kOptLn2 : -INFINITY;
        }
      }
    }
  }

  tc_fence_before();
  if constexpr (SPLIT) {
    cluster_sync();  // the others have read this CTA's share
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, bool SPLIT>
int launch_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
               const XFwdArgs& F, int ctas, cudaStream_t st) {
  using C = XFwdCfg<D>;
  auto kern = cross_fwd_kernel<D, SPLIT>;
  static PerDeviceInit init;
  const cudaError_t attr = once_per_device(init, [&](long long*) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (attr != cudaSuccess) return MC_ERR_CUDA;
  const cudaError_t e =
      launch_kernel(kern, dim3(static_cast<unsigned>(ctas)), dim3(kXFwdThreads), C::kSmem, st,
                    SPLIT ? static_cast<unsigned>(F.shares) : 1u, tq, tk, tv, F);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MC_OK : MC_ERR_CUDA;
}

template <int D>
int launch_fwd_d(const uint16_t* q, const uint16_t* k, const uint16_t* v, XFwdArgs& F,
                 cudaStream_t st) {
  const CrossArgs& A = F.c;
  // Shares of an item: as many as SMs are left for, each a key block at least
  // (96 items of 1000 keys, D = 64: 13.5 us one CTA each, 18.8 in pairs that start in
  // two rounds; 32 items of 8192 keys, D = 128: 43.5 us in shares of two, 27.3 of
  // four).
  const int sms = num_sms(), blocks = (A.max_kv + kXKeys - 1) / kXKeys;
  F.shares = 1;
  while (F.shares < 8 && F.items * F.shares * 2 <= sms && F.shares * 2 <= blocks) F.shares *= 2;
  if (F.shares == 1 && (D == 64 || A.max_kv <= kXPairKeys))
    return launch_attention_cross_pair(q, k, v, F.out, F.lse, A, D, st);
  CUtensorMap tq, tk, tv;
  if (!cross_q_map(&tq, q, D, A, A.ld_q) || !cross_kv_map(&tk, k, D, A) ||
      !cross_kv_map(&tv, v, D, A))
    return MC_ERR_CUDA;
  if constexpr (D == 128) {
    if (F.shares == 1) {
      F.sort = cross_sorts(A) && F.items > sms ? 1 : 0;
      F.steal = F.items > 4 * sms || F.sort ? 1 : 0;
      return launch_fwd<D, false>(tq, tk, tv, F, F.steal || F.items < sms ? F.items : sms, st);
    }
  }
  return launch_fwd<D, true>(tq, tk, tv, F, F.items * F.shares, st);
}

}  // namespace

int launch_attention_cross_fwd(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                               uint16_t* o, float* lse, const mc_cross_attention& c, int* status,
                               cudaStream_t st) {
  XFwdArgs F = {};
  F.c = cross_args(c, status);
  F.out = o;
  F.lse = lse;
  F.items = F.c.n * F.c.KV * F.c.nqb;
  return c.head_dim == 64 ? launch_fwd_d<64>(q, k, v, F, st) : launch_fwd_d<128>(q, k, v, F, st);
}

}  // namespace mc
