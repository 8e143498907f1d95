// Attention to keys of another length, backward (sm_103a, tcgen05).  With
// P = exp(z - lse), z = scale Q K^T and delta = rowsum(dO O):
//   dV = P^T dO,  dP = dO V^T,  dz = P (dP - delta),
//   dQ = scale dz K,  dK = scale dz^T Q,
// dK and dV summed over the query heads that share a key head: those are rows
// of the same blocks (attention_cross.cuh), so the products sum them.
//
//   delta: one pass over O and dO; the dkdv kernel forms that of sequences of up to 128
//          keys itself (and there is no pass where the bound on the keys is 128 or less).
//   dkdv:  a block of 128 keys against its sequence's blocks of queries,
//          accumulates dV and dK and writes each block pair's dz^T tile as bf16.
//   dq:    a block of queries: the product of its tiles with K (bound by the
//          tiles' traffic, against three products if the scores were formed
//          again).
// Key heads are taken in groups whose tiles fit the workspace.
//
// 4096 queries to 8192 keys, 16 heads of 128: delta 10 us, dkdv 490-500 (4,500 clocks a
// pair of blocks; its four products are 2,048 at the tensor pipe's rate, and some 3,100
// with their operands of 128 x 128 out of shared memory, which the loads and the tile's
// way out share, about 320 KB a pair: what is beyond is the chain of S^T, P, dP and dz),
// dq 180 (6 TB/s); heads of 64: 533 us in all, floor 176.  Nine packed sequences of up to
// 700 queries of 64 heads and 900 keys of 8: 25 (5.4 TB/s), 229-235 and 78 us; the tiles
// are 340 of dkdv's 570 MB and most of dq's.
//
// P and dz are rounded to bf16, each by at most 2^-8 of itself: an operand of a
// tcgen05 product has the type of the other one, dO's, Q's and K's.  dK and dQ
// take the same rounded dz.  dz itself is formed in 32 bits from the unrounded P;
// sums and accumulators are 32-bit and dQ, dK and dV are rounded once more when
// stored.  delta of a sequence of more than 128 keys is formed from the stored bf16 O, of
// a shorter one from P and dP: its own length decides, not the call's bound or the others.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attention_cross.cuh"

namespace mc {
namespace {

constexpr int64_t kXTileBytes = 128 * 128 * 2;  // one bf16 dz^T tile (128 keys x 128 rows)

struct XBwdArgs {
  CrossArgs c;
  uint16_t *dq, *dk, *dv;
  const float* lse;
  const float* delta;
  uint8_t* tiles;
  int hk0, heads;      // the key heads of this launch
  int kv_items, q_items;
  int shares;          // SPLIT: CTAs of a cluster
  int kv_steal, q_steal;
  int sort;
};

// Tile (query block, key block) of a (sequence, key head) in the workspace.
__device__ __forceinline__ int64_t cross_tile(const XBwdArgs& B, int n, int hk, int qb, int kb) {
  return ((static_cast<int64_t>(n) * B.heads + (hk - B.hk0)) * B.c.nqb + qb) * B.c.nkb + kb;
}

// ---------------------------------------------------------------- delta
// D/8 threads share a (row, head), each loading 16 bytes of O and of dO, four
// of them per thread with all loads issued first.
constexpr int kXDeltaThreads = 256;
constexpr int kXDeltaPasses = 4;

template <int D>
__global__ void __launch_bounds__(kXDeltaThreads)
    cross_delta_kernel(const uint16_t* __restrict__ o, const uint16_t* __restrict__ dout,
                       float* __restrict__ delta, int rows, int H, int64_t ld) {
  pdl_wait();  // the previous kernel on the stream has completed
  pdl_launch();
  constexpr int TPR = D / 8;                 // threads per (row, head)
  constexpr int RPP = kXDeltaThreads / TPR;  // of them per pass of the block
  const int sub = static_cast<int>(threadIdx.x) % TPR;
  const int64_t all = static_cast<int64_t>(rows) * H;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * RPP * kXDeltaPasses + threadIdx.x / TPR;
  uint4 xo[kXDeltaPasses], xd[kXDeltaPasses];
  int64_t to[kXDeltaPasses];
#pragma unroll
  for (int p = 0; p < kXDeltaPasses; ++p) {
    const int64_t r = r0 + p * RPP;  // r = row * H + head
    xo[p] = make_uint4(0u, 0u, 0u, 0u);
    xd[p] = make_uint4(0u, 0u, 0u, 0u);
    to[p] = -1;
    if (r < all) {
      const int64_t row = r / H;
      const int hd = static_cast<int>(r - row * H);
      const int64_t off = row * ld + static_cast<int64_t>(hd) * D + sub * 8;
      xo[p] = __ldg(reinterpret_cast<const uint4*>(o + off));
      xd[p] = __ldg(reinterpret_cast<const uint4*>(dout + off));
      to[p] = static_cast<int64_t>(hd) * rows + row;
    }
  }
#pragma unroll
  for (int p = 0; p < kXDeltaPasses; ++p) {
    float acc = bf16_lo(xo[p].x) * bf16_lo(xd[p].x) + bf16_hi(xo[p].x) * bf16_hi(xd[p].x) +
                bf16_lo(xo[p].y) * bf16_lo(xd[p].y) + bf16_hi(xo[p].y) * bf16_hi(xd[p].y) +
                bf16_lo(xo[p].z) * bf16_lo(xd[p].z) + bf16_hi(xo[p].z) * bf16_hi(xd[p].z) +
                bf16_lo(xo[p].w) * bf16_lo(xd[p].w) + bf16_hi(xo[p].w) * bf16_hi(xd[p].w);
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (sub == 0 && to[p] >= 0) delta[to[p]] = acc;
  }
}

// ---------------------------------------------------------------- dK, dV
// What every role needs to know of an item: a block of keys.
struct alignas(16) XKvItem {
  int k0, real, slot;  // its first key row; keys of the block that are real, that have rows
  int count;           // blocks of queries (-1: no more items)
  int q0, queries;     // the sequence's first query row, and its real queries
  int n, hk, kb;
  int first;           // its first block of queries
  int whole;           // it holds all keys of its sequence
  int pad;
};
constexpr int kXKvRing = 4;
constexpr int kXKvThreads = 640;
// 128 x 56 + 512 x 104 of the launch's 640 x 96 registers.
constexpr int kXKvRegsIo = 56, kXKvRegsCompute = 104;
constexpr int kXKvWarps = 16;  // compute warps

template <int D>
struct XKvCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = 128 * D * 2;
  // K, V, the Q_i and dO_i stages (apart, Q_i first: S^T_{i+1} runs ahead of
  // the products of block i), the dz^T tile for its bulk store, lse / delta
  // [2][128], items, barriers.  The dynamic shared memory starts 1024-byte
  // aligned (checked at run time).
  static constexpr int kQ = D == 64 ? 3 : 2, kdO = 2;
  static constexpr int kUsed = (2 + kQ + kdO) * kTile + static_cast<int>(kXTileBytes) +
                               4 * 128 * 4 + kXKvRing * static_cast<int>(sizeof(XKvItem)) + 40 * 8 +
                               kCrossSorted;
  // one CTA per SM: it takes all 512 TMEM columns
  static constexpr int kSmem = kUsed > 116 * 1024 ? kUsed : 116 * 1024;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kUsed <= 227 * 1024, "dkdv kernel shared memory");
  // SPLIT: the share's sums in 32 bits, rows padded to spread banks
  static constexpr int kPitch = D + 4;
  static_assert(2 * 128 * kPitch * 4 <= (2 + kQ + kdO) * kTile, "a share's sums fit");
};

// Persistent: one CTA per SM walks the (key block, key head) items, each against
// the sequence's blocks of queries (i; g counts them across items).  640 threads:
// warp 0 loads, warp 1 issues, warp 2 stores dz^T tiles, warps 4..19 compute.
// TMEM: S^T [0, 128), dP^T [128, 256), dV [256, 256 + D), dK [384, 384 + D).
// Per block i of queries:
//   MMA      S^T_i = K Q_i^T (as soon as the compute warps hold S^T_{i-1} in
//            registers), then dV += P^T_{i-1} dO_{i-1}, dK += dz^T_{i-1} Q_{i-1},
//            then (those done) dP^T_i = V dO_i^T.
//   compute  P^T from S^T_i while the products above run, then dz^T from dP^T_i.
// A compute thread owns one key row and 32 query columns: the 16 queries of
// group g (dP^T columns [16g, 16g + 16)) leave P at columns [16g, 16g + 8) and
// dz at [16g + 8, 16g + 16), over columns that the thread itself has read.
// An item's dV and dK are stored during the next item's first block: its
// S^T and weights run meanwhile, as do the loads of its K and V.
//
// Where key blocks do not fill the SMs (few key heads) a cluster of up to 8 CTAs
// takes an item, each a share of its queries, and adds up its part of the rows of
// dV and dK from all shares, read in their order from the others' shared memory
// (SPLIT; 2048 queries to 4096 keys, 16 heads on 2 key heads, both passes 141 us
// against 262).
template <int D, bool SPLIT, bool WHOLE>
__global__ void __launch_bounds__(kXKvThreads, 1)
    cross_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_do,
                      const __grid_constant__ XBwdArgs B) {
  using C = XKvCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const CrossArgs& A = B.c;
  int* status = A.status;
  if (smem_u32(smem) & 1023u) {  // the 128-byte swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) record_error(status, MC_ERR_DEVICE_BOUNDS, kSiteCross);
    return;
  }
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::kTile;
  uint8_t* sQ = smem + 2 * C::kTile;             // [kQ]
  uint8_t* sdO = smem + (2 + C::kQ) * C::kTile;  // [kdO]
  uint8_t* sDs = sdO + C::kdO * C::kTile;        // dz^T tile image (swizzled), 32 KB
  float* sL = reinterpret_cast<float*>(sDs + kXTileBytes);  // [2][128] lse * log2(e)
  float* sD = sL + 256;                                      // [2][128] delta
  XKvItem* items = reinterpret_cast<XKvItem*>(sD + 256);
  uint64_t* bars = reinterpret_cast<uint64_t*>(items + kXKvRing);
  uint64_t* k_full = bars + 0;
  uint64_t* k_empty = bars + 1;    // the item's last S^T
  uint64_t* v_full = bars + 2;
  uint64_t* v_empty = bars + 3;    // the item's last dP^T
  uint64_t* q_full = bars + 4;     // [kQ]
  uint64_t* q_empty = bars + 7;    // [kQ]  after the products
  uint64_t* do_full = bars + 10;   // [kdO]
  uint64_t* do_empty = bars + 12;  // [kdO] after the products
  uint64_t* s_full = bars + 14;    // S^T_i in TMEM
  uint64_t* s_free = bars + 15;    // compute warps hold S^T_i in registers (16 warps)
  uint64_t* dp_full = bars + 16;   // dP^T_i in TMEM
  uint64_t* p_full = bars + 17;    // P^T_i, dz^T_i in TMEM (16 warps)
  uint64_t* acc_done = bars + 18;  // dV, dK products of block i complete
  uint64_t* drain = bars + 19;
  uint64_t* lse_ready = bars + 20;  // [2] (4 warps)
  uint64_t* it_full = bars + 22;    // [kXKvRing]
  uint64_t* it_empty = bars + 26;   // [kXKvRing] read by MMA, tile and compute warps (18)
  uint64_t* steal_bar = bars + 30;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 31);
  void* response = bars + 32;     // 16 bytes, aligned as the items are
  uint64_t* ds_full = bars + 34;  // the dz^T tile of block i is in sDs (16 warps)
  uint64_t* ds_free = bars + 35;  // its bulk store has read sDs
  uint64_t* meet_bar = bars + 36;  // [4] per group: sums over the keys (4 warps)
  int8_t* order = reinterpret_cast<int8_t*>(bars + 40);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(&meet_bar[i], 4);
    mbar_init(k_full, 1);
    mbar_init(k_empty, 1);
    mbar_init(v_full, 1);
    mbar_init(v_empty, 1);
    for (int i = 0; i < C::kQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < C::kdO; ++i) {
      mbar_init(&do_full[i], 1);
      mbar_init(&do_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&lse_ready[i], 4);
    mbar_init(ds_full, kXKvWarps);
    mbar_init(ds_free, 1);
    mbar_init(s_full, 1);
    mbar_init(s_free, kXKvWarps);
    mbar_init(dp_full, 1);
    mbar_init(p_full, kXKvWarps);
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    mbar_init(steal_bar, 1);
    for (int i = 0; i < kXKvRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], 2 + kXKvWarps);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_do);
  }
  // (rows that no box fills take part in the products: they stay zeros)
  for (int i = 0; i < C::kQ + C::kdO; ++i)
    cross_clear_rows<D>(sQ + i * C::kTile, A, threadIdx.x, kXKvThreads);
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
  const uint32_t tS = tmem, tdP = tmem + 128, tdV = tmem + 256, tdK = tmem + 384;

  if (!SPLIT && B.sort) {
    if (warp == 3) cross_order(A, false, order, lane);
    __syncthreads();
  }
  const int share = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  auto item_of = [&](int k) -> XKvItem {
    XKvItem it = {};
    const CrossItem which = cross_item(k, B.heads, A.nkb);
    it.n = !SPLIT && B.sort ? order[which.n] : which.n;
    it.hk = B.hk0 + which.hk;
    it.kb = which.block;
    const CrossRows q = cross_queries(A, it.n), kv = cross_keys(A, it.n);
    it.k0 = kv.first + it.kb * 128;
    it.real = min(max(kv.real - it.kb * 128, 0), 128);
    it.slot = min(max(kv.slot - it.kb * 128, 0), 128);
    it.whole = kv.real <= 128 ? 1 : 0;
    it.q0 = q.first;
    it.queries = q.real;
    it.count = it.real > 0 ? (q.real + A.pq - 1) / A.pq : 0;
    if constexpr (SPLIT) {
      it.first = it.count * share / B.shares;
      it.count = it.count * (share + 1) / B.shares - it.first;
    }
    return it;
  };

  if (warp < 4) {
    setmaxnreg_dec<kXKvRegsIo>();
    if (warp == 0) {
      if (lane == 0) {
        // -------------------------------------------------------- producer
        int g = 0, n = 0;  // query blocks and items (with blocks) loaded
        int q_n = 0, do_n = 0;
        bool ok = true, v_loaded = true;
        const uint32_t q_bytes = static_cast<uint32_t>(A.G * A.pq * 128 * C::kChunks);
        OptItems steal(response, steal_bar, B.kv_items, B.kv_steal);
        if constexpr (SPLIT) steal.k = static_cast<int>(blockIdx.x) / B.shares;
        struct Cur {
          int k0, count, q0, hk;
        };
        Cur cur, next;
        auto announce = [&](int r, Cur& c) -> bool {
          XKvItem it = {};
          it.count = -1;
          if (steal.more) it = item_of(steal.k);
          c = {it.k0, it.count, it.q0 + it.first * A.pq, it.hk};
          const int slot = r % kXKvRing;
          if (!mbar_wait(&it_empty[slot], ((r / kXKvRing) & 1) ^ 1u, status, kSiteCross))
            return false;
          items[slot] = it;
          mbar_arrive(&it_full[slot]);
          return true;
        };
        ok = announce(0, cur);
        // (an item's first loads are issued before the next item is asked about)
        auto go_on = [&](int r) -> bool {
          if constexpr (SPLIT)
            steal.more = false;
          else if (steal.more && !steal.next(status))
            return false;
          return announce(r + 1, next);
        };
        for (int r = 0; ok && cur.count >= 0; ++r, cur = next) {
          const bool early = r > 0 || cur.count == 0;  // (the first item's loads go first)
          if (early && !(ok = go_on(r))) break;
          for (int i = 0; ok && i < cur.count; ++i, ++g) {
            if (i == 0) {
              if (!(ok = mbar_wait(k_empty, (n & 1) ^ 1u, status, kSiteCross))) break;
              mbar_arrive_expect_tx(k_full, C::kTile);
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_2d(sK + c * 16384, &tm_k, k_full, cur.hk * D + c * 64, cur.k0);
              v_loaded = false;
            }
            const int row = cur.q0 + i * A.pq;
            const int qs = g % C::kQ, ds = g % C::kdO;
            if (!(ok = mbar_wait(&q_empty[qs], ((g / C::kQ) & 1) ^ 1u, status, kSiteCross))) break;
            mbar_arrive_expect_tx(&q_full[qs], q_bytes);
            for (int c = 0; c < C::kChunks; ++c)
              cross_load_q(sQ + qs * C::kTile + c * 16384, &tm_q, &q_full[qs], A, D, c, cur.hk, row);
            ++q_n;
            if (!(ok = mbar_wait(&do_empty[ds], ((g / C::kdO) & 1) ^ 1u, status, kSiteCross)))
              break;
            mbar_arrive_expect_tx(&do_full[ds], q_bytes);
            for (int c = 0; c < C::kChunks; ++c)
              cross_load_q(sdO + ds * C::kTile + c * 16384, &tm_do, &do_full[ds], A, D, c, cur.hk,
                           row);
            ++do_n;
            if (i == 0) {
              if (!(ok = mbar_wait(v_empty, (n & 1) ^ 1u, status, kSiteCross))) break;
              mbar_arrive_expect_tx(v_full, C::kTile);
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_2d(sV + c * 16384, &tm_v, v_full, cur.hk * D + c * 64, cur.k0);
              v_loaded = true;
              ++n;
              if (!early && !(ok = go_on(r))) break;
            }
          }
        }
        if constexpr (!SPLIT) steal.finish(status);
        pdl_launch();  // every load of this CTA is issued
        // Copies still in flight must land before the CTA exits.
        const int kn = v_loaded ? n : n + 1;  // K tiles issued
        if (kn > 0) mbar_wait(k_full, (kn - 1) & 1, status, kSiteCross, 200000000ull, false);
        if (n > 0) mbar_wait(v_full, (n - 1) & 1, status, kSiteCross, 200000000ull, false);
        for (int i = q_n - 1; i >= 0 && i >= q_n - C::kQ; --i)
          mbar_wait(&q_full[i % C::kQ], (i / C::kQ) & 1, status, kSiteCross, 200000000ull, false);
        for (int i = do_n - 1; i >= 0 && i >= do_n - C::kdO; --i)
          mbar_wait(&do_full[i % C::kdO], (i / C::kdO) & 1, status, kSiteCross, 200000000ull,
                    false);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      // The whole warp walks the loop, so that addresses and descriptors stay
      // in uniform registers; one lane issues.
      constexpr uint32_t kIdescSq = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t kIdescAcc = idesc_bf16_f32(128, D, false, true);
      constexpr int kLead = 6;
      const bool leader = elect_one();
      const uint64_t k_desc = smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(smem_u32(sV), 16, 1024);
      // Q_i and dO_i, K-major (S, dP) and MN-major (dK, dV)
      const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t do_desc = smem_desc_sw128(smem_u32(sdO), 16, 1024);
      const uint64_t qt_desc = smem_desc_sw128(smem_u32(sQ), 16384, 1024);
      const uint64_t dot_desc = smem_desc_sw128(smem_u32(sdO), 16384, 1024);
      int g = 0, n = 0;     // blocks, items with blocks
      bool pend = false;    // the products of block g - 1 are still to be issued,
      bool pend_first = false;  // as the first ones of their item
      bool ok = true;
      auto products = [&](int pg) -> bool {
        if (!mbar_wait_warp(p_full, pg & 1, status, kSiteCross)) return false;
        tc_fence_after();
        const int qs = pg % C::kQ, ds = pg % C::kdO;
        const uint64_t qd = smem_desc_add(qt_desc, qs * C::kTile);
        const uint64_t dod = smem_desc_add(dot_desc, ds * C::kTile);
        const uint32_t acc0 = pend_first ? 0u : 1u;
        if (leader) {
          // 16 queries = group kk: P at columns 16 kk, dz at 16 kk + 8.  dK goes
          // ahead, kLead groups of dV behind, so that Q_i is released for the
          // load of Q_{i+2} before dV is done.
#pragma unroll
          for (int kk = 0; kk < 8 + kLead; ++kk) {
            if (kk < 8)
              umma_bf16_ts(tdK, tdP + 16 * kk + 8, smem_desc_add(qd, kk * 2048), kIdescAcc,
                           kk > 0 ? 1u : acc0);
            if (kk == 7) umma_commit(&q_empty[qs]);
            if (kk >= kLead)
              umma_bf16_ts(tdV, tdP + 16 * (kk - kLead), smem_desc_add(dod, (kk - kLead) * 2048),
                           kIdescAcc, kk > kLead ? 1u : acc0);
          }
          umma_commit(&do_empty[ds]);
          umma_commit(acc_done);
        }
        __syncwarp();
        return true;
      };
      for (int r = 0; ok; ++r) {
        const int slot = r % kXKvRing;
        if (!(ok = mbar_wait_warp(&it_full[slot], (r / kXKvRing) & 1, status, kSiteCross))) break;
        const int count = __shfl_sync(0xffffffffu, items[slot].count, 0);
        // (those from its first block on)
        const int queries = __shfl_sync(0xffffffffu, items[slot].queries - items[slot].first * A.pq, 0);
        __syncwarp();
        if (leader) mbar_arrive(&it_empty[slot]);
        if (count < 0) break;
        if (count == 0 && pend) {
          // nothing to overlap with, and the items behind may wait for this one
          if (!(ok = products(g - 1))) break;
          pend = false;
        }
        for (int i = 0; ok && i < count; ++i, ++g) {
          const int qs = g % C::kQ, ds = g % C::kdO;
          if (i == 0) {
            // S^T_g before the products of block g - 1, unless those are ready
            // first (an item's first S^T waits for its K).
            if (pend) {
              const int first =
                  mbar_wait_first(k_full, n & 1, p_full, (g - 1) & 1, status, kSiteCross);
              if (__all_sync(0xffffffffu, first == 2)) {
                if (!(ok = products(g - 1))) break;
                pend = false;
              }
            }
            if (!(ok = mbar_wait_warp(k_full, n & 1, status, kSiteCross))) break;
          }
          // rows of the block that hold a real query (the others are zeroed: they
          // take part in the products)
          const int rows = min(queries - i * A.pq, A.pq) * A.G;
          if (!(ok = mbar_wait_warp(&q_full[qs], (g / C::kQ) & 1, status, kSiteCross))) break;
          if (rows < A.G * A.pq) cross_clear_tail<D>(sQ + qs * C::kTile, rows, lane);
          // tS was read into registers for block g - 1.
          if (g > 0 && !(ok = mbar_wait_warp(s_free, (g - 1) & 1, status, kSiteCross))) break;
          tc_fence_after();
          const uint64_t qd = smem_desc_add(q_desc, qs * C::kTile);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
              umma_bf16(tS, smem_desc_add(k_desc, off), smem_desc_add(qd, off), kIdescSq,
                        kk > 0 ? 1u : 0u);
            }
            umma_commit(s_full);
            if (i == count - 1) umma_commit(k_empty);
          }
          __syncwarp();
          if (pend && !(ok = products(g - 1))) break;
          pend = true;
          pend_first = i == 0;
          if (i == 0 && !(ok = mbar_wait_warp(v_full, n & 1, status, kSiteCross))) break;
          if (!(ok = mbar_wait_warp(&do_full[ds], (g / C::kdO) & 1, status, kSiteCross))) break;
          if (rows < A.G * A.pq) cross_clear_tail<D>(sdO + ds * C::kTile, rows, lane);
          // dP^T_g overwrites the P^T / dz^T that the products above read.
          if (g > 0 && !(ok = mbar_wait_warp(acc_done, (g - 1) & 1, status, kSiteCross))) break;
          tc_fence_after();
          const uint64_t dod = smem_desc_add(do_desc, ds * C::kTile);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
              umma_bf16(tdP, smem_desc_add(v_desc, off), smem_desc_add(dod, off), kIdescSq,
                        kk > 0 ? 1u : 0u);
            }
            umma_commit(dp_full);
            if (i == count - 1) umma_commit(v_empty);
          }
          __syncwarp();
          if (i == 0) ++n;
        }
      }
      if (ok && pend) products(g - 1);
      if (leader) {
        umma_commit(drain);
        mbar_wait(drain, 0, status, kSiteCross, 200000000ull, false);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------------------------------------------------- tile stores
      // dz^T of a block pair goes to the workspace for the dQ product, as one bulk
      // store of the image the compute warps assembled.
      if (lane == 0) {
        int g = 0;
        bool ok = true;
        for (int r = 0; ok; ++r) {
          const int slot = r % kXKvRing;
          if (!mbar_wait(&it_full[slot], (r / kXKvRing) & 1, status, kSiteCross)) break;
          const int count = items[slot].count, n = items[slot].n, hk = items[slot].hk,
                    kb = items[slot].kb, first = items[slot].first;
          mbar_arrive(&it_empty[slot]);
          if (count < 0) break;
          for (int i = 0; i < count; ++i, ++g) {
            if (!(ok = mbar_wait(ds_full, g & 1, status, kSiteCross))) break;
            bulk_store(B.tiles + cross_tile(B, n, hk, first + i, kb) * kXTileBytes, sDs,
                       static_cast<uint32_t>(kXTileBytes));
            bulk_commit();
            bulk_wait_read();
            mbar_arrive(ds_free);
          }
        }
        bulk_wait_all();  // complete before the CTA exits
      }
    }
    if constexpr (SPLIT) {
      __syncwarp();
      cluster_sync();  // the shares are in shared memory
    }
  } else {
    // ---------------------------------------------------------- compute
    setmaxnreg_inc<kXKvRegsCompute>();
    // Four warps per TMEM lane quarter; `grp` picks 32 of the 128 query columns.
    const int quarter = warp & 3;
    const int grp = (warp - 4) >> 2;
    const int t = quarter * 32 + lane;  // key row within the block; row of a query block to stage
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t my_cols = lane_off + static_cast<uint32_t>(grp * 32);
    const float mul = A.scale * kOptLog2e;
    const int my_query = cross_query(A, t), my_head = t - my_query * A.G;
    bool ok = true;
    // What row t of the next block brings, loaded one block ahead (group 0) and
    // first used when it is staged: an operation on it here would wait for the
    // loads.  Rows without a real query get a log-sum-exp of infinity (their
    // scores are 0: P = 0) and no delta.
    float q_lse = 0.f, q_delta = 0.f;
    bool q_in = false;
    auto load_query = [&](int q0, int queries, int hk, int qb) {
      const int qi = qb * A.pq + my_query;
      q_in = my_query < A.pq && qi < queries;
      if (q_in) {
        const int64_t at =
            (static_cast<int64_t>(hk) * A.G + my_head) * A.q_rows + q0 + qi;
        q_lse = B.lse[at];
        if constexpr (!WHOLE) q_delta = B.delta[at];
      }
    };
    bool have = false;  // loaded and not yet staged
    auto stage_query = [&](int st) {
      have = false;
      if (grp != 0) return;
      sL[st * 128 + t] = q_in ? q_lse * kOptLog2e : INFINITY;
      // (what a whole item forms itself takes its place)
      if constexpr (!WHOLE) sD[st * 128 + t] = q_in ? q_delta : 0.f;
      mbar_arrive_warp(&lse_ready[st], lane);
    };
    // waits for item r's announcement and loads its first block's queries
    auto look_ahead = [&](int r) {
      const int slot = r % kXKvRing;
      if (!mbar_wait_warp(&it_full[slot], (r / kXKvRing) & 1, status, kSiteCross)) {
        ok = false;
        return;
      }
      const XKvItem& it = items[slot];
      have = it.count > 0;
      if (have && grp == 0) load_query(it.q0, it.queries, it.hk, it.first);
    };
    // A block that holds all keys of its sequence (`whole`; WHOLE: the call has no other)
    // forms delta itself, sum_j P dP in 32 bits.  (From the stored bf16 O it is off by up
    // to 2^-8 of O dO, which where few keys share the weight is as much as all of dP -
    // delta: with one key it would leave dQ, which is 0, with nothing but that.)  Sums
    // over a warp's 32 keys leave column `lane` to lane `lane`; then over the four warps
    // of the group in a fixed order, through the places of sDs that this group's dz goes
    // to (rows 0..7: a warp's 32 columns in two of them), once the store of the block
    // before has read them, into sD.  dP^T is loaded again behind it: kept in registers,
    // it costs the other items 1% more.  4 x 1037 queries to 128 keys, 64 heads of 128: 95
    // us against 112 with the pass over O and dO; 4096 queries of 16 heads to 100 keys of
    // 2: 107 against 90; one of four sequences of 1037 with 300 keys, the others with 40
    // to 128: 182 against 163 with delta from O for all.
    auto meet = [&](uint32_t phase) -> bool {  // (twice a block)
      mbar_arrive_warp(&meet_bar[grp], lane);
      return mbar_wait_warp(&meet_bar[grp], phase, status, kSiteCross);
    };
    auto part = [&](int q) -> float* {
      const int r = 2 * q + (lane >> 4), side = ((r >> 2) ^ grp) & 1;
      return reinterpret_cast<float*>(sDs + (grp >> 1) * 16384 + r * 128 + side * 64) + (lane & 15);
    };
    auto sum_delta = [&](const float (&p)[32], bool mine, int g) -> bool {
      float dp[32];
      tmem_ld_32x32b_x32(tdP + my_cols, dp);
#pragma unroll
      for (int e = 0; e < 32; ++e) dp[e] = mine ? dp[e] : 0.f;
      if (g > 0 && !mbar_wait_warp(ds_free, (g - 1) & 1, status, kSiteCross)) return false;
      auto both = [&](float a, float b, int o) {
        return (lane & o ? b : a) + __shfl_xor_sync(0xffffffffu, lane & o ? a : b, o);
      };
      // (depth first: few sums at a time are in registers)
      auto sum16 = [&](int e) { return both(p[e] * dp[e], p[e + 16] * dp[e + 16], 16); };
      auto sum8 = [&](int e) { return both(sum16(e), sum16(e + 8), 8); };
      auto sum4 = [&](int e) { return both(sum8(e), sum8(e + 4), 4); };
      auto sum2 = [&](int e) { return both(sum4(e), sum4(e + 2), 2); };
      *part(quarter) = both(sum2(0), sum2(1), 1);
      if (!meet(0)) return false;
      if (quarter == 0)
        sD[(g & 1) * 128 + grp * 32 + lane] = (*part(0) + *part(1)) + (*part(2) + *part(3));
      return meet(1);
    };
    // dV and dK of the item before, in TMEM until its last products are done,
    // or (keys that no query sees) zeros.
    bool pending = false;
    int p_k0 = 0, p_real = 0, p_slot = 0, p_hk = 0;
    auto store_item = [&](bool from_tmem, int k0, int real, int slot, int hk) {
      // 32 columns of dV (w = 0) and dK (1: scaled) a warp, or of one of them (d = 64)
#pragma unroll 1
      for (int task = grp; task < D / 16; task += 4) {
        const int w = task / (D / 32), c = task % (D / 32);
        const float sc = w == 0 ? 1.f : A.scale;
        uint16_t* base = (w == 0 ? B.dv : B.dk) +
                         (static_cast<int64_t>(k0) + quarter * 32) * A.ld_kv + hk * D;
        // (a block behind its sequence has no rows, and may start behind all rows)
        const bool in_range = MC_DCHECK(slot == 0 || (k0 + slot <= A.kv_rows && hk < A.KV),
                                        status, kSiteCross);
        float v[32] = {};
        if (from_tmem) {
          tmem_ld_32x32b_x32((w == 0 ? tdV : tdK) + lane_off + c * 32, v);
          if (t >= real) {  // padding
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
          }
        }
        store_rows32(base + c * 32, A.ld_kv, in_range ? slot - quarter * 32 : 0, v, sc, lane);
      }
    };
    look_ahead(0);
    if (have) stage_query(0);
    int g = 0;
    for (int r = 0; ok; ++r) {
      const XKvItem& it = items[r % kXKvRing];
      const int count = it.count;
      if (count < 0) break;
      const int q0 = it.q0, queries = it.queries, hk = it.hk, first = it.first;
      const bool edge = it.real < 128, mine = t < it.real;
      const bool whole = WHOLE || it.whole;
      for (int i = 0; i < count; ++i, ++g) {
        const float* l2 = sL + (g & 1) * 128 + grp * 32;
        const float* dl = sD + (g & 1) * 128 + grp * 32;
        if (!mbar_wait_warp(&lse_ready[g & 1], (g >> 1) & 1, status, kSiteCross) ||
            !mbar_wait_warp(s_full, g & 1, status, kSiteCross)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float p[32];
        tmem_ld_32x32b_x32(tS + my_cols, p);
        tc_fence_before();
        mbar_arrive_warp(s_free, lane);
        // the next block's queries: loaded here, staged behind this block's work
        if (i + 1 < count) {
          have = true;
          if (grp == 0) load_query(q0, queries, hk, first + i + 1);
        } else {
          look_ahead(r + 1);
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 lv = *reinterpret_cast<const float4*>(l2 + e);
          const float2 y0 = __ffma2_rn(make_float2(p[e], p[e + 1]), make_float2(mul, mul),
                                       make_float2(-lv.x, -lv.y));
          const float2 y1 = __ffma2_rn(make_float2(p[e + 2], p[e + 3]), make_float2(mul, mul),
                                       make_float2(-lv.z, -lv.w));
          p[e] = fast_exp2(y0.x);
          p[e + 1] = fast_exp2(y0.y);
          p[e + 2] = fast_exp2(y1.x);
          p[e + 3] = fast_exp2(y1.y);
        }
        if (edge) {  // (keys behind the sequence)
#pragma unroll
          for (int e = 0; e < 32; ++e) p[e] = mine ? p[e] : 0.f;
          if (whole && it.real == 1) {  // the weight of a sequence's only key is 1, and dz = dP - dP
#pragma unroll
            for (int e = 0; e < 32; ++e) p[e] = rintf(p[e]);
          }
        }
        if (pending) {
          if (!mbar_wait_warp(acc_done, (g - 1) & 1, status, kSiteCross)) {
            ok = false;
            break;
          }
          tc_fence_after();
          store_item(true, p_k0, p_real, p_slot, p_hk);
          tc_fence_before();
          pending = false;
        }
        if (!mbar_wait_warp(dp_full, g & 1, status, kSiteCross)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (whole && !(ok = sum_delta(p, mine, g))) break;
        uint32_t pp[16];  // dz
        {
          float dv[32];
          tmem_ld_32x32b_x32(tdP + my_cols, dv);
          if (edge) {  // (V behind the sequence may be anything)
#pragma unroll
            for (int e = 0; e < 32; ++e) dv[e] = mine ? dv[e] : 0.f;
          }
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
            uint32_t w[16];  // [P of 16 queries | their dz], bf16 (see the top)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const int at = gr * 16 + e;
              const float4 dlv = *reinterpret_cast<const float4*>(dl + at);
              const float* dq = dv + gr * 16 + e;
              const float2 d0 = __fmul2_rn(make_float2(p[at], p[at + 1]),
                                           __fadd2_rn(make_float2(dq[0], dq[1]),
                                                      make_float2(-dlv.x, -dlv.y)));
              const float2 d1 = __fmul2_rn(make_float2(p[at + 2], p[at + 3]),
                                           __fadd2_rn(make_float2(dq[2], dq[3]),
                                                      make_float2(-dlv.z, -dlv.w)));
              w[e / 2] = pack_bf16x2(p[at], p[at + 1]);
              w[e / 2 + 1] = pack_bf16x2(p[at + 2], p[at + 3]);
              w[8 + e / 2] = pack_bf16x2(d0.x, d0.y);
              w[8 + e / 2 + 1] = pack_bf16x2(d1.x, d1.y);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) pp[gr * 8 + e] = w[8 + e];
            // over this thread's own dP^T columns, already in registers
            tmem_st_32x32b_x16(tdP + my_cols + gr * 16, w);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(p_full, lane);
        // The 128-byte-swizzled shared-memory image of an MN-major A operand:
        // 64-query chunks 16 KB apart, key row t at 128 B, the 16-byte unit
        // of queries [8u, 8u + 8) at unit u ^ (t & 7); the store of the
        // block before must have read sDs first.
        if (g > 0 && !mbar_wait_warp(ds_free, (g - 1) & 1, status, kSiteCross)) {
          ok = false;
          break;
        }
        uint8_t* ds_row = sDs + (grp >> 1) * 16384 + t * 128;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint4*>(ds_row + (((u + 4 * (grp & 1)) ^ (t & 7)) << 4)) =
              make_uint4(pp[4 * u], pp[4 * u + 1], pp[4 * u + 2], pp[4 * u + 3]);
        fence_proxy_async_smem();  // visible to the bulk copy
        mbar_arrive_warp(ds_full, lane);
        if (have) stage_query((g + 1) & 1);
      }
      if (!ok) break;
      if (count > 0 || SPLIT) {
        p_k0 = it.k0;
        p_real = it.real;
        p_slot = it.slot;
        p_hk = it.hk;
        pending = true;
        if (SPLIT && count == 0) look_ahead(r + 1);
      } else {
        store_item(false, it.k0, it.real, it.slot, it.hk);
        look_ahead(r + 1);
        if (have) stage_query(g & 1);
      }
      mbar_arrive_warp(&it_empty[r % kXKvRing], lane);
    }
    if constexpr (!SPLIT) {
      if (ok && pending && mbar_wait_warp(acc_done, (g - 1) & 1, status, kSiteCross)) {
        tc_fence_after();
        store_item(true, p_k0, p_real, p_slot, p_hk);
      }
    } else {
      // This share's dV and dK into shared memory, over K, V, Q and dO: every
      // product that read them is complete.
      if (g > 0 && !mbar_wait_warp(acc_done, (g - 1) & 1, status, kSiteCross)) ok = false;
      tc_fence_after();
      float* sums = reinterpret_cast<float*>(smem);  // [2][128][kPitch]
      const bool has = ok && g > 0;
#pragma unroll 1
      for (int task = grp; task < D / 16; task += 4) {
        const int w = task / (D / 32), c = task % (D / 32);
        float v[32] = {};
        if (has) tmem_ld_32x32b_x32((w == 0 ? tdV : tdK) + lane_off + c * 32, v);
        float* to = sums + (w * 128 + t) * C::kPitch + c * 32;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(to + 4 * i) =
              make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
      __syncwarp();
      cluster_sync();  // (every thread of every CTA, whatever it met)
      constexpr int kPer = D / 4;  // threads of a row, four columns each
      const int at = static_cast<int>(threadIdx.x) - 128, col = (at % kPer) * 4;
      for (int rr = share + (at / kPer) * B.shares; rr < p_slot;
           rr += (kXKvWarps * 32 / kPer) * B.shares) {
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int s = 0; s < B.shares; ++s) {
            const float4 v = ld_cluster_v4(mapa_shared(sums + (w * 128 + rr) * C::kPitch + col, s));
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
          }
          const float sc = w == 0 ? 1.f : A.scale;
          uint2 out = make_uint2(pack_bf16x2(sum.x * sc, sum.y * sc), pack_bf16x2(sum.z * sc, sum.w * sc));
          if (rr >= p_real) out = make_uint2(0u, 0u);  // padding
          if (MC_DCHECK(p_k0 + rr < A.kv_rows && p_hk < A.KV, status, kSiteCross))
            *reinterpret_cast<uint2*>((w == 0 ? B.dv : B.dk) +
                                      (static_cast<int64_t>(p_k0) + rr) * A.ld_kv + p_hk * D + col) =
                out;
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

// ---------------------------------------------------------------- dQ
template <int D>
struct XDqCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kKTile = 128 * D * 2;
  static constexpr int kStage = static_cast<int>(kXTileBytes) + kKTile;
  static constexpr int kStages = 3;
  static constexpr int kUsed = kStages * kStage + 24 * 8 + 4 * 48 + kCrossSorted;  // barriers, items, order
  // one CTA per SM, so that the CTAs that do not start are there to be stolen
  static constexpr int kSmem = kUsed + 1024 > 116 * 1024 ? kUsed + 1024 : 116 * 1024;
  static_assert(kSmem <= 227 * 1024, "dq kernel shared memory");
  static constexpr uint32_t kTmemCols = 256;  // two accumulators of 128 columns
};

// What every role needs to know of an item: a block of queries.
struct alignas(16) XDqItem {
  int q0, real, slot;  // its first query row; queries of the block that are real, that have rows
  int count;           // key blocks (-1: no more items)
  int k0, keys;        // the sequence's first key row, and its real keys
  int n, hk, qb;
  int pad[3];
};
constexpr int kXDqRing = 4;

// Persistent, 192 threads: warp 0 loads per key block the dz^T tile (one bulk
// copy of its swizzled image) and K_j into a 3-deep ring that runs on across
// items, warp 1 issues dQ += dz_j K_j (items alternate accumulators), warps
// 2..5 write scale dQ of the item before.
template <int D>
__global__ void __launch_bounds__(192, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ XBwdArgs B) {
  using C = XDqCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const CrossArgs& A = B.c;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStage);
  uint64_t* full = bars + 0;       // [3]
  uint64_t* empty = bars + 3;      // [3]
  uint64_t* acc_full = bars + 6;   // [2]  an item's dQ is complete in accumulator a
  uint64_t* acc_empty = bars + 8;  // [2]  the epilogue has read accumulator a (4 warps)
  uint64_t* drain = bars + 10;
  uint64_t* it_full = bars + 11;   // [kXDqRing]
  uint64_t* it_empty = bars + 15;  // [kXDqRing] read by the MMA and epilogue warps (5)
  uint64_t* steal_bar = bars + 19;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 20);
  void* response = bars + 22;  // 16 bytes, aligned as the stages are
  XDqItem* items = reinterpret_cast<XDqItem*>(bars + 24);
  int8_t* order = reinterpret_cast<int8_t*>(items + 4);
  int* status = A.status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(drain, 1);
    mbar_init(steal_bar, 1);
    for (int i = 0; i < kXDqRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], 5);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // the dK/dV kernel (the tiles) has completed

  // (the heads whose tiles were written last come first: they are still in L2)
  if (B.sort) {
    if (warp == 3) cross_order(A, true, order, lane);
    __syncthreads();
  }
  auto item_of = [&](int k) -> XDqItem {
    XDqItem it = {};
    const CrossItem which = cross_item(k, B.heads, A.nqb);
    it.n = B.sort ? order[which.n] : A.n - 1 - which.n;
    it.hk = B.hk0 + B.heads - 1 - which.hk;
    it.qb = which.block;
    const CrossRows q = cross_queries(A, it.n), kv = cross_keys(A, it.n);
    const int at = it.qb * A.pq;
    it.q0 = q.first + at;
    it.real = min(max(q.real - at, 0), A.pq);
    it.slot = min(max(q.slot - at, 0), A.pq);
    it.k0 = kv.first;
    it.keys = kv.real;
    it.count = it.real > 0 ? (kv.real + 127) / 128 : 0;
    return it;
  };

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------------- producer
      int gt = 0;  // tiles issued, across items
      bool ok = true;
      OptItems steal(response, steal_bar, B.q_items, B.q_steal);
      for (int r = 0;; ++r) {
        XDqItem cur = {};
        cur.count = -1;
        if (steal.more) cur = item_of(steal.k);
        const int slot = r % kXDqRing;
        if (!mbar_wait(&it_empty[slot], ((r / kXDqRing) & 1) ^ 1u, status, kSiteCross)) break;
        items[slot] = cur;
        mbar_arrive(&it_full[slot]);
        if (cur.count < 0) break;
        for (int j = 0; j < cur.count; ++j, ++gt) {
          const int st = gt % C::kStages;
          if (!mbar_wait(&empty[st], ((gt / C::kStages) & 1) ^ 1u, status, kSiteCross)) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + st * C::kStage;
          mbar_arrive_expect_tx(&full[st], C::kStage);
          bulk_load(dst, B.tiles + cross_tile(B, cur.n, cur.hk, cur.qb, j) * kXTileBytes,
                    static_cast<uint32_t>(kXTileBytes), &full[st]);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_2d(dst + kXTileBytes + c * 16384, &tm_k, &full[st], cur.hk * D + c * 64,
                        cur.k0 + j * 128);
        }
        if (!ok || !steal.next(status)) break;
      }
      steal.finish(status);
      pdl_launch();  // every load of this CTA is issued
      for (int g = gt - 1; g >= 0 && g >= gt - C::kStages; --g)
        mbar_wait(&full[g % C::kStages], (g / C::kStages) & 1, status, kSiteCross, 200000000ull,
                  false);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // (converged, as in the dK/dV kernel)
    constexpr uint32_t kIdesc = idesc_bf16_f32(128, D, true, true);
    const bool leader = elect_one();
    // both operands MN-major: 16 keys per step are 16 rows of 128 B; 64-wide
    // query (A) or d (B) chunks 16 KB apart
    const uint64_t a_desc = smem_desc_sw128(smem_u32(smem), 16384, 1024);
    bool ok = true;
    int gt = 0;
    for (int r = 0; ok; ++r) {
      const int slot = r % kXDqRing;
      if (!mbar_wait_warp(&it_full[slot], (r / kXDqRing) & 1, status, kSiteCross)) break;
      const int nj = __shfl_sync(0xffffffffu, items[slot].count, 0);
      const int keys = __shfl_sync(0xffffffffu, items[slot].keys, 0);
      __syncwarp();
      if (leader) mbar_arrive(&it_empty[slot]);
      if (nj < 0) break;
      const int acc = r & 1;
      // the epilogue of item r - 2 has read this accumulator
      if (!mbar_wait_warp(&acc_empty[acc], ((r >> 1) & 1) ^ 1u, status, kSiteCross)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem + static_cast<uint32_t>(acc * 128);
      for (int j = 0; j < nj; ++j, ++gt) {
        const int st = gt % C::kStages;
        if (!mbar_wait_warp(&full[st], (gt / C::kStages) & 1, status, kSiteCross)) {
          ok = false;
          break;
        }
        // dz is 0 for keys behind the sequence, K may be anything there
        if (keys - j * 128 < 128)
          cross_clear_tail<D>(smem + st * C::kStage + kXTileBytes, keys - j * 128, lane);
        tc_fence_after();
        const uint64_t ad = smem_desc_add(a_desc, st * C::kStage);
        const uint64_t kd = smem_desc_add(ad, static_cast<uint32_t>(kXTileBytes));
        const uint32_t acc0 = j > 0 ? 1u : 0u;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16(d_tmem, smem_desc_add(ad, kk * 2048), smem_desc_add(kd, kk * 2048), kIdesc,
                      kk > 0 ? 1u : acc0);
          umma_commit(&empty[st]);
        }
        __syncwarp();
      }
      if (ok && leader) umma_commit(&acc_full[acc]);
      __syncwarp();
    }
    if (leader) {
      umma_commit(drain);
      mbar_wait(drain, 0, status, kSiteCross, 200000000ull, false);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- epilogue
    const int quarter = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    for (int r = 0;; ++r) {
      const int slot = r % kXDqRing;
      if (!mbar_wait_warp(&it_full[slot], (r / kXDqRing) & 1, status, kSiteCross)) break;
      const XDqItem it = items[slot];
      mbar_arrive_warp(&it_empty[slot], lane);
      if (it.count < 0) break;
      const int acc = r & 1;
      if (!mbar_wait_warp(&acc_full[acc], (r >> 1) & 1, status, kSiteCross)) break;
      tc_fence_after();
      const int my_query = cross_query(A, quarter * 32 + lane);
      const bool mine = my_query < it.real;  // (padded queries get zeros)
      const int64_t head0 = static_cast<int64_t>(it.hk) * A.G;
      uint16_t* to[4];  // 4 lanes store 64 bytes of row k of their four
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r4 = quarter * 32 + (lane & ~3) + k;
        const int qi = cross_query(A, r4), hd = r4 - qi * A.G;
        const bool in = qi < it.slot && qi < A.pq &&
                        MC_DCHECK(it.q0 + qi < A.q_rows && head0 + hd < A.H, status, kSiteCross);
        to[k] = in ? B.dq + (static_cast<int64_t>(it.q0) + qi) * A.ld_q + (head0 + hd) * D +
                         (lane & 3) * 8
                   : nullptr;
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float v[32] = {};
        if (it.count > 0)
          tmem_ld_32x32b_x32(tmem + static_cast<uint32_t>(acc * 128) + lane_off + c * 32, v);
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = mine ? pack_bf16x2(v[2 * i] * A.scale, v[2 * i + 1] * A.scale) : 0u;
        transpose_16b_x4(w, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (to[k])
            *reinterpret_cast<uint4*>(to[k] + c * 32) =
                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
      }
      tc_fence_before();
      mbar_arrive_warp(&acc_empty[acc], lane);  // the accumulator may take the item after next
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- launches
// Key heads whose tiles are in the workspace at a time.
constexpr int64_t kXTilesAtOnce = 2ll << 30;
constexpr int64_t kXMostTiles = 1ll << 40;  // of a key head: what a workspace is for ends far below
int64_t head_tiles(const CrossArgs& A) {
  return static_cast<int64_t>(A.n) * A.nqb * A.nkb * kXTileBytes;
}
int heads_at_once(const CrossArgs& A) {
  const int64_t fit = kXTilesAtOnce / head_tiles(A);
  if (fit >= A.KV) return A.KV;
  // equal groups
  const int64_t groups = (A.KV + (fit < 1 ? 1 : fit) - 1) / (fit < 1 ? 1 : fit);
  return static_cast<int>((A.KV + groups - 1) / groups);
}

template <class K>
cudaError_t cross_smem(PerDeviceInit& init, K kern, int bytes) {
  return once_per_device(init, [&](long long*) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}

template <int D>
int launch_bwd(const uint16_t* q, const uint16_t* k, const uint16_t* v, const uint16_t* o,
               const uint16_t* dout, float* delta, XBwdArgs& B, cudaStream_t st) {
  const CrossArgs& A = B.c;
  CUtensorMap tq, tk, tv, td;
  if (!cross_q_map(&tq, q, D, A, A.ld_q) || !cross_kv_map(&tk, k, D, A) ||
      !cross_kv_map(&tv, v, D, A) || !cross_q_map(&td, dout, D, A, A.ld_o))
    return MC_ERR_CUDA;
  static PerDeviceInit init_kv[2], init_split[2], init_q;
  const int whole = A.nkb == 1 ? 1 : 0;
  auto kv = whole ? cross_dkdv_kernel<D, false, true> : cross_dkdv_kernel<D, false, false>;
  auto kv_split = whole ? cross_dkdv_kernel<D, true, true> : cross_dkdv_kernel<D, true, false>;
  auto dq = cross_dq_kernel<D>;
  if (cross_smem(init_kv[whole], kv, XKvCfg<D>::kSmem) != cudaSuccess ||
      cross_smem(init_split[whole], kv_split, XKvCfg<D>::kSmem) != cudaSuccess ||
      cross_smem(init_q, dq, XDqCfg<D>::kSmem) != cudaSuccess)
    return MC_ERR_CUDA;
  if (!whole) {
    const int64_t per_block = kXDeltaThreads / (D / 8) * kXDeltaPasses;
    const int64_t blocks = (static_cast<int64_t>(A.q_rows) * A.H + per_block - 1) / per_block;
    launch_kernel(cross_delta_kernel<D>, dim3(static_cast<unsigned>(blocks)), dim3(kXDeltaThreads),
                  0, st, 1, o, dout, delta, A.q_rows, A.H, A.ld_o);
    if (cudaGetLastError() != cudaSuccess) return MC_ERR_CUDA;
  }
  const int at_once = heads_at_once(A), sms = num_sms();
  B.sort = cross_sorts(A) ? 1 : 0;
  // (items of unequal sequences are taken over by the CTAs that are done, whatever
  // their number: the request's time is behind an item's)
  auto ctas = [&](int items, int* steal) {
    *steal = items > (B.sort ? sms : 4 * sms) ? 1 : 0;
    return dim3(static_cast<unsigned>(*steal || items < sms ? items : sms));
  };
  for (B.hk0 = 0; B.hk0 < A.KV; B.hk0 += at_once) {
    B.heads = A.KV - B.hk0 < at_once ? A.KV - B.hk0 : at_once;
    B.kv_items = A.n * B.heads * A.nkb;
    B.q_items = A.n * B.heads * A.nqb;
    const dim3 kv_grid = ctas(B.kv_items, &B.kv_steal), q_grid = ctas(B.q_items, &B.q_steal);
    // shares of an item: as many as SMs are left for, each four blocks at least
    B.shares = 1;
    while (B.shares < 8 && B.kv_items * B.shares * 2 <= sms && B.shares * 8 <= A.nqb) B.shares *= 2;
    if (B.shares > 1)
      launch_kernel(kv_split, dim3(static_cast<unsigned>(B.kv_items * B.shares)), dim3(kXKvThreads),
                    XKvCfg<D>::kSmem, st, static_cast<unsigned>(B.shares), tq, tk, tv, td, B);
    else
      launch_kernel(kv, kv_grid, dim3(kXKvThreads), XKvCfg<D>::kSmem, st, 1, tq, tk, tv, td, B);
    if (cudaGetLastError() != cudaSuccess) return MC_ERR_CUDA;
    launch_kernel(dq, q_grid, dim3(192), XDqCfg<D>::kSmem, st, 1, tk, B);
    if (cudaGetLastError() != cudaSuccess) return MC_ERR_CUDA;
  }
  return MC_OK;
}

}  // namespace

size_t attention_cross_ws_bytes(const mc_cross_attention& c) {
  const CrossArgs A = cross_args(c, nullptr);
  // (sequences by blocks are below 2^30, key blocks below 2^22)
  if (static_cast<int64_t>(A.n) * A.nqb * A.nkb > kXMostTiles) return 0;
  return static_cast<size_t>(heads_at_once(A) * head_tiles(A));
}

int launch_attention_cross_bwd(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                               const uint16_t* o, const float* lse, const uint16_t* dout,
                               uint16_t* dq, uint16_t* dk, uint16_t* dv, float* delta,
                               const mc_cross_attention& c, uint8_t* ws, size_t, int* status,
                               cudaStream_t st) {
  XBwdArgs B = {};
  B.c = cross_args(c, status);
  B.dq = dq;
  B.dk = dk;
  B.dv = dv;
  B.lse = lse;
  B.delta = delta;
  B.tiles = ws;
  return c.head_dim == 64 ? launch_bwd<64>(q, k, v, o, dout, delta, B, st)
                          : launch_bwd<128>(q, k, v, o, dout, delta, B, st);
}

}  // namespace mc
