// Attention backward over interval masks (sm_103a, tcgen05), scores optionally
// capped by a tanh and biased by the distance.  With P = exp(z - lse) over the
// visible keys, delta = rowsum(dO O) and t = tanh of the capped score:
//   dV = P^T dO,  dP = dO V^T,  dz = P (dP - delta) (1 - t^2),
//   dQ = dz K / sqrt(d),  dK = dz^T Q / sqrt(d).
// Masked places get P = 0 by a select, so rows that see nothing (lse =
// -infinity) give and receive nothing.
//
//   dkdv: a 128-key block against the query blocks that see it (the mask's
//         key table), accumulates dV and dK and, given a workspace, writes
//         each block pair's dz^T tile as bf16.
//   dq:   a 128-query block: with the tiles dQ is their product with K
//         (persistent, bound by the tiles' traffic); without, S and dP are
//         formed again.
//
// P and dz are rounded to bf16, each by at most 2^-8 of itself: an operand of a
// tcgen05 product has the type of the other one, dO's, Q's and K's.  dK and dQ
// take the same rounded dz.  dz itself is formed in 32 bits from the unrounded P;
// sums and accumulators are 32-bit and dQ, dK and dV are rounded once more when
// stored.  With delta's rounding (attention_opt.cu) that is the kernels' whole
// error, 0.0024 to 0.0027 of the result over long rows, up to 0.0035 over short
// ones; with everything but the results in 32 bits 0.0017.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attention_opt.cuh"

namespace mc {
namespace {

constexpr int64_t kOptTileBytes = 128 * 128 * 2;  // one bf16 dz^T tile (128 keys x 128 queries)

struct OptBwdArgs {
  uint16_t* dqkv;
  const float* lse;
  const float* delta;
  const int32_t* key_lo;
  const int32_t* key_hi;
  const int32_t* tables;  // the query entries; the key entries follow
  const float* slopes;
  uint8_t* ds_tiles;
  float softcap;
  int b, s, H;
  int head_major;         // the dQ kernel without tiles
  int steal, head_group;  // the persistent kernels
  int ctas;
  int causal;  // the tiles are of the lower triangle only
  int* status;
};

// Tile (query block, key block) of a (head, batch) in the workspace.
__device__ __forceinline__ int64_t opt_tile(int causal, int nb, int64_t hb, int qb, int kb) {
  const int64_t n = nb;
  return causal ? hb * (n * (n + 1) / 2) + static_cast<int64_t>(qb) * (qb + 1) / 2 + kb
                : (hb * n + qb) * n + kb;
}

// ---------------------------------------------------------------- dK, dV
// What every role needs to know of an item: a (key block, head) pair.
struct alignas(16) OptKvItem {
  int4 entry;  // sequence, key block, first query block, query blocks (-1: no more items)
  int head;
  int pad[3];
};
constexpr int kOptKvRing = 4;

template <int D>
struct OptBwdCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = 128 * D * 2;
  // K, V, the Q_i and dO_i stages (apart, Q_i first: S^T_{i+1} runs ahead of
  // the products of block i), the dz^T tile for its bulk store, lse / delta
  // [2][128], the queries' key ranges relative to the block [2][128] (two
  // bytes each), their edge flags [2][4], items, barriers.  The dynamic
  // shared memory starts 1024-byte aligned (checked at run time).
  static constexpr int kQ = D == 64 ? 3 : 2, kdO = 2;
  static constexpr int kUsed = (2 + kQ + kdO) * kTile + static_cast<int>(kOptTileBytes) +
                               4 * 128 * 4 + 2 * 128 * 2 + 2 * 4 * 4 +
                               kOptKvRing * static_cast<int>(sizeof(OptKvItem)) + 36 * 8;
  // one CTA per SM: it takes all 512 TMEM columns
  static constexpr int kSmem = kUsed > 116 * 1024 ? kUsed : 116 * 1024;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kUsed <= 227 * 1024, "dkdv kernel shared memory");
};

// Bit i of lane j becomes bit j of lane i (a 32 x 32 transpose in five steps).
__device__ __forceinline__ uint32_t bit_transpose(uint32_t x, int lane) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const uint32_t low = d == 16  ? 0x0000FFFFu
                         : d == 8 ? 0x00FF00FFu
                         : d == 4 ? 0x0F0F0F0Fu
                         : d == 2 ? 0x33333333u
                                  : 0x55555555u;
    // lanes without bit d keep their low columns and take the partner's low
    // ones as high; the others the reverse
    const bool up = lane & d;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, x, d);
    x = up ? (x & ~low) | ((got & ~low) >> d) : (x & low) | ((got & low) << d);
  }
  return x;
}

constexpr int kOptKvThreads = 640;
// 128 x 56 + 512 x 104 of the launch's 640 x 96 registers.
constexpr int kOptKvRegsIo = 56, kOptKvRegsCompute = 104;
constexpr int kOptKvWarps = 16;  // compute warps

// Persistent: one CTA per SM walks the (key block, head) items, each against
// the query blocks that see it (blocks i, counted across items).  640 threads:
// warp 0 loads, warp 1 issues, warp 2 stores dz^T tiles, warps 4..19 compute.
// TMEM: S^T [0, 128), dP^T [128, 256), dV [256, 256 + D), dK [384, 384 + D).
// Per query block i:
//   MMA      S^T_i = K Q_i^T (as soon as the compute warps hold S^T_{i-1} in
//            registers), then dV += P^T_{i-1} dO_{i-1}, dK += dz^T_{i-1} Q_{i-1},
//            then (those done) dP^T_i = V dO_i^T.
//   compute  P^T (and the cap's derivative) from S^T_i while the products
//            above run, then dz^T from dP^T_i.
// A compute thread owns one key row and 32 query columns: the 16 queries of
// group g (dP^T columns [16g, 16g + 16)) leave P at columns [16g, 16g + 8) and
// dz at [16g + 8, 16g + 16), over columns that the thread itself has read.
// An item's dV and dK are stored during the next item's first block: its
// S^T and weights run meanwhile, as do the loads of its K and V.
//
// A block takes about 4200 clocks, its four products 3100, which share the
// shared memory with the loads and the tile's way out (192 + 64 + 64 KB); where
// documents are short HBM counts too (the dz^T tiles). Sixteen compute warps
// against eight of 64 columns: 452 against 476 us for a capped backward over
// 8192 tokens and 16 heads, 22.1 against 23.1 us for 4 x 509 tokens and 12
// heads, 263 against 266 us for 4096 packed tokens of 64 heads, but 722 against
// 712 us for the same without a mask but the causal one. Shorter chains from one
// block's products to the next were slower in all: P^T over S^T's columns with
// dz^T read from shared memory, so that dP^T runs ahead (776 us, 757 with dK
// issued earlier), P^T over dP^T's as soon as that is in registers (824 us), dV
// and dK through the tile's buffer and TMA (722 us with eight warps), the
// queries' lse, delta and masks staged by a warp of their own (753 us).
template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kOptKvThreads, 1)
    attn_opt_dkdv_kernel(const __grid_constant__ CUtensorMap tm_qkv,
                         const __grid_constant__ CUtensorMap tm_do,
                         const __grid_constant__ OptBwdArgs A) {
  using C = OptBwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  int* status = A.status;
  if (smem_u32(smem) & 1023u) {  // the 128-byte swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) record_error(status, MC_ERR_DEVICE_BOUNDS, kSiteAttention);
    return;
  }
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::kTile;
  uint8_t* sQ = smem + 2 * C::kTile;             // [kQ]
  uint8_t* sdO = smem + (2 + C::kQ) * C::kTile;  // [kdO]
  uint8_t* sDs = sdO + C::kdO * C::kTile;  // dz^T tile image (swizzled), 32 KB
  float* sL = reinterpret_cast<float*>(sDs + kOptTileBytes);  // [2][128] lse * log2(e)
  float* sD = sL + 256;                                        // [2][128] delta
  OptKvItem* items = reinterpret_cast<OptKvItem*>(sD + 256);
  uint64_t* bars = reinterpret_cast<uint64_t*>(items + kOptKvRing);
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
  uint64_t* it_full = bars + 22;    // [kOptKvRing]
  uint64_t* it_empty = bars + 26;   // [kOptKvRing] read by MMA, tile and compute warps (18)
  uint64_t* steal_bar = bars + 30;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 31);
  void* response = bars + 32;  // 16 bytes, aligned as the items are
  uint64_t* ds_full = bars + 34;  // the dz^T tile of block i is in sDs (16 warps)
  uint64_t* ds_free = bars + 35;  // its bulk store has read sDs
  uint16_t* sM = reinterpret_cast<uint16_t*>(bars + 36);  // [2][128] first | end << 8
  int* sF = reinterpret_cast<int*>(sM + 256);             // [2][4] the 32 queries see the whole block

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = A.s, H = A.H, a = A.H * D;
  const int nb = (s + 127) / 128;
  if (threadIdx.x == 0) {
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
    mbar_init(ds_full, kOptKvWarps);
    mbar_init(ds_free, 1);
    mbar_init(s_full, 1);
    mbar_init(s_free, kOptKvWarps);
    mbar_init(dp_full, 1);
    mbar_init(p_full, kOptKvWarps);
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    mbar_init(steal_bar, 1);
    for (int i = 0; i < kOptKvRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], 2 + kOptKvWarps);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_qkv);
    tma_prefetch_desc(&tm_do);
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
  const uint32_t tS = tmem, tdP = tmem + 128, tdV = tmem + 256, tdK = tmem + 384;

  if (warp < 4) {
    setmaxnreg_dec<kOptKvRegsIo>();
    if (warp == 0) {
      if (lane == 0) {
        // -------------------------------------------------------- producer
        int g = 0, n = 0;  // query blocks and items (with blocks) loaded
        int q_n = 0, do_n = 0;
        bool ok = true, v_loaded = true;
        int4 e_next = make_int4(0, 0, 0, 0);
        int h_next = 0;
        OptItems steal(response, steal_bar, A.b * nb * H, A.steal);
        const int32_t* table = A.tables + 4ll * A.b * nb;  // the key entries
        auto read_entry = [&]() {
          int rank = 0;
          if (steal.more) {
            opt_item(steal.k, A.b * nb, H, A.head_group, rank, h_next);
            e_next = *reinterpret_cast<const int4*>(table + 4ll * rank);
          }
        };
        auto announce = [&](int r, OptKvItem& it) -> bool {
          it.entry = make_int4(0, 0, 0, -1);
          it.head = h_next;
          if (steal.more) {
            const int4 e = opt_checked(e_next, A.b, nb, status);
            const int first = max(e.z, 0);
            it.entry = make_int4(e.x, e.y, first, max(min(e.w, nb) - first, 0));
          }
          const int slot = r % kOptKvRing;
          if (!mbar_wait(&it_empty[slot], ((r / kOptKvRing) & 1) ^ 1u, status, kSiteAttention))
            return false;
          items[slot].entry = it.entry;
          items[slot].head = it.head;
          mbar_arrive(&it_full[slot]);
          return true;
        };
        OptKvItem cur, next;
        read_entry();
        ok = announce(0, cur);
        // (an item's first loads are issued before the next item is asked about)
        auto go_on = [&](int r) -> bool {
          if (steal.more) {
            if (!steal.next(status)) return false;
            read_entry();
          }
          return announce(r + 1, next);
        };
        for (int r = 0; ok && cur.entry.w >= 0; ++r, cur = next) {
          const int bi = cur.entry.x, r0 = cur.entry.y * 128, hh = cur.head;
          const int cq = hh * D, ck = a + hh * D, cv = 2 * a + hh * D;
          const bool early = r > 0 || cur.entry.w == 0;  // (the first item's loads go first)
          if (early && !(ok = go_on(r))) break;
          for (int i = 0; ok && i < cur.entry.w; ++i, ++g) {
            if (i == 0) {
              if (!(ok = mbar_wait(k_empty, (n & 1) ^ 1u, status, kSiteAttention))) break;
              mbar_arrive_expect_tx(k_full, C::kTile);
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_3d(sK + c * 16384, &tm_qkv, k_full, ck + c * 64, r0, bi);
              v_loaded = false;
            }
            const int row = (cur.entry.z + i) * 128;
            const int qs = g % C::kQ, ds = g % C::kdO;
            if (!(ok = mbar_wait(&q_empty[qs], ((g / C::kQ) & 1) ^ 1u, status, kSiteAttention)))
              break;
            mbar_arrive_expect_tx(&q_full[qs], C::kTile);
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_3d(sQ + qs * C::kTile + c * 16384, &tm_qkv, &q_full[qs], cq + c * 64, row,
                          bi);
            ++q_n;
            if (!(ok = mbar_wait(&do_empty[ds], ((g / C::kdO) & 1) ^ 1u, status, kSiteAttention)))
              break;
            mbar_arrive_expect_tx(&do_full[ds], C::kTile);
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_3d(sdO + ds * C::kTile + c * 16384, &tm_do, &do_full[ds], hh * D + c * 64,
                          row, bi);
            ++do_n;
            if (i == 0) {
              if (!(ok = mbar_wait(v_empty, (n & 1) ^ 1u, status, kSiteAttention))) break;
              mbar_arrive_expect_tx(v_full, C::kTile);
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_3d(sV + c * 16384, &tm_qkv, v_full, cv + c * 64, r0, bi);
              v_loaded = true;
              ++n;
              if (!early && !(ok = go_on(r))) break;
            }
          }
        }
        steal.finish(status);
        pdl_launch();  // every load of this CTA is issued
        // Copies still in flight must land before the CTA exits.
        const int kn = v_loaded ? n : n + 1;  // K tiles issued
        if (kn > 0) mbar_wait(k_full, (kn - 1) & 1, status, kSiteAttention, 200000000ull, false);
        if (n > 0) mbar_wait(v_full, (n - 1) & 1, status, kSiteAttention, 200000000ull, false);
        for (int i = q_n - 1; i >= 0 && i >= q_n - C::kQ; --i)
          mbar_wait(&q_full[i % C::kQ], (i / C::kQ) & 1, status, kSiteAttention, 200000000ull,
                    false);
        for (int i = do_n - 1; i >= 0 && i >= do_n - C::kdO; --i)
          mbar_wait(&do_full[i % C::kdO], (i / C::kdO) & 1, status, kSiteAttention, 200000000ull,
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
        if (!mbar_wait_warp(p_full, pg & 1, status, kSiteAttention)) return false;
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
        const int slot = r % kOptKvRing;
        if (!(ok = mbar_wait_warp(&it_full[slot], (r / kOptKvRing) & 1, status, kSiteAttention)))
          break;
        const int count = __shfl_sync(0xffffffffu, items[slot].entry.w, 0);
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
              const int first = mbar_wait_first(k_full, n & 1, p_full, (g - 1) & 1, status,
                                                kSiteAttention);
              if (__all_sync(0xffffffffu, first == 2)) {
                if (!(ok = products(g - 1))) break;
                pend = false;
              }
            }
            if (!(ok = mbar_wait_warp(k_full, n & 1, status, kSiteAttention))) break;
          }
          if (!(ok = mbar_wait_warp(&q_full[qs], (g / C::kQ) & 1, status, kSiteAttention))) break;
          // tS was read into registers for block g - 1.
          if (g > 0 && !(ok = mbar_wait_warp(s_free, (g - 1) & 1, status, kSiteAttention))) break;
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
          if (i == 0 && !(ok = mbar_wait_warp(v_full, n & 1, status, kSiteAttention))) break;
          if (!(ok = mbar_wait_warp(&do_full[ds], (g / C::kdO) & 1, status, kSiteAttention))) break;
          // dP^T_g overwrites the P^T / dz^T that the products above read.
          if (g > 0 && !(ok = mbar_wait_warp(acc_done, (g - 1) & 1, status, kSiteAttention))) break;
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
        mbar_wait(drain, 0, status, kSiteAttention, 200000000ull, false);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------------------------------------------------- tile stores
      // dz^T of a block pair goes to `ds_tiles` for the dQ product, as one bulk
      // store of the image the compute warps assembled.
      if (lane == 0) {
        int g = 0;
        bool ok = true;
        for (int r = 0; ok; ++r) {
          const int slot = r % kOptKvRing;
          if (!mbar_wait(&it_full[slot], (r / kOptKvRing) & 1, status, kSiteAttention)) break;
          const int4 e = items[slot].entry;
          const int hh = items[slot].head;
          mbar_arrive(&it_empty[slot]);
          if (e.w < 0) break;
          if (!A.ds_tiles) continue;
          const int64_t hb = static_cast<int64_t>(e.x) * H + hh;
          for (int i = 0; i < e.w; ++i, ++g) {
            if (!(ok = mbar_wait(ds_full, g & 1, status, kSiteAttention))) break;
            const int qb = e.z + i;
            // the workspace of a causal mask has no tile above the diagonal
            if (check_index(!A.causal || e.y <= qb, status, kSiteAttention)) {
              bulk_store(A.ds_tiles + opt_tile(A.causal, nb, hb, qb, e.y) * kOptTileBytes, sDs,
                         static_cast<uint32_t>(kOptTileBytes));
              bulk_commit();
              bulk_wait_read();
            }
            mbar_arrive(ds_free);
          }
        }
        bulk_wait_all();  // complete before the CTA exits
      }
    }
  } else {
    // ---------------------------------------------------------- compute
    setmaxnreg_inc<kOptKvRegsCompute>();
    // Four warps per TMEM lane quarter; `grp` picks 32 of the 128 query columns.
    const int quarter = warp & 3;
    const int grp = (warp - 4) >> 2;
    const int t = quarter * 32 + lane;  // key row within the block
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t my_cols = lane_off + static_cast<uint32_t>(grp * 32);
    bool ok = true;
    // What query t of the next block brings, loaded one block ahead (group 0)
    // and first used when it is staged: an operation on it here would wait for
    // the loads.  Queries past the sequence see the whole block, so that they do
    // not make it an edge, with a log-sum-exp of infinity: P = exp(z - lse) is 0
    // whatever the bias (a negative slope's grows with the distance, and an
    // infinite P would not be cancelled by their dO of zeros).
    float q_lse = 0.f, q_delta = 0.f;
    int q_lo = 0, q_hi = 0, q_r0 = 0;  // and the first key of its block
    bool q_in = false;
    auto load_query = [&](int bi, int hh, int r0, int qn) {
      q_in = qn < s;
      q_r0 = r0;
      if (q_in) {
        const int64_t hrow = (static_cast<int64_t>(bi) * H + hh) * s + qn;
        const int64_t brow = static_cast<int64_t>(bi) * s + qn;
        q_lse = A.lse[hrow];
        q_delta = A.delta[hrow];
        q_lo = A.key_lo[brow];
        q_hi = A.key_hi[brow];
      }
    };
    bool have = false;  // loaded and not yet staged
    auto stage_query = [&](int st) {
      have = false;
      if (grp != 0) return;
      // (the bounds, any 32-bit integers, cut to the sequence first)
      const int first = min(max(max(q_lo, 0) - q_r0, 0), 128);
      const int end = min(max(max(min(q_hi, s), 0) - q_r0, 0), 128);
      const int range = q_in ? first | (end << 8) : 128 << 8;
      sL[st * 128 + t] = q_in ? q_lse * kOptLog2e : INFINITY;
      sD[st * 128 + t] = q_in ? q_delta : 0.f;
      sM[st * 128 + t] = static_cast<uint16_t>(range);
      const bool whole = __all_sync(0xffffffffu, range == (128 << 8));
      if (lane == 0) sF[st * 4 + quarter] = whole ? 1 : 0;
      mbar_arrive_warp(&lse_ready[st], lane);
    };
    float slope = 0.f, n_slope = 0.f;
    // waits for item r's announcement and loads its first block's queries
    auto look_ahead = [&](int r) {
      const int slot = r % kOptKvRing;
      if (!mbar_wait_warp(&it_full[slot], (r / kOptKvRing) & 1, status, kSiteAttention)) {
        ok = false;
        return;
      }
      const int4 e = items[slot].entry;
      have = e.w > 0;
      if (have) {
        if (grp == 0) load_query(e.x, items[slot].head, e.y * 128, e.z * 128 + t);
        if constexpr (BIAS) n_slope = A.slopes[items[slot].head];
      }
    };
    // dV and dK of the item before, in TMEM until its last products are done,
    // or (a key block that no query sees) zeros.
    bool pending = false;
    int p_row = 0, p_bi = 0, p_head = 0;
    auto store_item = [&](bool from_tmem, int row0, int bi, int hh) {
      const int warp_row = row0 + quarter * 32;
      // 32 columns of dV (w = 0: V's columns of dqkv) and dK (1: scaled by
      // 1/sqrt(d)) a warp, or of one of them (d = 64)
#pragma unroll 1
      for (int task = grp; task < D / 16; task += 4) {
        const int w = task / (D / 32), c = task % (D / 32);
        const float mul = w == 0 ? 1.f : rsqrtf(static_cast<float>(D));
        const int col = (w == 0 ? 2 * a : a) + hh * D;
        uint16_t* base = A.dqkv + (static_cast<int64_t>(bi) * s + warp_row) * 3 * a + col;
        const bool in_range = MC_DCHECK(warp_row >= 0 && bi >= 0 && bi < A.b && col + D <= 3 * a,
                                        status, kSiteAttention);
        float v[32] = {};
        if (from_tmem) tmem_ld_32x32b_x32((w == 0 ? tdV : tdK) + lane_off + c * 32, v);
        store_rows32(base + c * 32, 3ll * a, in_range ? s - warp_row : 0, v, mul, lane);
      }
    };
    look_ahead(0);
    if (have) stage_query(0);
    int g = 0;
    for (int r = 0; ok; ++r) {
      const OptKvItem& it = items[r % kOptKvRing];
      const int count = it.entry.w;
      if (count < 0) break;
      const int bi = it.entry.x, r0 = it.entry.y * 128, qb0 = it.entry.z;
      const int hh = it.head;
      slope = n_slope;
      const ScoreConst sc =
          score_const<CAP, BIAS>(rsqrtf(static_cast<float>(D)), A.softcap, slope);
      const CapPoly poly = cap_poly(1.f, sc.arg);
      const float cap_limit = cap_small_limit(sc.arg);
      const float cap_limit2 = cap_limit * cap_limit;
      for (int i = 0; i < count; ++i, ++g) {
        const int c0 = (qb0 + i) * 128;  // first query of this block
        const float* l2 = sL + (g & 1) * 128 + grp * 32;
        const float* dl = sD + (g & 1) * 128 + grp * 32;
        if (!mbar_wait_warp(&lse_ready[g & 1], (g >> 1) & 1, status, kSiteAttention) ||
            !mbar_wait_warp(s_full, g & 1, status, kSiteAttention)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float p[32];
        tmem_ld_32x32b_x32(tS + my_cols, p);
        if constexpr (!CAP) {  // (a cap may need S^T once more)
          tc_fence_before();
          mbar_arrive_warp(s_free, lane);
        }
        // the next block's queries: loaded here, staged behind this block's work
        if (i + 1 < count) {
          have = true;
          if (grp == 0) load_query(bi, hh, r0, c0 + 128 + t);
        } else {
          look_ahead(r + 1);
        }
        const bool edge = sF[(g & 1) * 4 + grp] == 0;
        // bit e of vis: this key is visible to query e of the 32
        uint32_t vis = 0xFFFFFFFFu;
        if (edge) {
          const int range = sM[(g & 1) * 128 + grp * 32 + lane];
          vis = bit_transpose(
              bit_range((range & 255) - 32 * quarter, (range >> 8) - 32 * quarter), lane);
        }
        auto sees = [&](int e) { return ((vis >> e) & 1u) != 0; };
        // P (bf16 pairs in pp with a cap, else still in p), and in p what dP -
        // delta is multiplied by: P, with a cap P (1 - tanh^2).  pp ends up with
        // dz, pair for pair.
        uint32_t pp[16];
        const float d0 = static_cast<float>(c0 + grp * 32 - (r0 + t));  // query - key
        if constexpr (BIAS && !CAP) bias_scores<32>(p, sc.slope, d0);
        float u_max = 0.f;  // the largest square of a visible raw score
        auto weights = [&](auto edge_c, auto small_c) {
          constexpr bool EDGE = decltype(edge_c)::value;
          [[maybe_unused]] constexpr bool SMALL = decltype(small_c)::value;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 lv = *reinterpret_cast<const float4*>(l2 + e);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k = e + 2 * h;
              float2 add = h == 0 ? make_float2(-lv.x, -lv.y) : make_float2(-lv.z, -lv.w);
              if constexpr (BIAS && CAP) {
                add.x = fmaf(-sc.slope, fabsf(d0 + static_cast<float>(k)), add.x);
                add.y = fmaf(-sc.slope, fabsf(d0 + static_cast<float>(k + 1)), add.y);
              }
              const float2 x = make_float2(p[k], p[k + 1]);
              float2 y;
              [[maybe_unused]] float2 th;  // tanh
              if constexpr (CAP) {
                if constexpr (SMALL) {
                  const float2 u = __fmul2_rn(x, x);
                  if constexpr (EDGE)
                    u_max = fmax3f(u_max, sees(k) ? u.x : 0.f, sees(k + 1) ? u.y : 0.f);
                  else
                    u_max = fmax3f(u_max, u.x, u.y);
                  th = __fmul2_rn(x, cap_small(u, poly));
                } else {
                  th = __ffma2_rn(cap_r(x, sc.mul), make_float2(-2.f, -2.f), make_float2(1.f, 1.f));
                }
                y = __ffma2_rn(th, make_float2(sc.cap2, sc.cap2), add);
              } else {
                y = __ffma2_rn(x, make_float2(sc.mul, sc.mul), add);
              }
              float2 pv = make_float2(fast_exp2(y.x), fast_exp2(y.y));
              if constexpr (EDGE) {
                const bool v0 = sees(k), v1 = sees(k + 1);
                pv = make_float2(v0 ? pv.x : 0.f, v1 ? pv.y : 0.f);
                if constexpr (CAP) th = make_float2(v0 ? th.x : 0.f, v1 ? th.y : 0.f);
              }
              if constexpr (CAP) {
                pp[k / 2] = pack_bf16x2(pv.x, pv.y);  // dO's type (see the top)
                const float2 om = __ffma2_rn(make_float2(-th.x, -th.y), th, make_float2(1.f, 1.f));
                pv = __fmul2_rn(pv, om);
              }
              p[k] = pv.x;
              p[k + 1] = pv.y;
            }
          }
        };
        if (edge)
          weights(BoolC<true>{}, BoolC<true>{});
        else
          weights(BoolC<false>{}, BoolC<true>{});
        if constexpr (CAP) {
          // a visible score of the warp is not far enough below the cap (what is
          // masked must not decide how it is formed): the quotient form
          if (!__all_sync(0xffffffffu, u_max <= cap_limit2)) {
            tmem_ld_32x32b_x32(tS + my_cols, p);
            weights(BoolC<true>{}, BoolC<false>{});
          }
          tc_fence_before();
          mbar_arrive_warp(s_free, lane);
        }
        if (pending) {
          if (!mbar_wait_warp(acc_done, (g - 1) & 1, status, kSiteAttention)) {
            ok = false;
            break;
          }
          tc_fence_after();
          store_item(true, p_row, p_bi, p_head);
          tc_fence_before();
          pending = false;
        }
        if (!mbar_wait_warp(dp_full, g & 1, status, kSiteAttention)) {
          ok = false;
          break;
        }
        tc_fence_after();
        {
          float dv[32];
          tmem_ld_32x32b_x32(tdP + my_cols, dv);
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
              if constexpr (CAP) {
                w[e / 2] = pp[at / 2];
                w[e / 2 + 1] = pp[at / 2 + 1];
              } else {
                w[e / 2] = pack_bf16x2(p[at], p[at + 1]);
                w[e / 2 + 1] = pack_bf16x2(p[at + 2], p[at + 3]);
              }
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
        if (A.ds_tiles) {
          // The 128-byte-swizzled shared-memory image of an MN-major A operand:
          // 64-query chunks 16 KB apart, key row t at 128 B, the 16-byte unit
          // of queries [8u, 8u + 8) at unit u ^ (t & 7); the store of the
          // block before must have read sDs first.
          if (g > 0 && !mbar_wait_warp(ds_free, (g - 1) & 1, status, kSiteAttention)) {
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
        }
        if (have) stage_query((g + 1) & 1);
      }
      if (!ok) break;
      if (count > 0) {
        p_row = r0;
        p_bi = bi;
        p_head = hh;
        pending = true;
      } else {
        store_item(false, r0, bi, hh);
        look_ahead(r + 1);
        if (have) stage_query(g & 1);
      }
      mbar_arrive_warp(&it_empty[r % kOptKvRing], lane);
    }
    if (ok && pending && mbar_wait_warp(acc_done, (g - 1) & 1, status, kSiteAttention)) {
      tc_fence_after();
      store_item(true, p_row, p_bi, p_head);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- dQ, scores formed again
constexpr int kOptDqThreads = 384;
// As in the forward: 128 x 56 + 256 x 224 = 384 x 168.
constexpr int kOptDqRegsIo = 56, kOptDqRegsCompute = 224;

template <int D>
struct OptDqCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = 128 * D * 2;
  // Q, dO, three K stages, two V stages, barriers, alignment slack
  static constexpr int kUsed = 7 * kTile + 24 * 8 + 1024;
  static constexpr int kSmem = kUsed > 116 * 1024 ? kUsed : 116 * 1024;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kUsed <= 227 * 1024, "dq kernel shared memory");
};

// TMEM: S [0, 128), dP [128, 256), dQ [256, 256 + D), dz (bf16) [384, 448).
// The compute warps read S_j and dP_j into registers and release them at once
// (s_free), so S_{j+1} and dP_{j+1} run while dz_j is formed; dQ += dz_j K_j
// follows when dz_j is in TMEM (ds_full), and its completion (ds_free) lets
// dz_{j+1} be written.  Three products per block pair where the tiles need one:
// with the dK/dV kernel 297 us against 263 us for 4096 packed tokens of 64
// heads, 563 against 452 us for 8192 capped ones of 16; it needs no workspace.
template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kOptDqThreads, 1)
    attn_opt_dq_kernel(const __grid_constant__ CUtensorMap tm_qkv,
                       const __grid_constant__ CUtensorMap tm_do,
                       const __grid_constant__ OptBwdArgs A) {
  using C = OptDqCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sdO = smem + C::kTile;
  uint8_t* sK[3] = {smem + 2 * C::kTile, smem + 3 * C::kTile, smem + 4 * C::kTile};
  uint8_t* sV[2] = {smem + 5 * C::kTile, smem + 6 * C::kTile};
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + 7 * C::kTile);
  uint64_t* r_full = bars + 0;
  uint64_t* k_full = bars + 1;    // [3]
  uint64_t* k_empty = bars + 4;   // [3]
  uint64_t* v_full = bars + 7;    // [2]
  uint64_t* v_empty = bars + 9;   // [2]
  uint64_t* s_full = bars + 11;
  uint64_t* s_free = bars + 12;
  uint64_t* ds_full = bars + 13;
  uint64_t* ds_free = bars + 14;
  uint64_t* drain = bars + 15;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 16);
  int* status = A.status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = A.s, H = A.H, a = A.H * D;
  if (threadIdx.x == 0) {
    mbar_init(r_full, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, 8);
    mbar_init(ds_full, 8);
    mbar_init(ds_free, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_qkv);
    tma_prefetch_desc(&tm_do);
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
  const uint32_t tS = tmem, tdP = tmem + 128, tdQ = tmem + 256, tdS = tmem + 384;

  int4 entry;  // sequence, query block, lowest and highest visible key
  int hh;
  const bool ok_entry =
      opt_entry(A.tables, A.head_major != 0, A.b, (s + 127) / 128, entry, hh, status);
  const int bi = entry.x;
  const int q0 = entry.y * 128;
  const int k_lo = max(entry.z, 0), k_hi = min(entry.w, s);
  const int count = ok_entry && k_hi > k_lo ? (k_hi - k_lo + 127) / 128 : 0;

  if (warp < 4) {
    setmaxnreg_dec<kOptDqRegsIo>();
    if (warp == 0) {
      if (lane == 0 && count > 0) {
        // -------------------------------------------------------- producer
        mbar_arrive_expect_tx(r_full, 2 * C::kTile);
        for (int c = 0; c < C::kChunks; ++c) {
          tma_load_3d(sQ + c * 16384, &tm_qkv, r_full, hh * D + c * 64, q0, bi);
          tma_load_3d(sdO + c * 16384, &tm_do, r_full, hh * D + c * 64, q0, bi);
        }
        int k_issued = 0, v_issued = 0;
        for (int j = 0; j < count; ++j) {
          const int ks = j % 3, kph = (j / 3) & 1, vs = j & 1, vph = (j >> 1) & 1;
          if (!mbar_wait(&k_empty[ks], kph ^ 1u, status, kSiteAttention)) break;
          mbar_arrive_expect_tx(&k_full[ks], C::kTile);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(sK[ks] + c * 16384, &tm_qkv, &k_full[ks], a + hh * D + c * 64,
                        k_lo + j * 128, bi);
          ++k_issued;
          if (!mbar_wait(&v_empty[vs], vph ^ 1u, status, kSiteAttention)) break;
          mbar_arrive_expect_tx(&v_full[vs], C::kTile);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(sV[vs] + c * 16384, &tm_qkv, &v_full[vs], 2 * a + hh * D + c * 64,
                        k_lo + j * 128, bi);
          ++v_issued;
        }
        pdl_launch();  // every load of this CTA is issued
        mbar_wait(r_full, 0, status, kSiteAttention, 200000000ull, false);
        for (int j = k_issued - 1; j >= 0 && j >= k_issued - 3; --j)
          mbar_wait(&k_full[j % 3], (j / 3) & 1, status, kSiteAttention, 200000000ull, false);
        for (int j = v_issued - 1; j >= 0 && j >= v_issued - 2; --j)
          mbar_wait(&v_full[j & 1], (j >> 1) & 1, status, kSiteAttention, 200000000ull, false);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      // (converged, as in the dK/dV kernel)
      constexpr uint32_t kIdescSq = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t kIdescAcc = idesc_bf16_f32(128, D, false, true);
      const bool leader = elect_one();
      const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t do_desc = smem_desc_sw128(smem_u32(sdO), 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(smem_u32(sK[0]), 16, 1024);
      const uint64_t kt_desc = smem_desc_sw128(smem_u32(sK[0]), 16384, 1024);
      const uint64_t v_desc = smem_desc_sw128(smem_u32(sV[0]), 16, 1024);
      bool ok = count > 0 && mbar_wait_warp(r_full, 0, status, kSiteAttention);
      for (int j = 0; ok && j <= count; ++j) {
        if (j < count) {
          const int ks = j % 3, vs = j & 1;
          if (!mbar_wait_warp(&k_full[ks], (j / 3) & 1, status, kSiteAttention)) break;
          if (!mbar_wait_warp(&v_full[vs], (j >> 1) & 1, status, kSiteAttention)) break;
          // S / dP of block j - 1 are in the compute warps' registers.
          if (j > 0 && !mbar_wait_warp(s_free, (j - 1) & 1, status, kSiteAttention)) break;
          tc_fence_after();
          const uint64_t kd = smem_desc_add(k_desc, ks * C::kTile);
          const uint64_t vd = smem_desc_add(v_desc, vs * C::kTile);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
              umma_bf16(tS, smem_desc_add(q_desc, off), smem_desc_add(kd, off), kIdescSq,
                        kk > 0 ? 1u : 0u);
              umma_bf16(tdP, smem_desc_add(do_desc, off), smem_desc_add(vd, off), kIdescSq,
                        kk > 0 ? 1u : 0u);
            }
            umma_commit(s_full);
            umma_commit(&v_empty[vs]);  // V_j is done once dP_j is
          }
          __syncwarp();
        }
        if (j > 0) {
          const int pj = j - 1, pks = pj % 3;
          if (!mbar_wait_warp(ds_full, pj & 1, status, kSiteAttention)) break;
          tc_fence_after();
          const uint64_t kd = smem_desc_add(kt_desc, pks * C::kTile);
          const uint32_t acc0 = pj > 0 ? 1u : 0u;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 128 / 16; ++kk)
              umma_bf16_ts(tdQ, tdS + kk * 8, smem_desc_add(kd, kk * 2048), kIdescAcc,
                           kk > 0 ? 1u : acc0);
            umma_commit(&k_empty[pks]);
            umma_commit(ds_free);
          }
          __syncwarp();
        }
      }
      if (leader) {
        umma_commit(drain);
        mbar_wait(drain, 0, status, kSiteAttention, 200000000ull, false);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- compute
    setmaxnreg_inc<kOptDqRegsCompute>();
    const int quarter = warp & 3;
    const int half = (warp - 4) >> 2;   // 64 of the block's 128 key columns
    const int r = q0 + quarter * 32 + lane;  // this thread's query row
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const ScoreConst sc =
        score_const<CAP, BIAS>(rsqrtf(static_cast<float>(D)), A.softcap, BIAS ? A.slopes[hh] : 0.f);
    float my_l2 = 0.f, my_d = 0.f;
    int lo = 0, hi = 0x7fffffff;  // rows past the sequence: zeros, never stored
    if (ok_entry && r < s) {
      const int64_t hrow = (static_cast<int64_t>(bi) * H + hh) * s;
      my_l2 = A.lse[hrow + r] * kOptLog2e;
      my_d = A.delta[hrow + r];
      lo = max(A.key_lo[static_cast<int64_t>(bi) * s + r], 0);
      hi = max(min(A.key_hi[static_cast<int64_t>(bi) * s + r], s), 0);
    }
    const CapPoly poly = cap_poly(1.f, sc.arg);
    const float cap_limit = cap_small_limit(sc.arg);
    const float cap_limit2 = cap_limit * cap_limit;
    bool ok = true;
    for (int j = 0; j < count; ++j) {
      if (!mbar_wait_warp(s_full, j & 1, status, kSiteAttention)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float sv[64], dv[64];
      auto load = [&]() {
        tmem_ld_32x32b_x32_nowait(tS + lane_off + half * 64, sv);
        tmem_ld_32x32b_x32_nowait(tS + lane_off + half * 64 + 32, sv + 32);
        tmem_ld_32x32b_x32_nowait(tdP + lane_off + half * 64, dv);
        tmem_ld_32x32b_x32_nowait(tdP + lane_off + half * 64 + 32, dv + 32);
        tmem_ld_wait();
      };
      load();
      if constexpr (!CAP) {  // (a cap may need S and dP once more)
        tc_fence_before();
        mbar_arrive_warp(s_free, lane);
      }
      const int c0 = k_lo + j * 128 + half * 64;
      const bool edge = __any_sync(0xffffffffu, lo > c0 || hi < c0 + 64);
      // bit e of vis: this query sees key e of the 64
      uint32_t vis[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
      if (edge) {
        vis[0] = bit_range(lo - c0, hi - c0);
        vis[1] = bit_range(lo - c0 - 32, hi - c0 - 32);
      }
      uint32_t dw[32];
      const float2 nd2 = make_float2(-my_d, -my_d);
      const float d0 = static_cast<float>(c0 - r);  // key - query
      if constexpr (BIAS && !CAP) bias_scores<64>(sv, sc.slope, d0);
      float u_max = 0.f;  // the largest square of a visible raw score
      auto gradients = [&](auto edge_c, auto small_c) {
        constexpr bool EDGE = decltype(edge_c)::value;
        [[maybe_unused]] constexpr bool SMALL = decltype(small_c)::value;
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          float2 add = make_float2(-my_l2, -my_l2);
          if constexpr (BIAS && CAP) {
            add.x = fmaf(-sc.slope, fabsf(d0 + static_cast<float>(e)), add.x);
            add.y = fmaf(-sc.slope, fabsf(d0 + static_cast<float>(e + 1)), add.y);
          }
          const float2 x = make_float2(sv[e], sv[e + 1]);
          const bool v0 = !EDGE || ((vis[e >> 5] >> (e & 31)) & 1u);
          const bool v1 = !EDGE || ((vis[e >> 5] >> ((e + 1) & 31)) & 1u);
          float2 y;
          [[maybe_unused]] float2 th;
          if constexpr (CAP) {
            if constexpr (SMALL) {
              const float2 u = __fmul2_rn(x, x);
              u_max = fmax3f(u_max, v0 ? u.x : 0.f, v1 ? u.y : 0.f);
              th = __fmul2_rn(x, cap_small(u, poly));
            } else {
              th = __ffma2_rn(cap_r(x, sc.mul), make_float2(-2.f, -2.f), make_float2(1.f, 1.f));
            }
            th = make_float2(v0 ? th.x : 0.f, v1 ? th.y : 0.f);
            y = __ffma2_rn(th, make_float2(sc.cap2, sc.cap2), add);
          } else {
            y = __ffma2_rn(x, make_float2(sc.mul, sc.mul), add);
          }
          float2 pv = make_float2(fast_exp2(y.x), fast_exp2(y.y));
          pv = make_float2(v0 ? pv.x : 0.f, v1 ? pv.y : 0.f);
          if constexpr (CAP)
            pv = __fmul2_rn(pv, __ffma2_rn(make_float2(-th.x, -th.y), th, make_float2(1.f, 1.f)));
          const float2 ds = __fmul2_rn(pv, __fadd2_rn(make_float2(dv[e], dv[e + 1]), nd2));
          dw[e / 2] = pack_bf16x2(ds.x, ds.y);
        }
      };
      if (edge)
        gradients(BoolC<true>{}, BoolC<true>{});
      else
        gradients(BoolC<false>{}, BoolC<true>{});
      if constexpr (CAP) {
        // as in the dK/dV kernel: the quotient form where a score needs it
        if (!__all_sync(0xffffffffu, u_max <= cap_limit2)) {
          load();
          gradients(BoolC<true>{}, BoolC<false>{});
        }
        tc_fence_before();
        mbar_arrive_warp(s_free, lane);
      }
      // dz_{j-1} must have been consumed by its dQ product.
      if (j > 0 && !mbar_wait_warp(ds_free, (j - 1) & 1, status, kSiteAttention)) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_st_32x32b_x32(tdS + lane_off + half * 32, dw);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive_warp(ds_full, lane);
    }
    if (count > 0 && ok) ok = mbar_wait_warp(ds_free, (count - 1) & 1, status, kSiteAttention);
    if (ok && ok_entry) {
      tc_fence_after();
      const int warp_row = q0 + quarter * 32;
      uint16_t* base =
          A.dqkv + (static_cast<int64_t>(bi) * s + warp_row) * 3 * a + hh * D;
      const bool in_range = MC_DCHECK(warp_row >= 0 && hh * D + D <= a, status, kSiteAttention);
#pragma unroll 1
      for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {
        float v[32] = {};
        if (count > 0) tmem_ld_32x32b_x32(tdQ + lane_off + c * 32, v);
        store_rows32(base + c * 32, 3ll * a, in_range ? s - warp_row : 0, v,
                     rsqrtf(static_cast<float>(D)), lane);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- dQ from the dz^T tiles
template <int D>
struct OptDqGemmCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kKTile = 128 * D * 2;
  static constexpr int kStage = static_cast<int>(kOptTileBytes) + kKTile;
  static constexpr int kStages = 3;
  static constexpr int kUsed = kStages * kStage + 24 * 8 + 4 * 32;  // barriers, items
  // one CTA per SM, so that the CTAs that do not start are there to be stolen
  static constexpr int kSmem = kUsed + 1024 > 116 * 1024 ? kUsed + 1024 : 116 * 1024;
  static_assert(kSmem <= 227 * 1024, "dq gemm shared memory");
  static constexpr uint32_t kTmemCols = 256;  // two accumulators of 128 columns
};

// What every role needs to know of an item: a (query block, head) pair.
struct alignas(16) OptDqItem {
  int4 entry;  // sequence, query block, first key block, key blocks (-1: no more items)
  int head;
  int pad[3];
};
constexpr int kOptDqRing = 4;

// Persistent, 192 threads: warp 0 loads per key block the dz^T tile (one bulk
// copy of its swizzled image) and K_j into a 3-deep ring that runs on across
// items, warp 1 issues dQ += dz_j K_j (items alternate accumulators), warps
// 2..5 write dQ / sqrt(d) of the item before.  Bound by HBM: 4096 packed tokens
// of 64 heads move 423 MB in 68 us (6.2 TB/s), a causal mask over them 1.38 GB
// in 200 us (6.9 TB/s: what the dK/dV kernel wrote last is still in L2).
template <int D>
__global__ void __launch_bounds__(192, 1)
    attn_opt_dq_gemm_kernel(const __grid_constant__ CUtensorMap tm_qkv,
                            const __grid_constant__ OptBwdArgs A) {
  using C = OptDqGemmCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStage);
  uint64_t* full = bars + 0;       // [3]
  uint64_t* empty = bars + 3;      // [3]
  uint64_t* acc_full = bars + 6;   // [2]  an item's dQ is complete in accumulator a
  uint64_t* acc_empty = bars + 8;  // [2]  the epilogue has read accumulator a (4 warps)
  uint64_t* drain = bars + 10;
  uint64_t* it_full = bars + 11;   // [kOptDqRing]
  uint64_t* it_empty = bars + 15;  // [kOptDqRing] read by the MMA and epilogue warps (5)
  uint64_t* steal_bar = bars + 19;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 20);
  void* response = bars + 22;  // 16 bytes, aligned as the stages are
  OptDqItem* items = reinterpret_cast<OptDqItem*>(bars + 24);
  int* status = A.status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = A.s, H = A.H, a = A.H * D;
  const int nb = (s + 127) / 128;
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
    for (int i = 0; i < kOptDqRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], 5);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_qkv);
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

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------------- producer
      int gt = 0;  // tiles issued, across items
      bool ok = true;
      OptItems steal(response, steal_bar, A.b * nb * H, A.steal);
      int4 e_next = make_int4(0, 0, 0, 0);
      int h_next = 0;
      auto read_entry = [&]() {
        int rank = 0;
        if (steal.more) {
          opt_item(steal.k, A.b * nb, H, A.head_group, rank, h_next);
          h_next = H - 1 - h_next;  // the heads whose tiles were written last are still in L2
          e_next = *reinterpret_cast<const int4*>(A.tables + 4ll * rank);
        }
      };
      read_entry();
      for (int r = 0;; ++r) {
        int4 cur = make_int4(0, 0, 0, -1);
        const int hh = h_next;
        if (steal.more) {
          const int4 e = opt_checked(e_next, A.b, nb, status);
          const int lo = max(e.z, 0), hi = min(e.w, s);
          const int kb0 = lo / 128;
          int end = hi > lo ? (hi + 127) / 128 : kb0;
          if (A.causal) end = min(end, e.y + 1);  // the workspace has no other tiles
          cur = make_int4(e.x, e.y, kb0, max(end - kb0, 0));
        }
        const int slot = r % kOptDqRing;
        if (!mbar_wait(&it_empty[slot], ((r / kOptDqRing) & 1) ^ 1u, status, kSiteAttention)) break;
        items[slot].entry = cur;
        items[slot].head = hh;
        mbar_arrive(&it_full[slot]);
        if (cur.w < 0) break;
        const int64_t hb = static_cast<int64_t>(cur.x) * H + hh;
        for (int j = 0; j < cur.w; ++j, ++gt) {
          const int st = gt % C::kStages;
          if (!mbar_wait(&empty[st], ((gt / C::kStages) & 1) ^ 1u, status, kSiteAttention)) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + st * C::kStage;
          mbar_arrive_expect_tx(&full[st], C::kStage);
          bulk_load(dst,
                    A.ds_tiles + opt_tile(A.causal, nb, hb, cur.y, cur.z + j) * kOptTileBytes,
                    static_cast<uint32_t>(kOptTileBytes), &full[st]);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(dst + kOptTileBytes + c * 16384, &tm_qkv, &full[st], a + hh * D + c * 64,
                        (cur.z + j) * 128, cur.x);
        }
        if (!ok || !steal.next(status)) break;
        read_entry();
      }
      steal.finish(status);
      pdl_launch();  // every load of this CTA is issued
      for (int g = gt - 1; g >= 0 && g >= gt - C::kStages; --g)
        mbar_wait(&full[g % C::kStages], (g / C::kStages) & 1, status, kSiteAttention,
                  200000000ull, false);
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
      const int slot = r % kOptDqRing;
      if (!mbar_wait_warp(&it_full[slot], (r / kOptDqRing) & 1, status, kSiteAttention)) break;
      const int nj = __shfl_sync(0xffffffffu, items[slot].entry.w, 0);
      if (leader) mbar_arrive(&it_empty[slot]);
      if (nj < 0) break;
      const int acc = r & 1;
      // the epilogue of item r - 2 has read this accumulator
      if (!mbar_wait_warp(&acc_empty[acc], ((r >> 1) & 1) ^ 1u, status, kSiteAttention)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem + static_cast<uint32_t>(acc * 128);
      for (int j = 0; j < nj; ++j, ++gt) {
        const int st = gt % C::kStages;
        if (!mbar_wait_warp(&full[st], (gt / C::kStages) & 1, status, kSiteAttention)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t ad = smem_desc_add(a_desc, st * C::kStage);
        const uint64_t kd = smem_desc_add(ad, static_cast<uint32_t>(kOptTileBytes));
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
      mbar_wait(drain, 0, status, kSiteAttention, 200000000ull, false);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- epilogue
    const int quarter = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float scale = rsqrtf(static_cast<float>(D));
    for (int r = 0;; ++r) {
      const int slot = r % kOptDqRing;
      if (!mbar_wait_warp(&it_full[slot], (r / kOptDqRing) & 1, status, kSiteAttention)) break;
      const int4 e = items[slot].entry;
      const int hh = items[slot].head;
      mbar_arrive_warp(&it_empty[slot], lane);
      if (e.w < 0) break;
      const int bi = e.x, qb = e.y, nj = e.w;
      const int acc = r & 1;
      const int warp_row = qb * 128 + quarter * 32;
      if (!mbar_wait_warp(&acc_full[acc], (r >> 1) & 1, status, kSiteAttention)) break;
      tc_fence_after();
      uint16_t* base = A.dqkv + (static_cast<int64_t>(bi) * s + warp_row) * 3 * a + hh * D;
      const bool in_range = MC_DCHECK(warp_row >= 0 && hh * D + D <= a, status, kSiteAttention);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float v[32] = {};
        if (nj > 0)
          tmem_ld_32x32b_x32(tmem + static_cast<uint32_t>(acc * 128) + lane_off + c * 32, v);
        store_rows32(base + c * 32, 3ll * a, in_range ? s - warp_row : 0, v, scale, lane);
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
dim3 opt_dq_grid(const OptBwdArgs& A) {
  const unsigned n = static_cast<unsigned>(A.b) * static_cast<unsigned>((A.s + 127) / 128);
  return A.head_major ? dim3(static_cast<unsigned>(A.H), n, 1u)
                      : dim3(n, static_cast<unsigned>(A.H), 1u);
}

template <class K>
cudaError_t opt_smem(PerDeviceInit& init, K kern, int bytes) {
  return once_per_device(init, [&](long long*) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}

template <int D, bool CAP, bool BIAS>
int launch_bwd(const CUtensorMap& tq, const CUtensorMap& td, const OptBwdArgs& A,
               cudaStream_t st) {
  static PerDeviceInit init_kv, init_q;
  auto kv = attn_opt_dkdv_kernel<D, CAP, BIAS>;
  if (opt_smem(init_kv, kv, OptBwdCfg<D>::kSmem) != cudaSuccess) return MC_ERR_CUDA;
  launch_kernel(kv, dim3(static_cast<unsigned>(A.ctas)), dim3(kOptKvThreads), OptBwdCfg<D>::kSmem,
                st, 1, tq, td, A);
  if (cudaGetLastError() != cudaSuccess) return MC_ERR_CUDA;
  if (A.ds_tiles) return MC_OK;
  auto kq = attn_opt_dq_kernel<D, CAP, BIAS>;
  if (opt_smem(init_q, kq, OptDqCfg<D>::kSmem) != cudaSuccess) return MC_ERR_CUDA;
  launch_kernel(kq, opt_dq_grid(A), dim3(kOptDqThreads), OptDqCfg<D>::kSmem, st, 1, tq, td, A);
  return cudaGetLastError() == cudaSuccess ? MC_OK : MC_ERR_CUDA;
}

template <int D>
int launch_bwd_d(const uint16_t* qkv, const uint16_t* dout, const OptBwdArgs& A,
                 cudaStream_t st) {
  const uint64_t a = static_cast<uint64_t>(A.H) * D, s = static_cast<uint64_t>(A.s),
                 b = static_cast<uint64_t>(A.b);
  const uint32_t box[3] = {64, 128, 1};
  const uint64_t dq[3] = {3 * a, s, b}, sq[2] = {3 * a * 2, 3 * a * 2 * s};
  const uint64_t dd[3] = {a, s, b}, sd[2] = {a * 2, a * 2 * s};
  CUtensorMap tq, td;
  if (!make_tmap_bf16(&tq, qkv, 3, dq, sq, box) || !make_tmap_bf16(&td, dout, 3, dd, sd, box))
    return MC_ERR_CUDA;
  const bool cap = A.softcap > 0.f, bias = A.slopes != nullptr;
  int rc;
  if (cap)
    rc = bias ? launch_bwd<D, true, true>(tq, td, A, st) : launch_bwd<D, true, false>(tq, td, A, st);
  else
    rc = bias ? launch_bwd<D, false, true>(tq, td, A, st) : launch_bwd<D, false, false>(tq, td, A, st);
  if (rc != MC_OK || !A.ds_tiles) return rc;
  static PerDeviceInit init;
  auto kern = attn_opt_dq_gemm_kernel<D>;
  if (opt_smem(init, kern, OptDqGemmCfg<D>::kSmem) != cudaSuccess) return MC_ERR_CUDA;
  launch_kernel(kern, dim3(static_cast<unsigned>(A.ctas)), dim3(192), OptDqGemmCfg<D>::kSmem, st, 1,
                tq, A);
  return cudaGetLastError() == cudaSuccess ? MC_OK : MC_ERR_CUDA;
}

}  // namespace

int64_t attention_opt_ds_bytes(int64_t b, int64_t s, int64_t H, bool causal) {
  const int64_t nb = (s + 127) / 128;
  return b * H * (causal ? nb * (nb + 1) / 2 : nb * nb) * kOptTileBytes;
}

int launch_attention_opt_bwd(const uint16_t* qkv, const float* lse, const uint16_t* dout,
                             uint16_t* dqkv, const float* delta, int b, int s, int H, int d,
                             const mc_attention_options& opt, uint8_t* ds_tiles, int* status,
                             cudaStream_t st) {
  OptBwdArgs A = {};
  A.dqkv = dqkv;
  A.lse = lse;
  A.delta = delta;
  A.key_lo = opt.key_lo;
  A.key_hi = opt.key_hi;
  A.tables = opt.tables;
  A.slopes = opt.slopes;
  A.ds_tiles = ds_tiles;
  A.softcap = opt.softcap;
  A.b = b;
  A.s = s;
  A.H = H;
  A.head_major = attention_head_major(static_cast<int64_t>(b) * ((s + 127) / 128), H, 1) ? 1 : 0;
  const OptGrid grid = opt_grid(b, s, H, d);
  A.steal = grid.steal;
  A.head_group = grid.head_group;
  A.ctas = grid.ctas;
  A.causal = opt.causal ? 1 : 0;
  A.status = status;
  return d == 64 ? launch_bwd_d<64>(qkv, dout, A, st) : launch_bwd_d<128>(qkv, dout, A, st);
}

}  // namespace mc
