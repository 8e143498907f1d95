// Attention forward over interval masks (sm_103a, tcgen05), scores optionally
// capped by a tanh and biased by the distance:
//   O_i = sum_j P_ij V_j over the keys j in [lo_i, hi_i), P the softmax.
//
// Persistent: one CTA per SM walks the (128-query block, head) items, each
// over the 256-key blocks between its rows' lowest and highest key (the last
// one only half, where 128 keys or fewer are left) with one running maximum
// and sum per row.  384 threads:
//   warp 0       the items' table entries into shared memory, and TMA: Q once
//                per item, K blocks into a 2-deep ring, V as 128-key halves
//                into a ring, running on across items
//   warp 1       TMEM and the MMA thread: S = Q K^T, O += P V
//   warps 4..11  softmax, two warps per TMEM lane quarter: a thread takes 128
//                of its row's 256 scores; the two exchange maxima and sums
// S_{g+1} is formed while the softmax of block g runs (P has TMEM columns of
// its own), across items too: packed documents have items of one to a few
// blocks, which start-up and drain would dominate otherwise.
// TMEM: S [0, 256), O [256, 256 + D), P [384, 512) (bf16 pairs, 256 keys).
//
// Bound by the products (2870 clocks per block at D = 128) where nothing is
// capped or biased: causal over 16,384 tokens and 16 heads 703 us, 0.82 of the
// measured matrix rate.  With a cap (1035 to 1058 us, 4870 clocks per block) or a
// bias (867 us) neither the tensor pipe (45% active with a cap) nor the issue
// slots are full: the cap's multiply-adds take 1536 clocks and the exponentials
// 1024, on different units, and about 1600 are waits, the exchange of maxima and
// transfers, which nothing overlaps, because both warps of a lane quarter hold
// halves of the same rows and wait at the same barriers.  Over short documents
// (4096 tokens, 64 heads, 88 us, 3.0 TB/s) the partly masked blocks, the wait for
// an item's first S and the stores, 32 bytes per clock and SM, show.  128-key
// blocks in two CTAs per SM and softmax warps that take two passes were slower,
// as were sixteen softmax warps of 64 scores (packed 105 us, capped 1097 us) and
// storing O behind the next P (91, 1120 us).
//
// P is rounded to bf16, by at most 2^-8 of itself: an operand of a tcgen05
// product has the type of the other one, here V's.  The row sums take P before
// that, sums and statistics are 32-bit, and O is rounded once more when stored.
// Those two roundings are the kernel's whole error, 0.0017 to 0.0022 of the
// result; with P in 32 bits, O's alone leaves 0.0016 to 0.0017.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attention_opt.cuh"

namespace mc {
namespace {

constexpr int kOptFwdThreads = 384;
// The launch gives every thread 168 registers (384 x 168 = 64,512); the
// softmax warpgroups, which hold a row's 128 scores, take what the producer's
// leaves: 128 x 72 + 256 x 216 = 64,512.
constexpr int kOptRegsIo = 72, kOptRegsSoftmax = 216;
constexpr int kOptKeys = 256;  // keys per block
constexpr int kOptRing = 4;    // items in shared memory
// O is rescaled only when a row's maximum grows by more than this (log2
// units): P stays below 2^8 and the final division by the sum, taken against
// the same maximum, cancels the difference.
constexpr float kOptRescale = 8.0f;

// What every role needs to know of an item.
struct alignas(16) OptItem {
  int4 entry;  // sequence, query block, lowest visible key, 128-key halves (-1: no more items)
  int head;
  int pad[3];
};

template <int D>
struct OptFwdCfg {
  static constexpr int kChunks = D / 64;           // 128-byte boxes per row
  static constexpr int kQTile = 128 * D * 2;       // Q [128][D] bf16
  static constexpr int kKTile = kOptKeys * D * 2;  // K [256][D] bf16
  static constexpr int kChunkBytes = kOptKeys * 128;  // one 64-wide d chunk of 256 rows
  static constexpr int kHalf = 128 * D * 2;        // 128 rows of K or V
  static constexpr int kVSlots = D == 64 ? 4 : 2;
  static constexpr int kXch = 2 * 2 * 128 * 4;     // [parity][half][row] floats
  static constexpr int kBars = 38 * 8;  // and 16 bytes of work stealing
  // The dynamic shared memory starts 1024-byte aligned (checked at run time),
  // so no alignment slack is reserved: at D = 128 it would not fit.
  static constexpr int kUsed = kQTile + 2 * kKTile + kVSlots * kHalf + kXch +
                               kOptRing * static_cast<int>(sizeof(OptItem)) + kBars;
  static constexpr int kSmem = kUsed > 116 * 1024 ? kUsed : 116 * 1024;
  static_assert(kUsed <= 227 * 1024, "forward shared memory");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0, kColO = 256, kColP = 384;
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
  int steal, head_group;
  int* status;
};

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kOptFwdThreads, 1)
    attn_opt_fwd_kernel(const __grid_constant__ CUtensorMap tm,
                        const __grid_constant__ OptFwdArgs A) {
  using C = OptFwdCfg<D>;
  constexpr int VS = C::kVSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  int* status = A.status;
  if (smem_u32(smem) & 1023u) {  // the 128-byte swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) record_error(status, MC_ERR_DEVICE_BOUNDS, kSiteAttention);
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* sK[2] = {smem + C::kQTile, smem + C::kQTile + C::kKTile};
  uint8_t* sV0 = smem + C::kQTile + 2 * C::kKTile;
  float* xch = reinterpret_cast<float*>(sV0 + VS * C::kHalf);
  OptItem* items = reinterpret_cast<OptItem*>(reinterpret_cast<uint8_t*>(xch) + C::kXch);
  uint64_t* bars = reinterpret_cast<uint64_t*>(items + kOptRing);
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
  uint64_t* it_full = bars + 24;   // [kOptRing]
  uint64_t* it_empty = bars + 28;  // [kOptRing] read by the MMA thread and the softmax (257)
  uint64_t* steal_bar = bars + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 33);
  void* response = bars + 34;  // 16 bytes, aligned as the items are

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = A.s, a = A.H * D;
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
    for (int i = 0; i < kOptRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], 257);
    }
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
  const uint32_t tS = tmem + C::kColS, tO = tmem + C::kColO, tP = tmem + C::kColP;

  // Every role walks the same items (r) and blocks (g, across items).
  if (warp < 4) {
    setmaxnreg_dec<kOptRegsIo>();
    if (warp == 0) {
      if (lane == 0) {
        // -------------------------------------------------------- producer
        const int nb = (s + 127) / 128;
        int g = 0, u = 0, q_n = 0;  // K blocks, V halves and Q tiles issued
        bool ok = true;
        // V of a block is loaded after K of the next: what is left to load
        int v_halves = 0, v_row = 0, v_col = 0, v_bi = 0;
        auto load_v = [&]() {
          for (int h = 0; ok && h < v_halves; ++h) {
            const int slot = u % VS;
            if (!mbar_wait(&v_empty[slot], ((u / VS) & 1) ^ 1u, status, kSiteAttention)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&v_full[slot], C::kHalf);
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_3d(sV0 + slot * C::kHalf + c * 16384, &tm, &v_full[slot], v_col + c * 64,
                          v_row + h * 128, v_bi);
            ++u;
          }
          v_halves = 0;
        };
        // Items are announced one ahead, so that the softmax can fetch the next
        // one's intervals early, and their table entries are read two ahead.
        int4 e_next = make_int4(0, 0, 0, 0);
        int h_next = 0;
        OptItems steal(response, steal_bar, A.b * nb * A.H, A.steal);
        auto read_entry = [&]() {
          int rank = 0;
          if (steal.more) {
            opt_item(steal.k, A.b * nb, A.H, A.head_group, rank, h_next);
            e_next = *reinterpret_cast<const int4*>(A.tables + 4ll * rank);
          }
        };
        auto announce = [&](int r, OptItem& it) -> bool {
          it.entry = make_int4(0, 0, 0, -1);
          it.head = h_next;
          if (steal.more) {
            const int4 e = opt_checked(e_next, A.b, nb, status);
            const int k_lo = max(e.z, 0), k_hi = min(e.w, s);
            it.entry = make_int4(e.x, e.y, k_lo, k_hi > k_lo ? (k_hi - k_lo + 127) / 128 : 0);
          }
          const int slot = r % kOptRing;
          if (!mbar_wait(&it_empty[slot], ((r / kOptRing) & 1) ^ 1u, status, kSiteAttention))
            return false;
          items[slot].entry = it.entry;
          items[slot].head = it.head;
          mbar_arrive(&it_full[slot]);
          return true;
        };
        OptItem cur, next;
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
          const int bi = cur.entry.x, k_lo = cur.entry.z, halves = cur.entry.w;
          const int hh = cur.head;
          // Announcing waits for an earlier item's softmax, which waits for its
          // last V: with empty items in between that V is not left pending.
          if (halves == 0) load_v();
          const bool early = r > 0 || halves == 0;  // (the first item's loads go first)
          if (ok && early) ok = go_on(r);
          for (int j = 0; ok && 2 * j < halves; ++j, ++g) {
            if (j == 0) {
              if (!(ok = mbar_wait(q_empty, (q_n & 1) ^ 1u, status, kSiteAttention))) break;
              mbar_arrive_expect_tx(q_full, C::kQTile);
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_3d(sQ + c * 16384, &tm, q_full, hh * D + c * 64, cur.entry.y * 128, bi);
              ++q_n;
            }
            const int ks = g & 1, nh = min(2, halves - 2 * j);
            if (!(ok = mbar_wait(&k_empty[ks], ((g >> 1) & 1) ^ 1u, status, kSiteAttention))) break;
            mbar_arrive_expect_tx(&k_full[ks], nh * C::kHalf);
            for (int c = 0; c < C::kChunks; ++c)
              for (int h = 0; h < nh; ++h)
                tma_load_3d(sK[ks] + c * C::kChunkBytes + h * 16384, &tm, &k_full[ks],
                            a + hh * D + c * 64, k_lo + j * kOptKeys + h * 128, bi);
            if (j == 0 && !early && !(ok = go_on(r))) {
              ++g;
              break;
            }
            load_v();
            v_halves = nh;
            v_row = k_lo + j * kOptKeys;
            v_col = 2 * a + hh * D;
            v_bi = bi;
          }
        }
        if (ok) load_v();
        steal.finish(status);
        pdl_launch();  // every load of this CTA is issued
        // Copies still in flight must land before the CTA exits.
        if (q_n > 0) mbar_wait(q_full, (q_n - 1) & 1, status, kSiteAttention, 200000000ull, false);
        for (int i = g - 1; i >= 0 && i >= g - 2; --i)
          mbar_wait(&k_full[i & 1], (i >> 1) & 1, status, kSiteAttention, 200000000ull, false);
        for (int i = u - 1; i >= 0 && i >= u - VS; --i)
          mbar_wait(&v_full[i % VS], (i / VS) & 1, status, kSiteAttention, 200000000ull, false);
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
      int p_halves = 0;               // the block whose O += P V is still to be issued
      bool p_first = false, ok = true;
      auto issue_pv = [&](int gp) -> bool {
        if (!mbar_wait_warp(p_full, gp & 1, status, kSiteAttention)) return false;
        // the previous item's O has been read
        if (p_first && n_items > 1 &&
            !mbar_wait_warp(o_free, n_items & 1, status, kSiteAttention))
          return false;
        for (int h = 0; h < p_halves; ++h, ++u) {
          const int slot = u % VS;
          if (!mbar_wait_warp(&v_full[slot], (u / VS) & 1, status, kSiteAttention)) return false;
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
        const int slot = r % kOptRing;
        if (!(ok = mbar_wait_warp(&it_full[slot], (r / kOptRing) & 1, status, kSiteAttention)))
          break;
        const int halves = __shfl_sync(0xffffffffu, items[slot].entry.w, 0);
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
              const int first = mbar_wait_first(q_full, n_items & 1, p_full, (g - 1) & 1, status,
                                                kSiteAttention);
              if (__all_sync(0xffffffffu, first == 2)) {
                if (!(ok = issue_pv(g - 1))) break;
                p_halves = 0;
              }
            }
            if (!(ok = mbar_wait_warp(q_full, n_items & 1, status, kSiteAttention))) break;
          }
          if (!(ok = mbar_wait_warp(&k_full[ks], (g >> 1) & 1, status, kSiteAttention))) break;
          // S still holds block g - 1 until the softmax has it in registers.
          if (g > 0 && !(ok = mbar_wait_warp(s_free, (g - 1) & 1, status, kSiteAttention))) break;
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
          p_first = j == 0;
          if (j == 0) ++n_items;
        }
      }
      if (ok && p_halves > 0) issue_pv(g - 1);
      if (leader) {
        umma_commit(drain);
        mbar_wait(drain, 0, status, kSiteAttention, 200000000ull, false);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- softmax
    setmaxnreg_inc<kOptRegsSoftmax>();
    const int quarter = warp & 3;
    const int half = (warp - 4) >> 2;  // keys [128 half, 128 half + 128) of a block
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
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
      if (!mbar_wait(&xbar[quarter], xphase & 1, status, kSiteAttention)) ok = false;
      const float peer = xch[(xphase & 1) * 256 + (half ^ 1) * 128 + row];
      ++xphase;
      return peer;
    };
    // This row's interval and slope in item r, fetched one item ahead.  Rows
    // past the sequence (zeros from the TMA, never stored) see everything, so
    // that they do not make a block an edge.
    int lo = 0, hi = 0;
    float slope = 0.f;
    auto fetch = [&](int r) {
      const int slot = r % kOptRing;
      if (!mbar_wait_warp(&it_full[slot], (r / kOptRing) & 1, status, kSiteAttention)) {
        ok = false;
        return;
      }
      const OptItem& it = items[slot];
      lo = 0;
      hi = 0x7fffffff;
      const int q = it.entry.y * 128 + row;
      if (it.entry.w >= 0 && q < s) {
        lo = A.key_lo[static_cast<int64_t>(it.entry.x) * s + q];
        hi = A.key_hi[static_cast<int64_t>(it.entry.x) * s + q];
        if constexpr (BIAS) slope = A.slopes[it.head];
      }
    };
    fetch(0);
    // The item before, whose O is still in TMEM: its products run during this
    // item's first softmax, and it is stored once they are complete.
    bool pending = false;
    float p_l = 0.f, p_m = 0.f;
    int p_q = 0, p_bi = 0, p_head = 0;
    auto store_item = [&](bool from_tmem) {
      // a row that sees nothing: O = 0, log-sum-exp = -infinity
      const float inv = p_l == 0.f ? 0.f : 1.f / p_l;
      const int q_warp = p_q - lane;  // the warp's first row
      uint16_t* base = A.out + (static_cast<int64_t>(p_bi) * s + q_warp) * a + p_head * D +
                       half * (D / 2);
      const bool in_range = MC_DCHECK(q_warp >= 0 && p_bi >= 0 && p_bi < A.b && p_head * D + D <= a,
                                      status, kSiteAttention);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {  // this thread's half of the row's O
        float v[32] = {};
        if (from_tmem) {
          tmem_ld_32x32b_x32(tO + lane_off + half * (D / 2) + c * 32, v);
          if (c == D / 64 - 1) {
            tc_fence_before();
            mbar_arrive(o_free);  // the next products may overwrite O
          }
        }
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = p_l == 0.f ? 0u : pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
        transpose_16b_x4(w, lane);
        if (in_range) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r4 = (lane & ~3) + k;  // row of the warp: 4 lanes store its 64 bytes
            if (q_warp + r4 < s)
              *reinterpret_cast<uint4*>(base + static_cast<int64_t>(r4) * a + c * 32 +
                                        (lane & 3) * 8) =
                  make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
          }
        }
      }
      if (half == 0 && in_range && p_q < s)
        A.lse[(static_cast<int64_t>(p_bi) * A.H + p_head) * s + p_q] =
            p_l == 0.f ? -INFINITY : (p_m + log2f(p_l)) * kOptLn2;
    };
    int g = 0;
    for (int r = 0; ok; ++r) {
      const OptItem& it = items[r % kOptRing];
      const int halves = it.entry.w;
      if (halves < 0) break;
      const int q = it.entry.y * 128 + row, k_lo = it.entry.z;
      // cut to the sequence (a caller's bounds are any 32-bit integers, from which
      // nothing may be subtracted)
      const int row_lo = max(lo, 0), row_hi = q < s ? max(min(hi, s), 0) : hi;
      const ScoreConst sc =
          score_const<CAP, BIAS>(rsqrtf(static_cast<float>(D)), A.softcap, slope);
      const CapPoly poly = cap_poly(sc.cap2, sc.arg);
      const float cap_limit = cap_small_limit(sc.arg);
      const bool early = r > 0 || halves == 0;
      if (early) fetch(r + 1);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; 2 * j < halves; ++j, ++g) {
        if (!ok || !mbar_wait_warp(s_full, g & 1, status, kSiteAttention)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_ld_32x32b_x32_nowait(tS + lane_off + half * 128 + 32 * c, x + 32 * c);
        tmem_ld_wait();
        tc_fence_before();
        // (one arrival per warp: the same with a cap, 712 against 703 us without)
        mbar_arrive(s_free);
        const int key0 = k_lo + j * kOptKeys + half * 128;
        // ---- keys [first, end) of this half are visible (the last block may lack
        //      its second half, whose S is an older one)
        const int first = row_lo - key0;
        const int end = 2 * j + half < halves ? row_hi - key0 : 0;
        const bool cut = __any_sync(0xffffffffu, end < 128 || first > 0);
        // bit i of vis: key i is visible
        uint32_t vis[4] = {};
        if (cut) {
#pragma unroll
          for (int c = 0; c < 4; ++c) vis[c] = bit_range(first - 32 * c, end - 32 * c);
        }
        auto sees = [&](int i) { return ((vis[i >> 5] >> (i & 31)) & 1u) != 0; };
        // With a cap and a bias the scores are formed here, in log2 units; a bias
        // alone is taken off the raw scores.  Those stay raw until the exponent:
        // the scale is positive and the cap monotone, so the raw maximum gives
        // the row's.
        // A cap needs the lowest visible score too: whether the warp's visible
        // scores are far enough below it (masked ones must not decide how the
        // cap is formed).
        auto below_cap = [&](float high) {
          float low = INFINITY, lo1 = INFINITY;
          if (cut) {
#pragma unroll
            for (int i = 0; i < 128; i += 2) {
              low = fminf(low, sees(i) ? x[i] : INFINITY);
              lo1 = fminf(lo1, sees(i + 1) ? x[i + 1] : INFINITY);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 128; i += 4) {
              low = fmin3f(low, x[i], x[i + 1]);
              lo1 = fmin3f(lo1, x[i + 2], x[i + 3]);
            }
          }
          return __all_sync(0xffffffffu, fmaxf(high, -fminf(low, lo1)) <= cap_limit);
        };
        const float2 m2cap2 = make_float2(-2.f * sc.cap2, -2.f * sc.cap2);
        if constexpr (BIAS) {
          if constexpr (CAP) {
            float high = -INFINITY;
            if (cut) {
#pragma unroll
              for (int i = 0; i < 128; ++i)
                high = fmaxf(high, sees(i) ? x[i] : -INFINITY);
            } else {
#pragma unroll
              for (int i = 0; i < 128; i += 2) high = fmax3f(high, x[i], x[i + 1]);
            }
            if (below_cap(high)) {
#pragma unroll
              for (int i = 0; i < 64; ++i) {
                const float2 xi = make_float2(x[2 * i], x[2 * i + 1]);
                const float2 y = __fmul2_rn(xi, cap_small(__fmul2_rn(xi, xi), poly));
                x[2 * i] = y.x;
                x[2 * i + 1] = y.y;
              }
            } else {
#pragma unroll
              for (int i = 0; i < 64; ++i) {
                const float2 y = __ffma2_rn(cap_r(make_float2(x[2 * i], x[2 * i + 1]), sc.mul),
                                            m2cap2, make_float2(sc.cap2, sc.cap2));
                x[2 * i] = y.x;
                x[2 * i + 1] = y.y;
              }
            }
          }
          bias_scores<128>(x, sc.slope, static_cast<float>(key0 - q));
        }
        if (cut) {
#pragma unroll
          for (int i = 0; i < 128; ++i) x[i] = sees(i) ? x[i] : -INFINITY;
        }
        // ---- row maximum: four chains of three-input maxima, then a tree
        float mc[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int p = 0; p < 62; ++p) mc[p & 3] = fmax3f(mc[p & 3], x[4 + 2 * p], x[5 + 2 * p]);
        float mx = fmaxf(fmax3f(mc[0], mc[1], mc[2]), mc[3]);
        offer(mx);
        const bool small = CAP && !BIAS && below_cap(mx);  // while the other half's is awaited
        mx = fmaxf(mx, take());
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        if constexpr (!CAP) {
          mx *= sc.mul;
        } else if constexpr (!BIAS) {
          if (mx > -INFINITY) mx = fmaf(cap_r(make_float2(mx, mx), sc.mul).x, m2cap2.x, sc.cap2);
        }
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
        // ---- P, its row sum in 32 bits, and P as bf16 in registers, while the
        //      products of the block before may still run (in place: pair i of
        //      the bf16 P takes score i's register, which pair i / 2 was the
        //      last to need)
        float2 sm2[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
        // kForm 0: y = x mul - m, 1: x is y, 2: capped by the polynomial, 3: by
        // the quotient
        auto exponentials = [&](auto form_c, auto cut_c) {
          constexpr int kForm = decltype(form_c)::value;
          constexpr bool CUT = decltype(cut_c)::value;
          const float2 mul2 = make_float2(sc.mul, sc.mul), negm2 = make_float2(-m_use, -m_use);
          const float2 off2 = make_float2(sc.cap2 - m_use, sc.cap2 - m_use);
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            const float2 xi = make_float2(x[2 * i], x[2 * i + 1]);
            float2 y;
            if constexpr (kForm == 0) {
              y = __ffma2_rn(xi, mul2, negm2);
            } else if constexpr (kForm == 1) {
              y = __fadd2_rn(xi, negm2);
            } else {
              if constexpr (kForm == 2) {
                y = __ffma2_rn(xi, cap_small(__fmul2_rn(xi, xi), poly), negm2);
              } else {
                y = __ffma2_rn(cap_r(xi, sc.mul), m2cap2, off2);
              }
            }
            float2 pv = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            if constexpr (CUT)  // (the cap of -infinity is not -infinity)
              pv = make_float2(sees(2 * i) ? pv.x : 0.f, sees(2 * i + 1) ? pv.y : 0.f);
            sm2[i & 3] = __fadd2_rn(sm2[i & 3], pv);
            x[i] = __uint_as_float(pack_bf16x2(pv.x, pv.y));  // V's type (see the top)
          }
        };
        if constexpr (!CAP) {
          exponentials(IntC<0>{}, BoolC<false>{});
        } else if constexpr (BIAS) {
          exponentials(IntC<1>{}, BoolC<false>{});
        } else {
          if (small) {
            if (cut)
              exponentials(IntC<2>{}, BoolC<true>{});
            else
              exponentials(IntC<2>{}, BoolC<false>{});
          } else {
            if (!cut) vis[0] = vis[1] = vis[2] = vis[3] = 0xFFFFFFFFu;
            exponentials(IntC<3>{}, BoolC<true>{});
          }
        }
        const float2 s01 = __fadd2_rn(__fadd2_rn(sm2[0], sm2[1]), __fadd2_rn(sm2[2], sm2[3]));
        l += s01.x + s01.y;
        // The products of block g - 1 have to be complete before O is rescaled
        // or P overwritten.
        if (g > 0 && !mbar_wait_warp(pv_done, (g - 1) & 1, status, kSiteAttention)) {
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
        if (j == 0 && !early) fetch(r + 1);
      }
      if (!ok) break;
      if (halves > 0) {
        offer(l);
        l += take();  // both halves' sums, taken against the same maximum
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        p_l = l;
        p_m = m;
        p_q = q;
        p_bi = it.entry.x;
        p_head = it.head;
        pending = true;
      } else {
        // nothing to see: stored at once (what is pending waits in its TMEM)
        const float l0 = p_l, m0 = p_m;
        const int q0 = p_q, b0 = p_bi, h0 = p_head;
        p_l = 0.f;
        p_q = q;
        p_bi = it.entry.x;
        p_head = it.head;
        store_item(false);
        p_l = l0, p_m = m0, p_q = q0, p_bi = b0, p_head = h0;
      }
      mbar_arrive(&it_empty[r % kOptRing]);
    }
    if (ok && pending && mbar_wait_warp(pv_done, (g - 1) & 1, status, kSiteAttention)) {
      tc_fence_after();
      store_item(true);
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
int launch_fwd(const uint16_t* qkv, const OptFwdArgs& A, int ctas, cudaStream_t st) {
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
  launch_kernel(kern, dim3(static_cast<unsigned>(ctas)), dim3(kOptFwdThreads), C::kSmem, st, 1, tm,
                A);
  return cudaGetLastError() == cudaSuccess ? MC_OK : MC_ERR_CUDA;
}

template <int D>
int launch_fwd_d(const uint16_t* qkv, const OptFwdArgs& A, int ctas, cudaStream_t st) {
  const bool cap = A.softcap > 0.f, bias = A.slopes != nullptr;
  if (cap)
    return bias ? launch_fwd<D, true, true>(qkv, A, ctas, st)
                : launch_fwd<D, true, false>(qkv, A, ctas, st);
  return bias ? launch_fwd<D, false, true>(qkv, A, ctas, st)
              : launch_fwd<D, false, false>(qkv, A, ctas, st);
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
  const OptGrid grid = opt_grid(b, s, H, d);
  A.steal = grid.steal;
  A.head_group = grid.head_group;
  A.status = status;
  return d == 64 ? launch_fwd_d<64>(qkv, A, grid.ctas, st)
                 : launch_fwd_d<128>(qkv, A, grid.ctas, st);
}

}  // namespace mc
