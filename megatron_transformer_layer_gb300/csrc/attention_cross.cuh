// What the kernels of the attention to keys of another length share: the
// layout of its sequences, items, and tensor maps.
//
// A block of queries is 128 rows of a score tile: the G query heads that share
// a key head of each of pq = 128 / G (rounded down) queries, row r being head
// r % G of query r / G.  So grouped heads read their keys once, a single new
// token of G heads takes one tile, and dK and dV are summed over the group in
// the products themselves.  (G = 1: 128 queries of one head.)
#pragma once
#include "attention_opt.cuh"
#include "mc_layer_internal.h"
#include "ptx.cuh"

namespace mc {

struct CrossArgs {
  const int32_t *q_off, *q_len, *kv_off, *kv_len;
  int n, H, KV, G;
  int pq;           // queries of a block
  int nqb, nkb;     // blocks of a sequence, at most
  int q_rows, kv_rows;
  int max_q, max_kv;  // rows of a sequence: what the blocks cover, or the equal runs
  int64_t ld_q, ld_kv, ld_o;
  float scale;
  uint32_t div_g;   // fast division of a row by G
  int* status;
};

// A sequence's rows: where they start, how many there are, how many are real.
struct CrossRows {
  int first, slot, real;
};

__device__ __forceinline__ CrossRows cross_rows(const int32_t* off, const int32_t* len, int rows,
                                                int most, int n, int* status) {
  CrossRows r;
  r.first = n * most;
  r.slot = most;
  if (off) {
    r.first = min(max(off[n], 0), rows);
    r.slot = min(max(off[n + 1], r.first), rows) - r.first;
    if (r.slot > most) {
      record_error(status, MC_ERR_DEVICE_BOUNDS, kSiteCross);
      r.slot = most;
    }
  }
  r.real = len ? min(max(len[n], 0), r.slot) : r.slot;
  return r;
}
__device__ __forceinline__ CrossRows cross_queries(const CrossArgs& A, int n) {
  return cross_rows(A.q_off, A.q_len, A.q_rows, A.max_q, n, A.status);
}
__device__ __forceinline__ CrossRows cross_keys(const CrossArgs& A, int n) {
  return cross_rows(A.kv_off, A.kv_len, A.kv_rows, A.max_kv, n, A.status);
}

// Item k of the sequences by `heads` key heads by `blocks` blocks: the blocks of a
// head one after another, so that CTAs that run together read the same K and V (or Q
// and dO), which counts even where those stay in L2 either way: heads first, in groups
// of at most 32 MB of them, with one CTA per SM, 4 x 1037 queries of 64 heads to 256
// keys took 81 us against 74, 4096 to 8192 780 against 755.
struct CrossItem {
  int n, hk, block;
};
__device__ __forceinline__ CrossItem cross_item(int k, int heads, int blocks) {
  CrossItem it;
  const int per_seq = heads * blocks;
  it.n = k / per_seq;
  const int in = k - it.n * per_seq;
  it.hk = in / blocks;
  it.block = in - it.hk * blocks;
  return it;
}

// Row r of a block: its query and its head within the group.
__device__ __forceinline__ int cross_query(const CrossArgs& A, int r) {
  return A.div_g == 0 ? r : static_cast<int>(__umulhi(static_cast<uint32_t>(r), A.div_g));
}

// Tensor maps.  Boxes of 128 rows may run over the end of a sequence into the
// padding or the next one: what they bring from there never reaches a result
// (cross_clear_tail, and selects on the scores).
//   Q, O:  {head_dim, heads, rows}, boxes {64, G, pq}: the rows of a block
//          (G = 1: {heads head_dim, rows, 1}, boxes {64, 128, 1})
//   K, V:  {kv_heads head_dim, rows}, boxes {64, 128}
inline bool cross_q_map(CUtensorMap* map, const uint16_t* base, int d, const CrossArgs& A,
                        int64_t ld) {
  const uint64_t row = static_cast<uint64_t>(ld) * 2, rows = static_cast<uint64_t>(A.q_rows);
  if (A.G == 1) {
    const uint64_t dims[3] = {static_cast<uint64_t>(A.H) * d, rows, 1};
    const uint64_t strides[2] = {row, row * rows};
    const uint32_t box[3] = {64, 128, 1};
    return make_tmap_bf16(map, base, 3, dims, strides, box);
  }
  const uint64_t dims[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(A.H), rows};
  const uint64_t strides[2] = {static_cast<uint64_t>(d) * 2, row};
  const uint32_t box[3] = {64, static_cast<uint32_t>(A.G), static_cast<uint32_t>(A.pq)};
  return make_tmap_bf16(map, base, 3, dims, strides, box);
}
inline bool cross_kv_map(CUtensorMap* map, const uint16_t* base, int d, const CrossArgs& A) {
  const uint64_t dims[2] = {static_cast<uint64_t>(A.KV) * d, static_cast<uint64_t>(A.kv_rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(A.ld_kv) * 2};
  const uint32_t box[2] = {64, 128};
  return make_tmap_bf16(map, base, 2, dims, strides, box);
}

// Columns [64 c, 64 c + 64) of the heads of group hk, of pq queries from row q0
// on: the rows of a block, 128 bytes each.
__device__ __forceinline__ void cross_load_q(void* dst, const CUtensorMap* map, uint64_t* bar,
                                             const CrossArgs& A, int d, int c, int hk, int q0) {
  if (A.G == 1)
    tma_load_3d(dst, map, bar, hk * d + c * 64, q0, 0);
  else
    tma_load_3d(dst, map, bar, c * 64, hk * A.G, q0);
}

// Rows [valid, end) of a [128][D] tile (64-wide chunks 16 KB apart) become
// zeros, by a converged warp, before it issues products that contract over
// them: a weight of 0 there does not help against a NaN.
template <int D>
__device__ __forceinline__ void cross_clear_tail(uint8_t* tile, int valid, int lane,
                                                 int end = 128) {
#pragma unroll 1
  for (int at = valid * 128 + lane * 16; at < end * 128; at += 512) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      *reinterpret_cast<uint4*>(tile + c * 16384 + at) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();  // visible to the products
  __syncwarp();
}

// Sequences by the length of their items (their real keys, or queries), the
// longest first, ties in their order: order[i] is the i-th.  By a converged warp,
// into shared memory; up to kCrossSorted of them, where they can differ
// (cross_sorts).
constexpr int kCrossSorted = 64;
inline bool cross_sorts(const CrossArgs& A) {
  return A.n > 1 && A.n <= kCrossSorted && (A.q_off || A.q_len || A.kv_off || A.kv_len);
}
__device__ __forceinline__ void cross_order(const CrossArgs& A, bool by_keys, int8_t* order,
                                            int lane) {
  constexpr int kPer = kCrossSorted / 32;
  int len[kPer], rank[kPer] = {};
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int n = i * 32 + lane;
    len[i] = -1;
    if (n < A.n) {
      // (a sequence without the others has nothing to do)
      const int q = cross_queries(A, n).real, k = cross_keys(A, n).real;
      len[i] = q == 0 || k == 0 ? 0 : by_keys ? k : q;
    }
  }
  for (int m = 0; m < A.n; ++m) {
    int of_m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (m / 32 == i) of_m = __shfl_sync(0xffffffffu, len[i], m % 32);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      rank[i] += (of_m > len[i] || (of_m == len[i] && m < i * 32 + lane)) ? 1 : 0;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i * 32 + lane < A.n) order[rank[i]] = static_cast<int8_t>(i * 32 + lane);
}

// Rows of a [128][D] tile (64-wide chunks 16 KB apart) that no box covers: the
// last 128 - G pq.  Zeroed once, by `threads` threads of which this is `t`.
template <int D>
__device__ __forceinline__ void cross_clear_rows(uint8_t* tile, const CrossArgs& A, int t,
                                                 int threads) {
  const int first = A.G * A.pq;
  for (int i = t; i < (128 - first) * 8 * (D / 64); i += threads) {
    const int c = i / ((128 - first) * 8), at = i % ((128 - first) * 8);
    *reinterpret_cast<uint4*>(tile + c * 16384 + first * 128 + at * 16) = make_uint4(0, 0, 0, 0);
  }
}

inline CrossArgs cross_args(const mc_cross_attention& c, int* status) {
  CrossArgs A = {};
  A.q_off = c.q_offsets;
  A.q_len = c.q_lens;
  A.kv_off = c.kv_offsets;
  A.kv_len = c.kv_lens;
  A.n = c.sequences;
  A.H = c.heads;
  A.KV = c.kv_heads;
  A.G = c.heads / c.kv_heads;
  A.pq = 128 / A.G;
  A.q_rows = c.q_rows;
  A.kv_rows = c.kv_rows;
  auto most = [&](const int32_t* off, int rows, int bound) {
    if (!off) return rows / c.sequences;
    return bound > 0 && bound < rows ? bound : rows;
  };
  A.max_q = most(c.q_offsets, c.q_rows, c.max_q);
  A.max_kv = most(c.kv_offsets, c.kv_rows, c.max_kv);
  A.nqb = (A.max_q + A.pq - 1) / A.pq;
  A.nkb = (A.max_kv + 127) / 128;
  A.ld_q = c.ld_q;
  A.ld_kv = c.ld_kv;
  A.ld_o = c.ld_o;
  A.scale = c.scale > 0.f ? c.scale : c.head_dim == 64 ? 0.125f : 0.08838834764831845f;
  A.div_g = A.G == 1 ? 0u : static_cast<uint32_t>((0x100000000ull + A.G - 1) / A.G);
  A.status = status;
  return A;
}

// The forward of two CTAs per SM, attention_cross_pair.cu.
int launch_attention_cross_pair(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                uint16_t* o, float* lse, const CrossArgs& c, int d,
                                cudaStream_t st);

}  // namespace mc
