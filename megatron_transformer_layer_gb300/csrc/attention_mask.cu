// Interval masks of the attention stage: every query sees the keys
// [key_lo, key_hi) of its own sequence.  Documents packed into a sequence,
// prefixes that see themselves whole, sliding windows, padding (an empty
// interval) and their combinations are all such intervals, so the attention
// kernels test two bounds per row whatever the mask is.
//
// A warp forms a 128-row block's intervals and their union, then the query
// blocks that see a key block, then the two blocks' places in tables sorted by
// work, the longest first, so that the attention grids start their longest
// items first.  Bound by the latency of one launch and of a few dependent
// loads, not by its bytes (12 per token).  Up to 4096 blocks one cluster does
// all of it, the unions and ranges exchanged through its shared memory: 8 x
// 4096 tokens take 7.0 us, where two launches (rows, then a sort in one CTA)
// took 9.2, and the host pays for one launch.
#include <cuda_runtime.h>

#include "mc_layer_internal.h"
#include "ptx.cuh"

namespace mc {
namespace {

constexpr int kMaskRows = 128;
constexpr int kMaskWarps = 32;   // most warps per CTA of the table kernel
constexpr int kMaskCluster = 8;  // most CTAs of its cluster
// Tables of up to this many blocks are sorted (by comparing all pairs, in the
// shared memory of one cluster).  Longer ones keep the order of the sequence,
// query blocks backwards: their grids run for many waves, where the order of a
// few long items no longer shows, and the comparisons grow with the square.
constexpr int kMaskMaxSorted = 4096;

struct DocArgs {
  const int32_t* offsets;  // [n_docs + 1]
  const int32_t* prefix;   // [n_docs] or NULL
  int n_docs, causal, window;
};

// The numbers c0 and c1 of offsets[0, n) that are <= t0 and <= t1, found by a
// warp: each round splits the remaining ranges into 32 parts and counts the
// part starts that are <= t.  Offsets ascend.
__device__ __forceinline__ void count_le(const int32_t* offsets, int n, int64_t t0, int64_t t1,
                                         int* c0, int* c1) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  int lo[2] = {0, 0}, hi[2] = {n, n};  // offsets[0, lo) <= t, offsets[hi, n) > t
  const int64_t t[2] = {t0, t1};
  while (hi[0] > lo[0] || hi[1] > lo[1]) {
    int step[2];
    int64_t v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      step[i] = (hi[i] - lo[i] + 31) / 32;
      const int64_t at = lo[i] + static_cast<int64_t>(lane) * step[i];
      v[i] = at < hi[i] ? offsets[at] : int64_t(1) << 32;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int le = __popc(__ballot_sync(0xffffffffu, v[i] <= t[i]));
      if (le == 0) {
        hi[i] = lo[i];
      } else {
        const int64_t end = lo[i] + static_cast<int64_t>(le) * step[i];
        lo[i] += (le - 1) * step[i] + 1;  // offsets[lo - 1] <= t
        hi[i] = static_cast<int>(min(static_cast<int64_t>(hi[i]), end));
      }
    }
  }
  *c0 = lo[0];
  *c1 = lo[1];
}

// A warp: the intervals of query block e's rows (formed from the documents, or
// given), and in every lane their union, (0, 0) if all are empty.
template <bool DOCS>
__device__ __forceinline__ int2 block_rows(const DocArgs& A, int b, int s, int nb, int e,
                                           int32_t* key_lo, int32_t* key_hi, int* status) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int bi = e / nb, r0 = (e - bi * nb) * kMaskRows;
  const int64_t base = static_cast<int64_t>(bi) * s;
  int k0 = 0, k1 = 0;
  if constexpr (DOCS) {
    // the documents of the block's first and last token bound every row's
    count_le(A.offsets, A.n_docs + 1, base + r0, base + min(r0 + kMaskRows, s) - 1, &k0, &k1);
    --k0;
    --k1;
  }
  int ulo = 0x7fffffff, uhi = 0;
#pragma unroll
  for (int r = 0; r < kMaskRows / 32; ++r) {
    const int i = r0 + r * 32 + lane;
    const int64_t t = base + i;
    int lo = 0, hi = 0;
    if constexpr (DOCS) {
      if (i < s) {
        int k = k0, end = k1;
        while (k < end) {  // the last document that starts at or before t
          const int mid = k + (end - k + 1) / 2;
          if (A.offsets[mid] <= t)
            k = mid;
          else
            end = mid - 1;
        }
        const int pre = A.prefix && k >= 0 && k < A.n_docs ? A.prefix[k] : 0;
        if (k >= 0 && k < A.n_docs && pre >= 0) {
          // relative to the sequence; a document is cut at its ends
          const int64_t start = A.offsets[k] - base, stop = A.offsets[k + 1] - base;
          lo = static_cast<int>(max(start, int64_t(0)));
          const int last = static_cast<int>(max(min(stop, static_cast<int64_t>(s)), int64_t(0)));
          hi = last;
          if (A.causal)
            hi = max(i + 1, static_cast<int>(min(start + pre, static_cast<int64_t>(last))));
          if (A.window > 0) {
            lo = max(lo, i + 1 - A.window);
            hi = static_cast<int>(
                min(static_cast<int64_t>(hi), static_cast<int64_t>(i) + A.window));
          }
        }
        if (MC_DCHECK(t < static_cast<int64_t>(b) * s, status, kSiteMask)) {
          key_lo[t] = lo;
          key_hi[t] = hi;
        }
      }
    } else if (i < s) {
      lo = max(key_lo[t], 0);
      hi = min(key_hi[t], s);
    }
    if (lo < hi) {
      ulo = min(ulo, lo);
      uhi = max(uhi, hi);
    }
  }
  ulo = __reduce_min_sync(0xffffffffu, ulo);
  uhi = __reduce_max_sync(0xffffffffu, uhi);
  return make_int2(uhi > 0 ? ulo : 0, uhi);
}

// A warp: in every lane the query blocks [first, end) of a sequence that see
// key block k: those whose union meets it.  u(q) gives block q's union.
template <class F>
__device__ __forceinline__ int2 seen_by(int k, int nb, F&& u) {
  const int k0 = k * kMaskRows;
  int first = 0x7fffffff, end = 0;
  for (int q = static_cast<int>(threadIdx.x) & 31; q < nb; q += 32) {
    const int2 r = u(q);
    if (r.x < k0 + kMaskRows && r.y > k0 && r.y > r.x) {
      first = min(first, q);
      end = q + 1;
    }
  }
  first = __reduce_min_sync(0xffffffffu, first);
  end = __reduce_max_sync(0xffffffffu, end);
  return make_int2(end > 0 ? first : 0, end);
}

__device__ __forceinline__ void group_sync(int n_cta) {
  if (n_cta > 1)
    cluster_sync();
  else
    __syncthreads();
}

// v into *p of every CTA of the cluster, by one warp.
__device__ __forceinline__ void share(int2* p, int2 v, int n_cta) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  if (n_cta == 1) {
    if (lane == 0) *p = v;
  } else if (lane < n_cta) {
    st_cluster_v2(mapa_shared(p, static_cast<uint32_t>(lane)), v);
  }
}

// One cluster of the whole grid.  A warp takes every (warps of the cluster)th
// block of each phase: its rows' union, its key block's query range, its ranks
// in both tables.  The tables are ordered by the length of the ranges, longest
// first, ties by position.
template <bool DOCS>
__global__ void __launch_bounds__(kMaskWarps * 32, 1)
    mask_tables_kernel(DocArgs A, int b, int s, int nb, int32_t* key_lo, int32_t* key_hi,
                       int4* q_table, int4* k_table, int* status) {
  extern __shared__ int2 smem_mask[];
  const int n = b * nb;
  const int n_cta = static_cast<int>(gridDim.x), n_warps = static_cast<int>(blockDim.x) >> 5;
  const int w0 = static_cast<int>(blockIdx.x) * n_warps + (static_cast<int>(threadIdx.x) >> 5);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  int2* qr = smem_mask;      // [n] the query blocks' unions
  int2* kr = smem_mask + n;  // [n] the key blocks' query ranges
  group_sync(n_cta);         // every CTA runs before its shared memory is written
  pdl_wait();                // the previous kernel on the stream has completed
  pdl_launch();
  for (int e = w0; e < n; e += n_cta * n_warps)
    share(qr + e, block_rows<DOCS>(A, b, s, nb, e, key_lo, key_hi, status), n_cta);
  group_sync(n_cta);
  for (int e = w0; e < n; e += n_cta * n_warps) {
    const int b0 = e / nb * nb;
    share(kr + e, seen_by(e - b0, nb, [&](int q) { return qr[b0 + q]; }), n_cta);
  }
  group_sync(n_cta);
  for (int e = w0; e < n; e += n_cta * n_warps) {
    const int2 q = qr[e], k = kr[e];
    const int wq = q.y - q.x, wk = k.y - k.x;
    int rq = 0, rk = 0;
    for (int j = lane; j < n; j += 32) {
      const int vq = qr[j].y - qr[j].x, vk = kr[j].y - kr[j].x;
      rq += vq > wq || (vq == wq && j < e);
      rk += vk > wk || (vk == wk && j < e);
    }
    rq = __reduce_add_sync(0xffffffffu, rq);
    rk = __reduce_add_sync(0xffffffffu, rk);
    const int bi = e / nb, blk = e - bi * nb;
    if (lane == 0 && MC_DCHECK(rq < n && rk < n, status, kSiteMask)) {
      q_table[rq] = make_int4(bi, blk, q.x, q.y);
      k_table[rk] = make_int4(bi, blk, k.x, k.y);
    }
  }
}

// Unsorted tables: the query entries, the sequence backwards.
template <bool DOCS>
__global__ void __launch_bounds__(128)
    mask_rows_kernel(DocArgs A, int b, int s, int nb, int32_t* key_lo, int32_t* key_hi,
                     int4* q_table, int* status) {
  pdl_wait();  // the previous kernel on the stream has completed
  pdl_launch();
  const int n = b * nb;
  const int e = static_cast<int>(blockIdx.x) * 4 + (static_cast<int>(threadIdx.x) >> 5);
  if (e >= n) return;
  const int2 u = block_rows<DOCS>(A, b, s, nb, e, key_lo, key_hi, status);
  const int bi = e / nb;
  if ((threadIdx.x & 31) == 0) q_table[n - 1 - e] = make_int4(bi, e - bi * nb, u.x, u.y);
}

// Unsorted tables: the key entries, in sequence order.
__global__ void __launch_bounds__(128)
    mask_keys_kernel(const int4* __restrict__ q_table, int4* __restrict__ k_table, int n, int nb) {
  pdl_wait();  // mask_rows_kernel has completed
  pdl_launch();
  const int e = static_cast<int>(blockIdx.x) * 4 + (static_cast<int>(threadIdx.x) >> 5);
  if (e >= n) return;
  const int bi = e / nb, blk = e - bi * nb;
  const int2 r = seen_by(blk, nb, [&](int q) {
    const int4 v = q_table[n - 1 - (bi * nb + q)];
    return make_int2(v.z, v.w);
  });
  if ((threadIdx.x & 31) == 0) k_table[e] = make_int4(bi, blk, r.x, r.y);
}

int check_mask_shape(int b, int s) {
  if (b < 1 || s < 1) return MC_ERR_SHAPE;
  if (b > 65535 || static_cast<int64_t>(b) * s > (1 << 24)) return MC_ERR_UNSUPPORTED;
  return MC_OK;
}

template <bool DOCS>
int launch_mask(const DocArgs& A, int b, int s, int32_t* key_lo, int32_t* key_hi, int32_t* tables,
                int* status, cudaStream_t st) {
  const int nb = (s + kMaskRows - 1) / kMaskRows;
  const int n = b * nb;  // <= 2^24
  int4* q_table = reinterpret_cast<int4*>(tables);
  int4* k_table = q_table + n;
  if (n <= kMaskMaxSorted) {
    const size_t smem = 2 * sizeof(int2) * n;
    static PerDeviceInit init;
    const cudaError_t attr = once_per_device(init, [](long long*) {
      return cudaFuncSetAttribute(mask_tables_kernel<DOCS>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(2 * sizeof(int2)) * kMaskMaxSorted);
    });
    if (attr != cudaSuccess) return MC_ERR_CUDA;
    const int warps = n < kMaskWarps ? n : kMaskWarps;
    const int full = (n + kMaskWarps - 1) / kMaskWarps;
    const int ctas = full < kMaskCluster ? full : kMaskCluster;
    launch_kernel(mask_tables_kernel<DOCS>, dim3(static_cast<unsigned>(ctas)),
                  dim3(static_cast<unsigned>(warps) * 32), smem, st, static_cast<unsigned>(ctas), A,
                  b, s, nb, key_lo, key_hi, q_table, k_table, status);
  } else {
    const dim3 grid(static_cast<unsigned>((n + 3) / 4));
    launch_kernel(mask_rows_kernel<DOCS>, grid, dim3(128), 0, st, 1, A, b, s, nb, key_lo, key_hi,
                  q_table, status);
    if (cudaGetLastError() != cudaSuccess) return MC_ERR_CUDA;
    launch_kernel(mask_keys_kernel, grid, dim3(128), 0, st, 1, static_cast<const int4*>(q_table),
                  k_table, n, nb);
  }
  return cudaGetLastError() == cudaSuccess ? MC_OK : MC_ERR_CUDA;
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace
}  // namespace mc

using namespace mc;

extern "C" {

size_t mc_attention_mask_table_ints(int32_t micro_batch, int32_t seq_len) {
  if (check_mask_shape(micro_batch, seq_len) != MC_OK) return 0;
  return static_cast<size_t>(8) * micro_batch * ((seq_len + kMaskRows - 1) / kMaskRows);
}

int mc_attention_mask_documents(const int32_t* offsets, int32_t n_docs, const int32_t* prefix,
                                int32_t causal, int32_t window, int32_t micro_batch,
                                int32_t seq_len, int32_t* key_lo, int32_t* key_hi,
                                int32_t* tables, int* status, void* stream) {
  const int rc = check_mask_shape(micro_batch, seq_len);
  if (rc != MC_OK) return rc;
  if (n_docs < 0 || n_docs > (1 << 24) || window < 0) return MC_ERR_ARGUMENT;
  if (!offsets || !key_lo || !key_hi || !tables) return MC_ERR_NULLPTR;
  if (!aligned(offsets, 4) || !aligned(prefix, 4) || !aligned(key_lo, 4) || !aligned(key_hi, 4) ||
      !aligned(tables, 16))
    return MC_ERR_ALIGN;
  const DocArgs A = {offsets, prefix, n_docs, causal ? 1 : 0, window};
  return launch_mask<true>(A, micro_batch, seq_len, key_lo, key_hi, tables, status,
                           static_cast<cudaStream_t>(stream));
}

int mc_attention_mask_intervals(int32_t micro_batch, int32_t seq_len, const int32_t* key_lo,
                                const int32_t* key_hi, int32_t* tables, int* status,
                                void* stream) {
  const int rc = check_mask_shape(micro_batch, seq_len);
  if (rc != MC_OK) return rc;
  if (!key_lo || !key_hi || !tables) return MC_ERR_NULLPTR;
  if (!aligned(key_lo, 4) || !aligned(key_hi, 4) || !aligned(tables, 16)) return MC_ERR_ALIGN;
  // read only: mask_rows_kernel<false> writes neither
  return launch_mask<false>(DocArgs{}, micro_batch, seq_len, const_cast<int32_t*>(key_lo),
                            const_cast<int32_t*>(key_hi), tables, status,
                            static_cast<cudaStream_t>(stream));
}

}  // extern "C"
