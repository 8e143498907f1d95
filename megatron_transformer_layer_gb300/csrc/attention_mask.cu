// Interval masks of the attention stage: every query sees the keys
// [key_lo, key_hi) of its own sequence.  Documents packed into a sequence,
// prefixes that see themselves whole, sliding windows, padding (an empty
// interval) and their combinations are all such intervals, so the attention
// kernels test two bounds per row whatever the mask is.
//
// One kernel forms a 128-row block's intervals and their union, a second the
// query blocks that see each key block, and sorts both tables by work, the
// longest first, so that the attention grids start their longest CTAs first.
// Both are bound by the latency of their launches and of a few dependent
// loads, not by their bytes (12 per token).
#include <cuda_runtime.h>

#include "mc_layer_internal.h"
#include "ptx.cuh"

namespace mc {
namespace {

constexpr int kMaskRows = 128;
constexpr int kMaskSortThreads = 1024;
// Tables of up to this many blocks are sorted (by comparing all pairs, in one
// block's shared memory).  Longer ones keep the order of the sequence, query
// blocks backwards: their grids run for many waves, where the order of a few
// long CTAs no longer shows, and the comparisons grow with the square.
constexpr int kMaskMaxSorted = 4096;

struct DocArgs {
  const int32_t* offsets;  // [n_docs + 1]
  const int32_t* prefix;   // [n_docs] or NULL
  int n_docs, causal, window;
};

// The number of offsets[0, n) that are <= t, found by the whole block: each
// round splits the remaining range into 128 parts and counts the part starts
// that are <= t.  Offsets ascend.
__device__ __forceinline__ int count_le(const int32_t* offsets, int n, int64_t t) {
  int lo = 0, hi = n;  // offsets[0, lo) <= t, offsets[hi, n) > t
  while (hi > lo) {
    const int step = (hi - lo + kMaskRows - 1) / kMaskRows;
    const int64_t at = lo + static_cast<int64_t>(threadIdx.x) * step;
    const int le = __syncthreads_count(at < hi && offsets[at] <= t);
    if (le == 0) return lo;
    const int next = lo + (le - 1) * step + 1;  // offsets[next - 1] <= t
    hi = min(hi, lo + le * step);
    lo = next;
  }
  return lo;
}

// Block (batch, q): its rows' intervals (formed from the documents, or given)
// and their union into entries[q-order position].
template <bool DOCS>
__global__ void __launch_bounds__(kMaskRows)
    mask_rows_kernel(DocArgs A, int b, int s, int nb, int32_t* key_lo, int32_t* key_hi,
                     int4* entries, int reversed, int* status) {
  pdl_wait();  // the previous kernel on the stream has completed
  pdl_launch();
  const int e = static_cast<int>(blockIdx.x);
  const int bi = e / nb, q = e - bi * nb;
  const int i = q * kMaskRows + static_cast<int>(threadIdx.x);
  const int64_t base = static_cast<int64_t>(bi) * s;
  const int64_t t = base + i;
  int lo = 0, hi = 0;
  if constexpr (DOCS) {
    // the documents of the block's first and last token bound every row's
    const int64_t t_first = base + q * kMaskRows;
    const int64_t t_last = base + min(q * kMaskRows + kMaskRows, s) - 1;
    int k0 = count_le(A.offsets, A.n_docs + 1, t_first) - 1;
    int k1 = count_le(A.offsets, A.n_docs + 1, t_last) - 1;
    if (i < s) {
      while (k0 < k1) {  // the last document that starts at or before t
        const int mid = k0 + (k1 - k0 + 1) / 2;
        if (A.offsets[mid] <= t)
          k0 = mid;
        else
          k1 = mid - 1;
      }
      const int pre = A.prefix && k0 >= 0 && k0 < A.n_docs ? A.prefix[k0] : 0;
      if (k0 >= 0 && k0 < A.n_docs && pre >= 0) {
        // relative to the sequence; a document is cut at its ends
        const int64_t start = A.offsets[k0] - base, stop = A.offsets[k0 + 1] - base;
        const int first = static_cast<int>(max(start, int64_t(0)));
        const int last = static_cast<int>(min(stop, static_cast<int64_t>(s)));
        lo = first;
        hi = last;
        if (A.causal)
          hi = max(i + 1, static_cast<int>(min(start + pre, static_cast<int64_t>(last))));
        if (A.window > 0) {
          lo = max(lo, i + 1 - A.window);
          hi = static_cast<int>(min(static_cast<int64_t>(hi), static_cast<int64_t>(i) + A.window));
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
  // the union of the non-empty intervals
  if (lo >= hi) {
    lo = 0x7fffffff;
    hi = 0;
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  __shared__ int2 part[kMaskRows / 32];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_int2(lo, hi);
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < kMaskRows / 32; ++w) {
      lo = min(lo, part[w].x);
      hi = max(hi, part[w].y);
    }
    const int n = b * nb;
    const int at = reversed ? n - 1 - e : e;
    if (MC_DCHECK(at >= 0 && at < n, status, kSiteMask))
      entries[at] = make_int4(bi, q, hi > 0 ? lo : 0, hi);
  }
}

// Query blocks [first, end) of a sequence that see key block k: those whose
// union meets it.  u(q) gives block q's union.
template <class F>
__device__ __forceinline__ int2 seen_by(int k, int nb, F&& u) {
  const int k0 = k * kMaskRows;
  int first = 0x7fffffff, end = 0;
  for (int q = 0; q < nb; ++q) {
    const int2 r = u(q);
    if (r.x < k0 + kMaskRows && r.y > k0 && r.y > r.x) {
      first = min(first, q);
      end = q + 1;
    }
  }
  return make_int2(end > 0 ? first : 0, end);
}

// One block: reads the unsorted query entries (left in the key table by
// mask_rows_kernel), forms the key entries and writes both tables sorted by
// the length of their range, longest first, ties by position.
__global__ void __launch_bounds__(kMaskSortThreads)
    mask_sort_kernel(int4* q_table, int4* k_table, int n, int nb, int* status) {
  pdl_wait();  // mask_rows_kernel has completed
  pdl_launch();
  extern __shared__ int2 smem_mask[];
  int2* qr = smem_mask;       // [n] the query blocks' unions
  int2* kr = smem_mask + n;   // [n] the key blocks' query ranges
  for (int e = threadIdx.x; e < n; e += kMaskSortThreads) {
    const int4 v = k_table[e];
    qr[e] = make_int2(v.z, v.w);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += kMaskSortThreads) {
    const int b0 = e / nb * nb;
    kr[e] = seen_by(e - b0, nb, [&](int q) { return qr[b0 + q]; });
  }
  __syncthreads();
  // 4 lanes share an entry's comparisons
  const int lane4 = static_cast<int>(threadIdx.x) & 3;
  for (int e0 = 0; e0 < n; e0 += kMaskSortThreads / 4) {
    const int e = e0 + (static_cast<int>(threadIdx.x) >> 2);
    int rq = 0, rk = 0;
    if (e < n) {
      const int wq = qr[e].y - qr[e].x, wk = kr[e].y - kr[e].x;
      for (int j = lane4; j < n; j += 4) {
        const int vq = qr[j].y - qr[j].x, vk = kr[j].y - kr[j].x;
        rq += vq > wq || (vq == wq && j < e);
        rk += vk > wk || (vk == wk && j < e);
      }
    }
    rq += __shfl_xor_sync(0xffffffffu, rq, 1);
    rk += __shfl_xor_sync(0xffffffffu, rk, 1);
    rq += __shfl_xor_sync(0xffffffffu, rq, 2);
    rk += __shfl_xor_sync(0xffffffffu, rk, 2);
    if (e < n && lane4 == 0 && MC_DCHECK(rq < n && rk < n, status, kSiteMask)) {
      const int bi = e / nb, blk = e - bi * nb;
      q_table[rq] = make_int4(bi, blk, qr[e].x, qr[e].y);
      k_table[rk] = make_int4(bi, blk, kr[e].x, kr[e].y);
    }
  }
}

// Unsorted tables: the key entries in sequence order from the query table,
// which holds the sequence backwards.
__global__ void __launch_bounds__(256)
    mask_keys_kernel(const int4* __restrict__ q_table, int4* __restrict__ k_table, int n, int nb,
                     int* status) {
  pdl_wait();  // mask_rows_kernel has completed
  pdl_launch();
  const int e = static_cast<int>(blockIdx.x) * 256 + static_cast<int>(threadIdx.x);
  if (e >= n) return;
  const int bi = e / nb, blk = e - bi * nb;
  const int2 r = seen_by(blk, nb, [&](int q) {
    const int4 v = q_table[n - 1 - (bi * nb + q)];
    return make_int2(v.z, v.w);
  });
  if (MC_DCHECK(e < n, status, kSiteMask)) k_table[e] = make_int4(bi, blk, r.x, r.y);
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
  const bool sorted = n <= kMaskMaxSorted;
  launch_kernel(mask_rows_kernel<DOCS>, dim3(static_cast<unsigned>(n)), dim3(kMaskRows), 0, st, 1,
                A, b, s, nb, key_lo, key_hi, sorted ? k_table : q_table, sorted ? 0 : 1, status);
  if (cudaGetLastError() != cudaSuccess) return MC_ERR_CUDA;
  if (sorted) {
    static PerDeviceInit init;
    const cudaError_t attr = once_per_device(init, [&](long long*) {
      return cudaFuncSetAttribute(mask_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(2 * sizeof(int2)) * kMaskMaxSorted);
    });
    if (attr != cudaSuccess) return MC_ERR_CUDA;
    launch_kernel(mask_sort_kernel, dim3(1), dim3(kMaskSortThreads), 2 * sizeof(int2) * n, st, 1,
                  q_table, k_table, n, nb, status);
  } else {
    launch_kernel(mask_keys_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st,
                  1, static_cast<const int4*>(q_table), k_table, n, nb, status);
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
