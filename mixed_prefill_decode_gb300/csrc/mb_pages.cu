// Page operations on the KV pools of a stack: the accepted path of a
// drafted tree moved to the positions behind the prefix, and whole pages
// copied.  Pure data movement: each byte is read once and written once, so
// HBM bounds the large calls and the launch the small ones.  Measured: 256
// pages of 64 KB in 40 pools 193 us, 6.9 TB/s read and written (a plain copy:
// 6.8); one page in 32 pools 1.9 us in a graph; the accepted paths of 64 requests
// in 40 pools, 84 MB, 16.7 us, 5.0 TB/s (rows of 256 bytes, 4 KB apart).

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mb_launch.cuh"
#include "mb_ptx.cuh"
#include "mb_spec.h"

namespace mb {
namespace {

using namespace dev;

struct PoolList {
  uint4 *base[kMaxPoolsPerLaunch];
};

// ------------------------------------------------------------- compaction
// One CTA per (request, pool); a thread owns one 16-byte column (a piece of
// one head's K or V row) of every token that moves.  path is strictly
// increasing, so the token bound for index k comes from path[k] >= k: a
// thread that takes its moves in ascending order reads every source before
// it overwrites it, and no other thread touches its column.  Eight loads of a
// thread go out before the first store: with one at a time a path of 8 nodes
// would take eight round trips to HBM in a row.
constexpr int kCompactThreads = 256;
constexpr int kCompactBatch = 8;   // moves whose loads are in flight together

struct CompactParams {
  const int32_t *qo_indptr, *kv_len, *bt_indptr, *bt, *count, *path;
  int32_t *new_kv_len;
  int n_reqs, max_path, Hkv, vec_per_row, num_pages;
  int first_pool;
  int *err;
};

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const __grid_constant__ PoolList pools,
                                                                  const CompactParams p) {
  __shared__ int64_t s_from[kMaxTreeNodes], s_to[kMaxTreeNodes];   // vectors from the pool's start to (page, slot) of head 0's K
  __shared__ int s_n;
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  const int t0 = p.qo_indptr[r], t1 = p.qo_indptr[r + 1], kv = p.kv_len[r];
  const int b0 = p.bt_indptr[r], b1 = p.bt_indptr[r + 1];
  const int cnt = p.count[r];
  // (compared before they are subtracted: the words may be anything)
  const bool order = t0 >= 0 && t1 >= t0 && b0 >= 0 && b1 >= b0;
  const int n = order ? t1 - t0 : 0, pages = order ? b1 - b0 : 0, c = kv < n ? -1 : kv - n;
  if (threadIdx.x == 0) s_n = 0;
  bool bad = !order || n > kMaxTreeNodes || c < 0 || (static_cast<int64_t>(kv) + kPage - 1) / kPage > pages || cnt < 0 ||
             cnt > n || cnt > p.max_path;
  __syncthreads();
  if (!bad) {
    const int64_t page_vecs = 2ll * p.Hkv * kPage * p.vec_per_row;
    for (int k = threadIdx.x; k < cnt; k += kCompactThreads) {
      const int f = p.path[static_cast<int64_t>(r) * p.max_path + k];
      const int prev = k > 0 ? p.path[static_cast<int64_t>(r) * p.max_path + k - 1] : -1;
      bool ok = f > prev && f < n && f >= k;
      int64_t from = 0, to = 0;
      if (ok) {
        const int pf = p.bt[b0 + (c + f) / kPage], pt = p.bt[b0 + (c + k) / kPage];
        ok = pf >= 0 && pf < p.num_pages && pt >= 0 && pt < p.num_pages;
        from = pf * page_vecs + static_cast<int64_t>((c + f) % kPage) * p.vec_per_row;
        to = pt * page_vecs + static_cast<int64_t>((c + k) % kPage) * p.vec_per_row;
      }
      s_from[k] = from;
      s_to[k] = to;
      if (!ok) atomicOr(&s_n, 1);
    }
    __syncthreads();
    bad = s_n != 0;
  }
  if (bad) {   // nothing of the request moves
    if (threadIdx.x == 0) atomicExch(p.err, kErrBounds);
    return;
  }
  if (threadIdx.x == 0 && blockIdx.y == 0 && p.first_pool == 0) p.new_kv_len[r] = c + cnt;
  uint4 *pool = pools.base[blockIdx.y];
  const int cols = 2 * p.Hkv * p.vec_per_row;
  for (int v = threadIdx.x; v < cols; v += kCompactThreads) {
    // column v: row (K or V, head) v / vec_per_row of the page, vector v % vec_per_row of it
    const int64_t off = static_cast<int64_t>(v / p.vec_per_row) * kPage * p.vec_per_row + v % p.vec_per_row;
    for (int k0 = 0; k0 < cnt; k0 += kCompactBatch) {
      uint4 x[kCompactBatch];
#pragma unroll
      for (int b = 0; b < kCompactBatch; ++b)
        if (k0 + b < cnt && s_from[k0 + b] != s_to[k0 + b]) x[b] = pool[s_from[k0 + b] + off];
#pragma unroll
      for (int b = 0; b < kCompactBatch; ++b)
        if (k0 + b < cnt && s_from[k0 + b] != s_to[k0 + b]) pool[s_to[k0 + b] + off] = x[b];
    }
  }
}

// ------------------------------------------------------------- page copies
// One CTA per (slice of a page, pair, pool); the pairs travel as kernel
// arguments, so nothing is copied to the device first and a captured call
// keeps its own.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;   // 16-byte loads in flight per thread: 32 KB a CTA

template <int N>
struct PairList {
  int32_t src[N], dst[N];
};

template <int N>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ PoolList pools,
                                                                  const __grid_constant__ PairList<N> pairs,
                                                                  int64_t page_vecs) {
  pdl_wait();
  pdl_trigger();
  uint4 *pool = pools.base[blockIdx.z];
  const uint4 *src = pool + pairs.src[blockIdx.y] * page_vecs;
  uint4 *dst = pool + pairs.dst[blockIdx.y] * page_vecs;
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kCopyThreads * kCopyUnroll + threadIdx.x;
  uint4 x[kCopyUnroll];
#pragma unroll
  for (int k = 0; k < kCopyUnroll; ++k)
    if (v0 + k * kCopyThreads < page_vecs) x[k] = src[v0 + k * kCopyThreads];
#pragma unroll
  for (int k = 0; k < kCopyUnroll; ++k)
    if (v0 + k * kCopyThreads < page_vecs) dst[v0 + k * kCopyThreads] = x[k];
}

template <int N>
cudaError_t launch_copy(const PoolList &pl, int n_pools, const int32_t *src, const int32_t *dst, int n_pairs,
                        int64_t page_vecs, cudaStream_t st) {
  PairList<N> pairs;
  std::copy(src, src + n_pairs, pairs.src);
  std::copy(dst, dst + n_pairs, pairs.dst);
  const int per = kCopyThreads * kCopyUnroll;
  return launch_pdl(copy_pages_kernel<N>, dim3(static_cast<unsigned>((page_vecs + per - 1) / per), n_pairs, n_pools),
                    dim3(kCopyThreads), 0, st, 1, pl, pairs, page_vecs);
}

PoolList pool_list(void *const *pools, int first, int n) {
  PoolList pl;
  for (int i = 0; i < n; ++i) pl.base[i] = static_cast<uint4 *>(pools[first + i]);
  return pl;
}

}  // namespace

cudaError_t kv_compact_run(const CompactArgs &a, cudaStream_t st) {
  for (int first = 0; first < a.n_pools; first += kMaxPoolsPerLaunch) {
    const int np = std::min(kMaxPoolsPerLaunch, a.n_pools - first);
    const CompactParams p = {a.qo_indptr, a.kv_len, a.bt_indptr, a.bt,       a.count, a.path, a.new_kv_len,
                             a.n_reqs,    a.max_path, a.Hkv,     a.hd / 8, a.num_pages, first,  a.err};
    const cudaError_t e = launch_pdl(compact_kernel, dim3(a.n_reqs, np), dim3(kCompactThreads), 0, st, 1,
                                     pool_list(a.pools, first, np), p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t kv_copy_pages_run(void *const *pools, int n_pools, int Hkv, int hd, const int32_t *src, const int32_t *dst,
                              int n_pairs, cudaStream_t st) {
  const int64_t page_vecs = 2ll * Hkv * kPage * hd / 8;
  constexpr int kSmall = 128, kLarge = 2048;   // pairs per launch: they travel as kernel arguments (1 KB or 16 KB)
  for (int pf = 0; pf < n_pools; pf += kMaxPoolsPerLaunch) {
    const int np = std::min(kMaxPoolsPerLaunch, n_pools - pf);
    const PoolList pl = pool_list(pools, pf, np);
    for (int first = 0; first < n_pairs; first += kLarge) {
      const int m = std::min(kLarge, n_pairs - first);
      const cudaError_t e = m <= kSmall ? launch_copy<kSmall>(pl, np, src + first, dst + first, m, page_vecs, st)
                                        : launch_copy<kLarge>(pl, np, src + first, dst + first, m, page_vecs, st);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace mb
