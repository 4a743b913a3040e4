// A batch's descriptor, its block tables and the places of its new tokens,
// built on the GPU from the requests' lengths; and a request's pages given
// back.
//
// Request r (row `slots[r]` of the tables) has c_r tokens cached, m_r new ones
// and o_r pages.  With need_r = max(0, ceil((c_r + m_r) / 16) - o_r) it is
// granted its tokens if need_r = 0 or the needs of the requests up to and
// including it fit the free pages; otherwise it has none this time.  That
// rule makes the pages taken a prefix of the ring, and the place of each
// request's first page a prefix sum of the needs, so everything is two scans
// over the requests and one write per page and token.
//
// What bounds it: 4 bytes a page read and written and 12 a token; at 64
// requests that is tens of KB, and the launch, the chain of loads (a
// request's slot, its row's page count, the page) and the scans are the time.
// Every CTA scans all requests itself, so one launch does it: a second one
// would cost what the whole call does.  What changes in place (page counts,
// the ring's head) is written by the last CTA to have read it.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mb_latent.h"
#include "mb_launch.cuh"
#include "mb_ptx.cuh"

namespace mb {
namespace {

using namespace dev;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kElemsPerCta = kThreads;   // pages and tokens that a CTA writes, one a thread while there are SMs
// Sums stop here (2^30): no sum that is used is as large, and sums that stop
// are still sums of non-negative numbers, whatever the order.
constexpr uint32_t kSat = 1u << 30;

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }

// Exclusive prefix sums of two numbers per thread, and their totals.
__device__ __forceinline__ uint2 block_scan2(uint2 v, uint2 *sums, uint2 *total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint2 inc = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, inc.x, off), y = __shfl_up_sync(0xffffffffu, inc.y, off);
    if (lane >= off) {
      inc.x = sat_add(inc.x, x);
      inc.y = sat_add(inc.y, y);
    }
  }
  if (lane == 31) sums[warp] = inc;   // (each scan of a kernel has its own)
  __syncthreads();
  uint2 pre = make_uint2(0, 0), all = make_uint2(0, 0);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const uint2 s = sums[w];
    if (w < warp) pre = make_uint2(sat_add(pre.x, s.x), sat_add(pre.y, s.y));
    all = make_uint2(sat_add(all.x, s.x), sat_add(all.y, s.y));
  }
  *total = all;
  // (what this thread's lanes before it hold)
  const uint32_t ex = __shfl_up_sync(0xffffffffu, inc.x, 1), ey = __shfl_up_sync(0xffffffffu, inc.y, 1);
  return lane == 0 ? pre : make_uint2(sat_add(pre.x, ex), sat_add(pre.y, ey));
}

// The last index of first[0 .. n] (ascending, first[0] = 0) that is <= e.
__device__ __forceinline__ int owner(const int32_t *first, int n, int e) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= e) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Marks the slots that occur in row[0 .. n) (each thread its own range); `twice`
// those that occur again.  The bits were cleared before the last barrier.
__device__ __forceinline__ void mark_slots(const int32_t *row, int lo, int hi, int max_slots, uint32_t *once, uint32_t *twice) {
  for (int r = lo; r < hi; ++r) {
    const int s = row[r];
    if (s < 0 || s >= max_slots) continue;
    const uint32_t bit = 1u << (s & 31);
    if (atomicOr(&once[s >> 5], bit) & bit) atomicOr(&twice[s >> 5], bit);
  }
  __syncthreads();
}

// Counts this CTA among those that have read what the last one is to change
// (thread 0's: how many came before).  Called behind a barrier; the answer is
// asked for at the kernel's end only, so that nothing waits for it.
__device__ __forceinline__ int arrive(int32_t *ctr) {
  if (gridDim.x == 1 || threadIdx.x != 0) return 0;
  __threadfence();
  return atomicAdd(ctr, 1);
}
__device__ __forceinline__ bool last_cta(int32_t *ctr, int before) {
  __shared__ int last;
  if (threadIdx.x == 0) {
    last = before == static_cast<int>(gridDim.x) - 1;
    if (last && gridDim.x > 1) *ctr = 0;
  }
  __syncthreads();
  return last != 0;
}

__global__ void __launch_bounds__(kThreads) tables_kernel(const __grid_constant__ TablesArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ uint2 sums[2][kWarps];
  __shared__ uint32_t mosts[kWarps];
  int32_t *qo = sm, *bti = qo + a.n + 1, *ring0 = bti + a.n + 1, *have = ring0 + a.n, *first = have + a.n,
          *row = first + a.n;
  uint32_t *once = reinterpret_cast<uint32_t *>(row + a.n), *twice = once + (a.max_slots + 31) / 32;
  pdl_wait();
  pdl_trigger();
  const int n = a.n, per = (n + kThreads - 1) / kThreads;
  const int lo = min(n, static_cast<int>(threadIdx.x) * per), hi = min(n, lo + per);
  const int head = a.state[0], count = a.state[1];
  const bool ring_ok = head >= 0 && head < a.num_pages && count >= 0 && count <= a.num_pages;
  bool bad = !ring_ok;
  // ---- the requests' words: all loads before anything waits for one
  for (int r = lo; r < hi; ++r) {
    const int s = a.slots[r];
    first[r] = a.cached[r];
    qo[r] = a.new_tokens[r];
    row[r] = s;
    have[r] = s >= 0 && s < a.max_slots ? a.owned[s] : -1;
  }
  for (int i = threadIdx.x; i < (a.max_slots + 31) / 32; i += kThreads) once[i] = twice[i] = 0;
  __syncthreads();
  mark_slots(row, lo, hi, a.max_slots, once, twice);
  // ---- what they ask for
  uint2 sum = make_uint2(0, 0), total;
  for (int r = lo; r < hi; ++r) {
    const int s = row[r], c = first[r], m = qo[r], o = have[r];
    bool ok = ring_ok && s >= 0 && s < a.max_slots && !((twice[s >> 5] >> (s & 31)) & 1u);
    // (compared before they are added: the words may be anything)
    ok = ok && c >= 0 && m >= 0 && o >= 0 && o <= a.max_pages && c <= o * static_cast<int64_t>(kPage) &&
         static_cast<int64_t>(c) + m <= a.max_pages * static_cast<int64_t>(kPage);
    bad |= !ok;
    row[r] = ok ? s : -1;
    first[r] = ok ? c : 0;
    have[r] = ok ? o : 0;
    qo[r] = ok ? m : 0;
    const int need = ok ? max(0, (c + m + kPage - 1) / kPage - o) : 0;
    sum.x = sat_add(sum.x, need);
  }
  uint2 at = block_scan2(sum, sums[0], &total);
  // ---- who is granted, and their tokens and pages
  sum = make_uint2(0, 0);
  uint32_t taken = 0;   // pages taken up to this thread's last granted request
  for (int r = lo; r < hi; ++r) {
    const int c = first[r], m = qo[r], o = have[r];
    const int need = max(0, (c + m + kPage - 1) / kPage - o);
    ring0[r] = static_cast<int32_t>(at.x);
    at.x = sat_add(at.x, need);
    const bool granted = need == 0 || at.x <= static_cast<uint32_t>(count);
    if (!granted) qo[r] = 0;
    if (granted && need) taken = at.x;
    sum.x = sat_add(sum.x, granted ? m : 0);
    sum.y = sat_add(sum.y, (c + (granted ? m : 0) + kPage - 1) / kPage);
  }
  at = block_scan2(sum, sums[1], &total);
  const bool fits = total.x <= static_cast<uint32_t>(a.T) && total.y <= static_cast<uint32_t>(a.bt_cap);
  bad |= !fits;
  if (bad && blockIdx.x == 0) atomicExch(a.err, kErrBounds);
  const bool none = !fits;   // the caller's arrays are too short: nothing is granted, nothing changes
  for (int r = lo; r < hi; ++r) {
    const int c = none ? 0 : first[r], m = none ? 0 : qo[r];
    const int pages = (c + m + kPage - 1) / kPage;
    qo[r] = none ? 0 : static_cast<int32_t>(at.x);
    bti[r] = none ? 0 : static_cast<int32_t>(at.y);
    at = make_uint2(sat_add(at.x, m), sat_add(at.y, pages));
    if (blockIdx.x == 0) {
      a.qo_indptr[r] = qo[r];
      a.bt_indptr[r] = bti[r];
      a.kv_len[r] = c + m;
    }
  }
  const int tokens = none ? 0 : static_cast<int>(total.x), pages = none ? 0 : static_cast<int>(total.y);
  if (threadIdx.x == 0) {
    qo[n] = tokens;
    bti[n] = pages;
    if (blockIdx.x == 0) {
      a.qo_indptr[n] = tokens;
      a.bt_indptr[n] = pages;
    }
  }
  __syncthreads();   // qo and bti are written, and the words that the last CTA changes read
  const int before = arrive(a.state + 2);
  // ---- pages and tokens
  // page j of request r: in its row, or the ring's (j - have) after its first
  auto page_of = [&](int r, int j) {
    if (j < have[r]) return a.tables[static_cast<int64_t>(row[r]) * a.max_pages + j];
    int64_t i = static_cast<int64_t>(head) + ring0[r] + (j - have[r]);
    if (i >= a.num_pages) i -= a.num_pages;
    return a.ring[i];
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads, at0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
#pragma unroll 4
  for (int64_t e = at0; e < pages; e += step) {
    const int r = owner(bti, n, static_cast<int>(e)), j = static_cast<int>(e) - bti[r];
    const int page = page_of(r, j);
    a.bt[e] = page;
    if (j >= have[r]) a.tables[static_cast<int64_t>(row[r]) * a.max_pages + j] = page;
  }
#pragma unroll 4
  for (int64_t t = at0; t < a.T; t += step) {
    int r = -1, pos = -1, slot = -1;
    if (t < tokens) {
      r = owner(qo, n, static_cast<int>(t));
      pos = first[r] + static_cast<int>(t) - qo[r];
      const int page = page_of(r, pos / kPage);
      if (page < 0 || page >= a.num_pages) atomicExch(a.err, kErrBounds);
      else slot = page * kPage + pos % kPage;
    }
    a.tok_req[t] = r;
    a.tok_pos[t] = pos;
    a.tok_slot[t] = slot;
  }
  // ---- the rows' page counts, and the ring's head: needs of granted requests
  if (!last_cta(a.state + 2, before) || none) return;
  uint32_t most = taken;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
  if ((threadIdx.x & 31) == 0) mosts[threadIdx.x >> 5] = most;
  for (int r = lo; r < hi; ++r) {
    const int listed = bti[r + 1] - bti[r];
    if (row[r] >= 0 && listed > have[r]) a.owned[row[r]] = listed;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 0; w < kWarps; ++w) most = max(most, mosts[w]);
    if (most > 0) {
      a.state[0] = static_cast<int32_t>((static_cast<int64_t>(head) + most) % a.num_pages);
      a.state[1] = count - static_cast<int32_t>(most);
    }
  }
}

// The pages of the requests to the ring's end, in the requests' order and
// each request's in its table's; nothing moves if they are more than the ring
// has room for.
__global__ void __launch_bounds__(kThreads) release_kernel(const __grid_constant__ TablesArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ uint2 sums[kWarps];
  int32_t *at0 = sm, *row = at0 + a.n + 1;
  uint32_t *once = reinterpret_cast<uint32_t *>(row + a.n), *twice = once + (a.max_slots + 31) / 32;
  pdl_wait();
  pdl_trigger();
  const int n = a.n, per = (n + kThreads - 1) / kThreads;
  const int lo = min(n, static_cast<int>(threadIdx.x) * per), hi = min(n, lo + per);
  const int head = a.state[0], count = a.state[1];
  const bool ring_ok = head >= 0 && head < a.num_pages && count >= 0 && count <= a.num_pages;
  bool bad = !ring_ok;
  for (int r = lo; r < hi; ++r) {
    const int s = a.slots[r];
    row[r] = s;
    at0[r] = s >= 0 && s < a.max_slots ? a.owned[s] : -1;
  }
  for (int i = threadIdx.x; i < (a.max_slots + 31) / 32; i += kThreads) once[i] = twice[i] = 0;
  __syncthreads();
  mark_slots(row, lo, hi, a.max_slots, once, twice);
  uint2 sum = make_uint2(0, 0), total;
  for (int r = lo; r < hi; ++r) {
    const int s = row[r], o = at0[r];
    bool ok = ring_ok && s >= 0 && s < a.max_slots && !((twice[s >> 5] >> (s & 31)) & 1u);
    ok = ok && o >= 0 && o <= a.max_pages;
    bad |= !ok;
    row[r] = ok ? s : -1;
    at0[r] = ok ? o : 0;
    sum.x = sat_add(sum.x, ok ? o : 0);
  }
  uint2 at = block_scan2(sum, sums, &total);
  const bool fits = ring_ok && total.x <= static_cast<uint32_t>(a.num_pages - count);
  bad |= !fits;
  if (bad && blockIdx.x == 0) atomicExch(a.err, kErrBounds);
  for (int r = lo; r < hi; ++r) {
    const int o = at0[r];
    at0[r] = static_cast<int32_t>(at.x);
    at.x = sat_add(at.x, o);
  }
  if (threadIdx.x == 0) at0[n] = static_cast<int32_t>(total.x);
  __syncthreads();   // at0 is written, and the words that the last CTA changes read
  const int before = arrive(a.state + 2);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
#pragma unroll 4
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; fits && e < total.x; e += step) {
    const int r = owner(at0, n, static_cast<int>(e));
    int64_t i = static_cast<int64_t>(head) + count + e;
    if (i >= a.num_pages) i -= a.num_pages;
    a.ring[i] = a.tables[static_cast<int64_t>(row[r]) * a.max_pages + (e - at0[r])];
  }
  if (!last_cta(a.state + 2, before) || !fits) return;
  for (int r = lo; r < hi; ++r)
    if (row[r] >= 0) a.owned[row[r]] = 0;
  if (threadIdx.x == 0) a.state[1] = count + static_cast<int32_t>(total.x);
}

int tables_grid(int64_t elems) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(device_sm_count(), (elems + kElemsPerCta - 1) / kElemsPerCta)));
}

}  // namespace

cudaError_t batch_tables_run(const TablesArgs &a, cudaStream_t st) {
  const size_t words = 6 * static_cast<size_t>(a.n) + 2 + 2 * ((static_cast<size_t>(a.max_slots) + 31) / 32);
  const int most = (6 * kTablesMaxReqs + 2 + 2 * (kTablesMaxSlots / 32)) * 4;
  cudaError_t e = ensure_max_smem(reinterpret_cast<const void *>(tables_kernel), most);
  if (e != cudaSuccess) return e;
  return launch_pdl(tables_kernel, dim3(tables_grid(static_cast<int64_t>(a.bt_cap) + a.T)), dim3(kThreads), words * 4, st, 1, a);
}

cudaError_t tables_release_run(const TablesArgs &a, cudaStream_t st) {
  const size_t words = 2 * static_cast<size_t>(a.n) + 1 + 2 * ((static_cast<size_t>(a.max_slots) + 31) / 32);
  const int most = (2 * kTablesMaxReqs + 1 + 2 * (kTablesMaxSlots / 32)) * 4;
  cudaError_t e = ensure_max_smem(reinterpret_cast<const void *>(release_kernel), most);
  if (e != cudaSuccess) return e;
  const int64_t pages = std::min<int64_t>(a.num_pages, static_cast<int64_t>(a.n) * a.max_pages);
  return launch_pdl(release_kernel, dim3(tables_grid(pages)), dim3(kThreads), words * 4, st, 1, a);
}

}  // namespace mb
