// A batch's descriptor, its block tables and the places of its new tokens,
// built on the GPU from the requests' lengths; and a request's pages given
// back.
//
// Request r (row `slots[r]` of the tables) has c_r tokens cached, m_r new ones
// and o_r pages.  With need_r = max(0, ceil((c_r + m_r) / 16) - o_r) it is
// granted its tokens if need_r = 0 or the needs of the requests up to and
// including it fit the free pages; otherwise it has none this time.  That
// rule makes the pages taken a prefix of the ring, and the place of each
// request's first page a prefix sum of the needs, so everything is a scan over
// the requests (two where the pages run out) and one write per page and token.
//
// What bounds it: 4 bytes a page read and written and 12 a token; at 64
// requests that is tens of KB, and the launch, the chain of loads (a
// request's slot, its row's page count, the page) and the scans are the time.
// Every CTA scans all requests itself, so one launch does it: a second one
// would cost what the whole call does.  What changes in place (page counts,
// the ring's head) is written by the last CTA to have read it.
//
// Measured, replayed in a graph: 64 decodes at 1,125 keys 5.0 us (10.7 with one load
// waiting for the other, a scan for each sum and an element a thread at a time), 256
// decodes and two chunks of 3,967 tokens (512 to 32,768 keys) 5.7.

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
constexpr int kBatch = 2;                // of a thread, loaded together
// Sums stop here (2^30): no sum that is used is as large, and sums that stop
// are still sums of non-negative numbers, whatever the order.
constexpr uint32_t kSat = 1u << 30;

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }

// Exclusive prefix sums of N numbers per thread, and their totals.  (Each scan of
// a kernel has shared sums of its own, so one barrier does.)
template <int N>
__device__ __forceinline__ void block_scan(uint32_t (&v)[N], uint32_t (*sums)[N], uint32_t (&total)[N]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t inc[N];
#pragma unroll
  for (int k = 0; k < N; ++k) inc[k] = v[k];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc[k], off);
      if (lane >= off) inc[k] = sat_add(inc[k], x);
    }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < N; ++k) sums[warp][k] = inc[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    uint32_t w = lane < kWarps ? sums[lane][k] : 0;
#pragma unroll
    for (int off = 1; off < kWarps; off <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w = sat_add(w, x);
    }
    total[k] = __shfl_sync(0xffffffffu, w, kWarps - 1);
    const uint32_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    const uint32_t mine = __shfl_up_sync(0xffffffffu, inc[k], 1);   // what this thread's lanes before it hold
    v[k] = sat_add(warp > 0 ? before : 0, lane > 0 ? mine : 0);
  }
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
  return gridDim.x == 1 || threadIdx.x != 0 ? 0 : atomicAdd(ctr, 1);
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
  __shared__ uint32_t sums[kWarps][3], sums2[kWarps][2], mosts[kWarps];
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
  // ---- what they ask for: pages, tokens, and the pages listed if all is granted
  uint32_t at[3] = {0, 0, 0}, total[3];
  for (int r = lo; r < hi; ++r) {
    const int s = row[r], c = first[r], m = qo[r], o = have[r];
    bool ok = ring_ok && s >= 0 && s < a.max_slots && !((twice[s >> 5] >> (s & 31)) & 1u);
    // (compared before they are added: the words may be anything)
    ok = ok && c >= 0 && m >= 0 && o >= 0 && o <= a.max_pages && c <= o * kPage && m <= a.max_pages * kPage - c;
    bad |= !ok;
    row[r] = ok ? s : -1;
    first[r] = ok ? c : 0;
    have[r] = ok ? o : 0;
    qo[r] = ok ? m : 0;
    const int listed = ok ? (c + m + kPage - 1) / kPage : 0;
    at[0] = sat_add(at[0], ok ? max(0, listed - o) : 0);
    at[1] = sat_add(at[1], ok ? m : 0);
    at[2] = sat_add(at[2], listed);
  }
  block_scan<3>(at, sums, total);
  uint32_t taken = total[0];   // pages taken (where they run out: up to this thread's last granted request)
  if (taken > static_cast<uint32_t>(ring_ok ? count : 0)) {
    // the free pages run out: who is granted, and their tokens and pages
    uint32_t some[2] = {0, 0}, sub[2];
    taken = 0;
    uint32_t asked = at[0];
    for (int r = lo; r < hi; ++r) {
      const int c = first[r], m = qo[r], need = max(0, (c + m + kPage - 1) / kPage - have[r]);
      asked = sat_add(asked, need);
      const bool granted = need == 0 || asked <= static_cast<uint32_t>(count);
      if (!granted) qo[r] = -1 - m;   // (its need still counts for those behind it)
      else if (need) taken = asked;
      some[0] = sat_add(some[0], granted ? m : 0);
      some[1] = sat_add(some[1], (c + (granted ? m : 0) + kPage - 1) / kPage);
    }
    block_scan<2>(some, sums2, sub);
    at[1] = some[0];
    at[2] = some[1];
    total[1] = sub[0];
    total[2] = sub[1];
  }
  const bool fits = total[1] <= static_cast<uint32_t>(a.T) && total[2] <= static_cast<uint32_t>(a.bt_cap);
  bad |= !fits;
  if (bad && blockIdx.x == 0) atomicExch(a.err, kErrBounds);
  const bool none = !fits;   // the caller's arrays are too short: nothing is granted, nothing changes
  for (int r = lo; r < hi; ++r) {
    const int asked = qo[r] < 0 ? -1 - qo[r] : qo[r];
    const int c = none ? 0 : first[r], m = none || qo[r] < 0 ? 0 : qo[r];
    ring0[r] = static_cast<int32_t>(at[0]);
    at[0] = sat_add(at[0], max(0, (first[r] + asked + kPage - 1) / kPage - have[r]));
    qo[r] = none ? 0 : static_cast<int32_t>(at[1]);
    bti[r] = none ? 0 : static_cast<int32_t>(at[2]);
    at[1] = sat_add(at[1], m);
    at[2] = sat_add(at[2], (c + m + kPage - 1) / kPage);
    if (blockIdx.x == 0) {
      a.qo_indptr[r] = qo[r];
      a.bt_indptr[r] = bti[r];
      a.kv_len[r] = c + m;
    }
  }
  const int tokens = none ? 0 : static_cast<int>(total[1]), pages = none ? 0 : static_cast<int>(total[2]);
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
  // Pages, then tokens, kBatch at a time: their loads go out together.
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads, all = static_cast<int64_t>(pages) + a.T;
  for (int64_t e0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; e0 < all; e0 += kBatch * step) {
    int req[kBatch], place[kBatch], page[kBatch];   // the request, the page's place in its row or the token's position
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t e = e0 + k * step, t = e - pages;
      req[k] = place[k] = page[k] = -1;
      if (e < pages) {
        req[k] = owner(bti, n, static_cast<int>(e));
        place[k] = static_cast<int>(e) - bti[req[k]];
        page[k] = page_of(req[k], place[k]);
      } else if (t < tokens) {
        req[k] = owner(qo, n, static_cast<int>(t));
        place[k] = first[req[k]] + static_cast<int>(t) - qo[req[k]];
        page[k] = page_of(req[k], place[k] / kPage);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t e = e0 + k * step, t = e - pages;
      const bool known = page[k] >= 0 && page[k] < a.num_pages;
      if (!known && (e < pages || (e < all && t < tokens))) atomicExch(a.err, kErrBounds);
      if (e < pages) {
        a.bt[e] = page[k];
        if (place[k] >= have[req[k]]) a.tables[static_cast<int64_t>(row[req[k]]) * a.max_pages + place[k]] = page[k];
      } else if (e < all) {
        a.tok_req[t] = req[k];
        a.tok_pos[t] = place[k];
        a.tok_slot[t] = known ? page[k] * kPage + place[k] % kPage : -1;   // (behind the last token: page -1)
      }
    }
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
  __shared__ uint32_t sums[kWarps][1];
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
  uint32_t at[1] = {0}, total[1];
  for (int r = lo; r < hi; ++r) {
    const int s = row[r], o = at0[r];
    bool ok = ring_ok && s >= 0 && s < a.max_slots && !((twice[s >> 5] >> (s & 31)) & 1u);
    ok = ok && o >= 0 && o <= a.max_pages;
    bad |= !ok;
    row[r] = ok ? s : -1;
    at0[r] = ok ? o : 0;
    at[0] = sat_add(at[0], ok ? o : 0);
  }
  block_scan<1>(at, sums, total);
  const bool fits = ring_ok && total[0] <= static_cast<uint32_t>(a.num_pages - count);
  bad |= !fits;
  if (bad && blockIdx.x == 0) atomicExch(a.err, kErrBounds);
  for (int r = lo; r < hi; ++r) {
    const int o = at0[r];
    at0[r] = static_cast<int32_t>(at[0]);
    at[0] = sat_add(at[0], o);
  }
  if (threadIdx.x == 0) at0[n] = static_cast<int32_t>(total[0]);
  __syncthreads();   // at0 is written, and the words that the last CTA changes read
  const int before = arrive(a.state + 2);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
#pragma unroll 4
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; fits && e < total[0]; e += step) {
    const int r = owner(at0, n, static_cast<int>(e));
    int64_t i = static_cast<int64_t>(head) + count + e;
    if (i >= a.num_pages) i -= a.num_pages;
    a.ring[i] = a.tables[static_cast<int64_t>(row[r]) * a.max_pages + (e - at0[r])];
  }
  if (!last_cta(a.state + 2, before) || !fits) return;
  for (int r = lo; r < hi; ++r)
    if (row[r] >= 0) a.owned[row[r]] = 0;
  if (threadIdx.x == 0) a.state[1] = count + static_cast<int32_t>(total[0]);
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
