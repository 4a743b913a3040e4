// Attention for trees of drafted tokens over the paged KV cache.
//
// A request r brings n tokens (the nodes of a tree, or of several: parent[i] <
// i is the index of node i's parent within the request, -1 for a node that
// hangs on the cached prefix) whose keys and values already sit at positions
// c .. c + n - 1 of its cache, c = kv_len - n.  Node i sees the prefix, its
// ancestors and itself:
//
//   o_i = sum_j p_ij v_j,   p_i = softmax_j (q_i . k_j / sqrt(hd)),
//   j in {0 .. c - 1} + {c + a : a an ancestor of i, or i}
//
// for every q-head; q-head h reads KV head h / (Hq / Hkv).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mb_kernels.h"
#include "mb_launch.cuh"
#include "mb_ptx.cuh"

namespace mb {
namespace {

using namespace dev;

constexpr float kLog2e = 1.4426950408889634f;

struct TreeParams {
  const __nv_bfloat16 *q, *pool;
  __nv_bfloat16 *o;
  const int32_t *qo_indptr, *kv_len, *bt_indptr, *bt, *parent;
  int n_reqs, T, Hq, Hkv, num_pages;
  float scale_log2;
  int *err;
};

// One CTA per (token, KV head); each warp takes every fourth key.
template <int HD>
__global__ void __launch_bounds__(128) tree_simple_kernel(const TreeParams p) {
  constexpr int PER = HD / 32;
  __shared__ uint32_t sees[kMaxTreeNodes / 32];
  __shared__ float s_m[4][8], s_l[4][8], s_o[4][8][HD];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, hk = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  int lo = 0, hi = p.n_reqs;   // the request r with qo[r] <= t < qo[r + 1]
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (p.qo_indptr[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  if (lo == p.n_reqs) return;   // a row behind the last request
  const int r = lo, t0 = p.qo_indptr[r], n = p.qo_indptr[r + 1] - t0, kv = p.kv_len[r], c = kv - n;
  const int pages = p.bt_indptr[r + 1] - p.bt_indptr[r];
  if (n > kMaxTreeNodes || t0 < 0 || t0 + n > p.T || c < 0 || (kv + 15) / 16 > pages || p.bt_indptr[r] < 0) {
    if (threadIdx.x == 0) atomicExch(p.err, kErrBounds);
    return;
  }
  const int32_t *table = p.bt + p.bt_indptr[r];
  const int i = t - t0;
  if (threadIdx.x < kMaxTreeNodes / 32) sees[threadIdx.x] = 0;
  __syncthreads();
  if (threadIdx.x == 0) {
    int x = i;
    while (x >= 0) {
      sees[x >> 5] |= 1u << (x & 31);
      int up = p.parent[t0 + x];
      if (up < -1 || up >= x) {
        atomicExch(p.err, kErrBounds);
        up = -1;
      }
      x = up;
    }
  }
  __syncthreads();
  float q[8][PER], o[8][PER], m[8], l[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      o[g][k] = 0.f;
      q[g][k] = g < G ? __bfloat162float(p.q[(static_cast<size_t>(t) * p.Hq + hk * G + g) * HD + lane + 32 * k]) : 0.f;
    }
  }
  for (int j = warp; j < kv; j += 4) {
    if (j >= c && !((sees[(j - c) >> 5] >> ((j - c) & 31)) & 1u)) continue;
    const int page = table[j / kPage];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) atomicExch(p.err, kErrBounds);
      continue;
    }
    const __nv_bfloat16 *kr = p.pool + ((static_cast<size_t>(page) * 2 * p.Hkv + hk) * kPage + j % kPage) * HD;
    const __nv_bfloat16 *vr = kr + static_cast<size_t>(p.Hkv) * kPage * HD;
    float kx[PER], vx[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      kx[k] = __bfloat162float(kr[lane + 32 * k]);
      vx[k] = __bfloat162float(vr[lane + 32 * k]);
    }
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      if (g >= G) break;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < PER; ++k) s = fmaf(q[g][k], kx[k], s);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s *= p.scale_log2;
      const float mn = fmaxf(m[g], s);
      const float al = ex2_approx(m[g] - mn), pr = ex2_approx(s - mn);
      m[g] = mn;
      l[g] = fmaf(l[g], al, pr);
#pragma unroll
      for (int k = 0; k < PER; ++k) o[g][k] = fmaf(o[g][k], al, pr * vx[k]);
    }
  }
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    if (g >= G) break;
    if (lane == 0) {
      s_m[warp][g] = m[g];
      s_l[warp][g] = l[g];
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) s_o[warp][g][lane + 32 * k] = o[g][k];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < G * HD; e += 128) {
    const int g = e / HD, d = e % HD;
    float M = -INFINITY;
    for (int w = 0; w < 4; ++w) M = fmaxf(M, s_m[w][g]);
    float L = 0.f, acc = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float a = s_l[w][g] > 0.f ? ex2_approx(s_m[w][g] - M) : 0.f;
      L = fmaf(a, s_l[w][g], L);
      if (a > 0.f) acc = fmaf(a, s_o[w][g][d], acc);
    }
    p.o[(static_cast<size_t>(t) * p.Hq + hk * G + g) * HD + d] = __float2bfloat16_rn(acc / L);
  }
}

}  // namespace

size_t tree_workspace_bytes() { return 256; }

cudaError_t tree_attention_run(const TreeArgs &a, cudaStream_t st) {
  if (a.n_reqs <= 0 || a.T <= 0) return cudaSuccess;
  TreeParams p;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.pool = static_cast<const __nv_bfloat16 *>(a.pool);
  p.o = static_cast<__nv_bfloat16 *>(a.o);
  p.qo_indptr = a.qo_indptr;
  p.kv_len = a.kv_len;
  p.bt_indptr = a.bt_indptr;
  p.bt = a.bt;
  p.parent = a.parent;
  p.n_reqs = a.n_reqs;
  p.T = a.T;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.num_pages = a.num_pages;
  p.scale_log2 = kLog2e / sqrtf(static_cast<float>(a.hd));
  p.err = a.err;
  if (a.hd == 128) return launch_pdl(tree_simple_kernel<128>, dim3(a.T, a.Hkv), dim3(128), 0, st, 1, p);
  return launch_pdl(tree_simple_kernel<64>, dim3(a.T, a.Hkv), dim3(128), 0, st, 1, p);
}

}  // namespace mb
