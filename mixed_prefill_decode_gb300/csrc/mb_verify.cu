// Verification of drafted tokens against the target model's probabilities.
//
// Request r's nodes are a tree (parent[i] < i; node 0, the last sampled
// token, is the root).  Row i of the logits is the target's distribution
// after node i: p = softmax(logits / temperature).  From the root on, the
// children of the current node are tested in index order and the first one
// accepted becomes the current node; when none is, one more token is drawn
// from what the refusals left of p.  With given uniform numbers u:
//
//  * draft probabilities q (row i: the draft's distribution after node i, its
//    children drawn from it): a refusal turns p into norm(max(0, p - q))
//    (Leviathan et al., "Fast Inference from Transformers via Speculative
//    Decoding", 2023; for several children Miao et al., "SpecInfer", 2024).
//    k refusals in a row leave max(0, p - a q) / c with a_0 = 0, c_0 = 1,
//    a_{k+1} = a_k + c_k, c_k = sum max(0, p - a_k q): subtracting q from
//    max(0, p - a q) / c and scaling by c leaves max(0, p - (a + c) q).  So
//    child x passes if u c q(x) < p(x) - a q(x).
//  * no draft probabilities (each child was proposed for certain): child x
//    passes if u (1 - refused mass) < p(x); a refused token's p becomes 0.
//  * temperature 0: child x passes if it is the argmax.
//
// The walk from node to node is serial and reads one row per accepted node,
// so a request is given to a cluster of CTAs that shares each row, and the
// rows of nodes that are never reached are not read.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mb_fixexp.cuh"
#include "mb_kernels.h"
#include "mb_launch.cuh"
#include "mb_ptx.cuh"

namespace mb {
namespace {

using namespace dev;

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kMaxCluster = 16;

struct VerifyParams {
  const __nv_bfloat16 *logits;
  const int32_t *tokens;
  const float *probs;
  const int32_t *qo_indptr, *parent;
  const float *temperature, *u_accept, *u_final;
  int32_t *n_accepted, *path, *next_token;
  int vocab, T, max_path, cluster;
  FixExpTable tab;
  int *err;
};

// What the CTAs of a cluster tell each other in one round (two buffers, used
// in turn: a buffer is written again only after the round that follows its
// reading has passed its barrier).
struct Exchange {
  float m[2][kMaxCluster], z[2][kMaxCluster];
  int32_t idx[2][kMaxCluster];
  int64_t s[2][kMaxCluster];
};

__device__ __forceinline__ void st_cluster32(const void *local, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(local), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster64(const void *local, uint32_t rank, int64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(local), rank)), "l"(v) : "memory");
}

struct VerifySmem {
  Exchange ex;
  float tab_hi[32], tab_lo[32];
  float wm[kVerWarps], wz[kVerWarps];
  int32_t wi[kVerWarps];
  int64_t ws[kVerWarps];
  int16_t parent[kMaxTreeNodes];
  int16_t child[kMaxTreeNodes];
  int32_t gone[kMaxTreeNodes];   // refused tokens of the current node (no draft probabilities)
  int32_t n_child, n_gone, state, next;
  double a, c;
};

__global__ void __launch_bounds__(kVerThreads) verify_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ VerifySmem sm;
  const int C = p.cluster;
  const uint32_t rank = C > 1 ? cluster_ctarank() : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    sm.tab_hi[threadIdx.x] = p.tab.hi[threadIdx.x];
    sm.tab_lo[threadIdx.x] = p.tab.lo[threadIdx.x];
  }
  pdl_wait();
  pdl_trigger();
  cluster_sync();   // every CTA of the cluster runs before one writes into another
  const int r = blockIdx.x / C;
  const int t0 = p.qo_indptr[r], n = p.qo_indptr[r + 1] - t0;
  int32_t *path = p.path + static_cast<int64_t>(r) * p.max_path;
  const bool bad = t0 < 0 || n < 0 || n > kMaxTreeNodes || t0 + n > p.T;
  if (bad || n == 0) {
    if (rank == 0) {
      if (threadIdx.x == 0) {
        if (bad) atomicExch(p.err, kErrBounds);
        p.n_accepted[r] = 0;
        p.next_token[r] = -1;
      }
      for (int k = threadIdx.x; k < p.max_path; k += kVerThreads) path[k] = -1;
    }
    return;
  }
  float temp = p.temperature ? p.temperature[r] : 0.f;
  if (!(temp >= 0.f)) {
    if (threadIdx.x == 0) atomicExch(p.err, kErrBounds);
    temp = 0.f;
  }
  const bool greedy = temp == 0.f;
  const double kd = greedy ? 0.0 : fmin(1.4426950408889634074 / static_cast<double>(temp), 1e30);
  const float kh = static_cast<float>(kd), kl = static_cast<float>(kd - static_cast<double>(kh));
  for (int i = threadIdx.x; i < n; i += kVerThreads) {
    int up = p.parent[t0 + i];
    if (up < -1 || up >= i) {
      if (rank == 0) atomicExch(p.err, kErrBounds);
      up = -1;
    }
    sm.parent[i] = static_cast<int16_t>(up);
  }
  __syncthreads();

  // this CTA's vectors (of 8 logits) of a row, and this warp's part of them
  const int nv = p.vocab / 8;
  const int c0 = static_cast<int>(static_cast<int64_t>(nv) * rank / C), c1 = static_cast<int>(static_cast<int64_t>(nv) * (rank + 1) / C);
  const int w0 = c0 + static_cast<int>(static_cast<int64_t>(c1 - c0) * warp / kVerWarps);
  const int w1 = c0 + static_cast<int>(static_cast<int64_t>(c1 - c0) * (warp + 1) / kVerWarps);
  int parity = 0;
  int cur = 0, len = 1;

  // Integer weights of one vector: e = 2^((l - m) k), less a z q (as
  // az_hi + az_lo per unit of q) where draft probabilities take part, refused
  // tokens at 0; in units of 2^-40.
  auto weights = [&](const uint4 &raw, int v, float m, const float *qrow, float az_hi, float az_lo, int n_gone,
                     int64_t (&w)[8]) {
    const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
    float q[8];
    if (qrow) {
      const float4 qa = reinterpret_cast<const float4 *>(qrow)[2 * v], qb = reinterpret_cast<const float4 *>(qrow)[2 * v + 1];
      q[0] = qa.x, q[1] = qa.y, q[2] = qa.z, q[3] = qa.w, q[4] = qb.x, q[5] = qb.y, q[6] = qb.z, q[7] = qb.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float l = (e & 1) ? bf16hi(x[e >> 1]) : bf16lo(x[e >> 1]);
      float hi, lo;
      fix_exp(l, m, kh, kl, sm.tab_hi, sm.tab_lo, &hi, &lo);
      if (qrow) {
        const float ph = q[e] * az_hi, pl = fmaf(q[e], az_hi, -ph) + q[e] * az_lo;
        const float d = hi - ph, bb = d - hi;
        const float de = (hi - (d - bb)) - (ph + bb);
        lo = de + (lo - pl);
        hi = d;
        if (!(hi + lo > 0.f)) hi = lo = 0.f;
      }
      w[e] = to_fix(hi, lo);
      if (w[e] < 0) w[e] = 0;
    }
    for (int g = 0; g < n_gone; ++g) {
      const int tok = sm.gone[g];
      if ((tok >> 3) == v)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((tok & 7) == e) w[e] = 0;
    }
  };
  // Sums of the weights over this warp's part (sm.ws), this CTA's, and (from
  // the exchange) the row's; the sum before this CTA's part goes to *before.
  auto weight_sums = [&](const uint4 *row, float m, const float *qrow, float az_hi, float az_lo, int n_gone,
                         int64_t *before) -> int64_t {
    int64_t sum = 0;
    for (int v = w0 + lane; v < w1; v += 32) {
      int64_t w[8];
      weights(row[v], v, m, qrow, az_hi, az_lo, n_gone, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += w[e];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) sm.ws[warp] = sum;
    __syncthreads();
    int64_t mine = 0;
#pragma unroll
    for (int w = 0; w < kVerWarps; ++w) mine += sm.ws[w];
    if (threadIdx.x < C) st_cluster64(&sm.ex.s[parity][rank], threadIdx.x, mine);
    cluster_sync();
    int64_t total = 0, pre = 0;
    for (int k = 0; k < C; ++k) {
      if (k == static_cast<int>(rank)) pre = total;
      total += sm.ex.s[parity][k];
    }
    parity ^= 1;
    *before = pre;
    return total;
  };

  while (true) {
    const uint4 *row = reinterpret_cast<const uint4 *>(p.logits + (static_cast<size_t>(t0) + cur) * p.vocab);
    // children of cur, in index order
    if (warp == 0) {
      int cnt = 0;
      if (len < p.max_path)
        for (int b = 0; b < n; b += 32) {
          const bool is = b + lane < n && b + lane > 0 && sm.parent[b + lane] == cur;
          const uint32_t mask = __ballot_sync(0xffffffffu, is);
          if (is) sm.child[cnt + __popc(mask & ((1u << lane) - 1))] = static_cast<int16_t>(b + lane);
          cnt += __popc(mask);
        }
      if (lane == 0) sm.n_child = cnt;
    }
    // the row's maximum (and the lowest index that has it)
    float bm = -INFINITY;
    int bi = 0x7fffffff;
    for (int v = w0 + lane; v < w1; v += 32) {
      const uint4 raw = row[v];
      const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float l = (e & 1) ? bf16hi(x[e >> 1]) : bf16lo(x[e >> 1]);
        if (l > bm) {   // indices ascend within a thread: the first maximum stays
          bm = l;
          bi = 8 * v + e;
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, bm, off);
      const int oi = __shfl_xor_sync(0xffffffffu, bi, off);
      if (om > bm || (om == bm && oi < bi)) bm = om, bi = oi;
    }
    if (lane == 0) sm.wm[warp] = bm, sm.wi[warp] = bi;
    __syncthreads();
    bm = -INFINITY;
    bi = 0x7fffffff;
#pragma unroll
    for (int w = 0; w < kVerWarps; ++w)
      if (sm.wm[w] > bm || (sm.wm[w] == bm && sm.wi[w] < bi)) bm = sm.wm[w], bi = sm.wi[w];
    const int n_child = sm.n_child;
    float z = 0.f;
    if (!greedy && n_child > 0) {
      // sum of 2^((l - bm) k), relative to this CTA's maximum
      for (int v = w0 + lane; v < w1; v += 32) {
        const uint4 raw = row[v];
        const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float l = (e & 1) ? bf16hi(x[e >> 1]) : bf16lo(x[e >> 1]);
          z += l == bm ? 1.f : fmaxf(ex2_approx((l - bm) * kh), 0.f);   // a NaN counts 0
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
      if (lane == 0) sm.wz[warp] = z;
      __syncthreads();
      z = 0.f;
#pragma unroll
      for (int w = 0; w < kVerWarps; ++w) z += sm.wz[w];
      if (bm == -INFINITY) z = 0.f;
    }
    if (threadIdx.x < C) {
      st_cluster32(&sm.ex.m[parity][rank], threadIdx.x, __float_as_uint(bm));
      st_cluster32(&sm.ex.z[parity][rank], threadIdx.x, __float_as_uint(z));
      st_cluster32(&sm.ex.idx[parity][rank], threadIdx.x, static_cast<uint32_t>(bi));
    }
    cluster_sync();
    float m = -INFINITY;
    int top = 0x7fffffff;
    for (int k = 0; k < C; ++k) {
      const float om = sm.ex.m[parity][k];
      const int oi = sm.ex.idx[parity][k];
      if (om > m || (om == m && oi < top)) m = om, top = oi;
    }
    float Z = 0.f;
    for (int k = 0; k < C; ++k) {
      const float om = sm.ex.m[parity][k];
      Z += om == m ? sm.ex.z[parity][k] : sm.ex.z[parity][k] * ex2_approx((om - m) * kh);
    }
    parity ^= 1;
    if (m == -INFINITY) top = 0;   // no token has a chance: token 0

    // the children's tests: every CTA comes to the same answer
    int taken = -1;
    int64_t total = 0, before = 0;
    int final_gone = 0;
    const float *qrow = nullptr;
    float az_hi = 0.f, az_lo = 0.f;
    bool have_sums = false;
    if (greedy || m == -INFINITY) {
      if (greedy)
        for (int k = 0; k < n_child && taken < 0; ++k)
          if (p.tokens[t0 + sm.child[k]] == top) taken = sm.child[k];
      if (taken < 0) {
        if (rank == 0 && threadIdx.x == 0) p.next_token[r] = top;
        if (rank == 0 && threadIdx.x == 0) path[len - 1] = cur;
        break;
      }
    } else if (!p.probs) {
      if (threadIdx.x == 0) {
        double gone = 0.0;
        int n_gone = 0;
        sm.state = -1;
        for (int k = 0; k < n_child; ++k) {
          const int node = sm.child[k];
          const int x = p.tokens[t0 + node];
          if (x < 0 || x >= p.vocab) {
            atomicExch(p.err, kErrBounds);
            continue;
          }
          bool dup = false;
          for (int g = 0; g < n_gone; ++g) dup |= sm.gone[g] == x;
          if (dup) continue;
          const float l = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[x]);
          const float e = l == m ? 1.f : fmaxf(ex2_approx((l - m) * kh), 0.f);
          if (static_cast<double>(p.u_accept[t0 + node]) * (static_cast<double>(Z) - gone) < static_cast<double>(e)) {
            sm.state = node;
            break;
          }
          sm.gone[n_gone++] = x;
          gone += static_cast<double>(e);
        }
        sm.n_gone = n_gone;
      }
      __syncthreads();
      taken = sm.state;
      final_gone = sm.n_gone;
    } else {
      const float *q = p.probs + (static_cast<size_t>(t0) + cur) * p.vocab;
      double a = 0.0, c = 1.0, zd = Z;   // c in units of the row's sum z
      for (int k = 0; k < n_child; ++k) {
        if (threadIdx.x == 0) {
          const int node = sm.child[k];
          const int x = p.tokens[t0 + node];
          sm.state = 0;
          if (x < 0 || x >= p.vocab) {
            atomicExch(p.err, kErrBounds);
          } else {
            const float l = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[x]);
            float hi, lo;
            fix_exp(l, m, kh, kl, sm.tab_hi, sm.tab_lo, &hi, &lo);
            const double px = (static_cast<double>(hi) + static_cast<double>(lo)) / zd, qx = q[x];
            if (static_cast<double>(p.u_accept[t0 + node]) * c * qx < px - a * qx) sm.state = 1;
          }
        }
        __syncthreads();
        const bool pass = sm.state == 1;
        __syncthreads();
        if (pass) {
          taken = sm.child[k];
          break;
        }
        if (!qrow) {   // the first refusal: the row's sum to full accuracy
          zd = static_cast<double>(weight_sums(row, m, nullptr, 0.f, 0.f, 0, &before)) * 0x1p-40;
          qrow = q;
        }
        a += c;
        const double az = a * zd;
        az_hi = static_cast<float>(az);
        az_lo = static_cast<float>(az - static_cast<double>(az_hi));
        total = weight_sums(row, m, qrow, az_hi, az_lo, 0, &before);
        c = static_cast<double>(total) * 0x1p-40 / zd;
        have_sums = true;
      }
    }
    if (rank == 0 && threadIdx.x == 0) path[len - 1] = cur;
    if (taken >= 0) {
      cur = taken;
      ++len;
      __syncthreads();   // sm.child, sm.gone and sm.state are read before the next node writes them
      continue;
    }
    // none accepted: one token of what is left
    if (!have_sums) total = weight_sums(row, m, nullptr, 0.f, 0.f, final_gone, &before);
    if (total == 0) {    // the refusals left nothing: p itself
      qrow = nullptr;
      final_gone = 0;
      total = weight_sums(row, m, nullptr, 0.f, 0.f, 0, &before);
    }
    const double uf = static_cast<double>(p.u_final[r]);
    int64_t pick = uf > 0.0 ? static_cast<int64_t>(fmin(uf, 1.0) * static_cast<double>(total)) : 0;
    if (pick > total - 1) pick = total - 1;
    // the first token whose cumulative weight is above pick
    int64_t at = before;
    for (int w = 0; w < warp; ++w) at += sm.ws[w];
    if (at <= pick && pick < at + sm.ws[warp]) {
      for (int v0 = w0; v0 < w1; v0 += 32) {
        int64_t w[8], sum = 0;
        const int v = v0 + lane;
        if (v < w1) {
          weights(row[v], v, m, qrow, az_hi, az_lo, final_gone, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum += w[e];
        }
        int64_t inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
          if (lane >= off) inc += o;
        }
        int64_t run = at + inc - sum;
        if (run <= pick && pick < run + sum) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (run <= pick && pick < run + w[e]) p.next_token[r] = 8 * v + e;
            run += w[e];
          }
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
        if (at > pick) break;
      }
    }
    break;
  }
  if (rank == 0) {
    if (threadIdx.x == 0) p.n_accepted[r] = len;
    for (int k = len + threadIdx.x; k < p.max_path; k += kVerThreads) path[k] = -1;
  }
}

}  // namespace

cudaError_t verify_tree_run(const VerifyArgs &a, cudaStream_t st) {
  if (a.n_reqs <= 0) return cudaSuccess;
  VerifyParams p;
  p.logits = static_cast<const __nv_bfloat16 *>(a.logits);
  p.tokens = a.tokens;
  p.probs = a.probs;
  p.qo_indptr = a.qo_indptr;
  p.parent = a.parent;
  p.temperature = a.temperature;
  p.u_accept = a.u_accept;
  p.u_final = a.u_final;
  p.n_accepted = a.n_accepted;
  p.path = a.path;
  p.next_token = a.next_token;
  p.vocab = a.vocab;
  p.T = a.T;
  p.max_path = a.max_path;
  p.cluster = 1;
  static const FixExpTable table = fix_exp_table();
  p.tab = table;
  p.err = a.err;
  return launch_pdl(verify_kernel, dim3(a.n_reqs * p.cluster), dim3(kVerThreads), 0, st, p.cluster, p);
}

}  // namespace mb
