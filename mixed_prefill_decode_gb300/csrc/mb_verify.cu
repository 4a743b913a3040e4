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
// What bounds it: the walk from node to node is serial, and a step of it is the
// latency of one row (load, maximum and sum, exchange), so a request is given
// to a cluster of CTAs that shares each row, and the rows of nodes that are
// never reached are not read.  A thread keeps its part of the row in shared
// memory (copied asynchronously) between the maximum, the sum and the draw.
//
// The tests compare in fp32 (the special-function unit's exponentials).  Where
// that is too close to tell (so also where little is left of p: a child of p =
// 0.9999 refused), after a refusal with draft probabilities and for the draw at
// the end, the row is summed with accurate weights (mb_fixexp.cuh): as integers,
// so that no decision depends on how many CTAs share the row.  That is one pass
// over the last row as a rule, two after a refusal with draft probabilities.
// Its arithmetic is what a full GPU spends most of its time on.
//
// Measured (replays of a graph, the mean of four sets of inputs: a call takes as
// long as its longest walk): one chain of 5 drafted tokens, vocabulary 128,256,
// with draft probabilities, 30 us, some 3.5 us a node; 64 such 76 us, of which a
// node's step takes about 5 us and an accurate pass over the row 10 to 15 (the
// walks read 82 MB: 1.1 TB/s); 64 without draft probabilities 52 us; 16 trees of
// 24, vocabulary 50,264, 22.7 us; 6 tokens, greedy, vocabulary 32,000, 8 to 19 us
// by the length of the path.  Tried and dropped: a table of the weights of all
// bf16 logits in shared memory (its random 8-byte reads took 7 cycles a warp);
// accurate sums after every refusal (16 trees 29.3 us against 23.6: most tests
// are far from their border); an only child's row fetched over its parent's, with
// its maximum and sum computed during the parent's exchange (64 chains 80 us
// against 78: what it hides is latency that the SM's other CTAs hide already, and
// a refusal has to fetch the parent's row again).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mb_fixexp.cuh"
#include "mb_launch.cuh"
#include "mb_ptx.cuh"
#include "mb_spec.h"

namespace mb {
namespace {

using namespace dev;

constexpr int kVerThreads = 256;   // (512 and two CTAs an SM: 64 chains 84 us against 79, 256 of 3 317 against 239)
constexpr int kVerPerSm = 4;       // CTAs an SM holds
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kMaxCluster = 16;
// A test in fp32, u (z - refused) q < e, is repeated with accurate sums where
// its sides are apart by less than this part of u z q + e.  The exponent of a
// weight, at most 126 (m - l) k, is rounded three times: e is off by 126 ln 2 3
// 2^-24 = 1.6e-5; in z and the refused ones' sum weights below 2^-45 count
// nothing: 6e-6 each, and up to 80 and 127 additions in a row: 1.3e-5.  In all
// 1.6e-5 e + 2.6e-5 u z q.
constexpr float kNear = 0x1p-14f;
constexpr int kMaxVocab = 1 << 19;
constexpr int kMaxHeld = kMaxVocab / 8 / kMaxCluster / kVerThreads;   // vectors that a thread holds at most
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
  int64_t vec[32 * kMaxHeld];    // the drawing warp: weights of its vectors
  uint32_t tab_fix[32];
  float tab_scaled[32];
  float wm[kVerWarps], wz[kVerWarps];
  int32_t wi[kVerWarps];
  int64_t ws[kVerWarps];
  int16_t parent[kMaxTreeNodes];
  int16_t child[kMaxTreeNodes];
  int32_t token[kMaxTreeNodes];
  float u[kMaxTreeNodes], logit[kMaxTreeNodes], q[kMaxTreeNodes];   // of the node's token in its parent's rows
  int32_t gone[kMaxTreeNodes];   // refused tokens of the current node (no draft probabilities)
  int64_t gone_w[kMaxTreeNodes]; // their weights, of those refused since the row was summed
  int32_t n_child, n_gone, at, state, low;
  float kh, kl, az_hi, az_lo, u_final;
  int64_t pick;
};

// What a child's test comes to (also where a child's index may stand).
enum : int { kRefused = -1, kNearBorder = -2, kPassed = -3, kNoToken = -4 };

// (at file scope, so that the functions below address it as shared memory)
__shared__ VerifySmem sm;

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The larger of two pairs of bf16, a NaN giving way to a number.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float bf16_of(const uint4 &raw, int e) {
  const uint32_t w = e < 4 ? (e < 2 ? raw.x : raw.y) : (e < 6 ? raw.z : raw.w);
  return (e & 1) ? bf16hi(w) : bf16lo(w);
}

// What a weight depends on beside its logit and draft probability.
struct WeightCtx {
  float m, kh32, kl32;     // weight 2^((l - m) k), 32 k = kh32 + kl32
  float d_max;             // m - l from which on it is 2^-48
  float az_hi, az_lo;      // less az q (both times 2^20)
  float q_small, q_any;    // q from which on az q is above 2^-11, above 1
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Two weights as fix_exp computes them, in packed fp32: v 2^(11 - s) in units
// of 2^-41, to be rounded.  D: m - l.
__device__ __forceinline__ void weight_pair(const WeightCtx &c, float2 D, uint32_t *v, int32_t *s) {
  D.x = fminf(D.x, c.d_max);   // (an infinity, a NaN: 2^-48, which rounds to 0)
  D.y = fminf(D.y, c.d_max);
  const float2 t = __ffma2_rn(D, both(c.kh32), both(kFixMagic));
  const float2 n = __fadd2_rn(t, both(-kFixMagic));
  const float2 f = __ffma2_rn(D, both(-c.kl32), __ffma2_rn(D, both(-c.kh32), n));
  float2 g = __ffma2_rn(f, both(kFixC4), both(kFixC3));
  g = __ffma2_rn(g, f, both(kFixC2));
  g = __ffma2_rn(g, f, both(kFixC1));
  g = __fmul2_rn(g, f);
  const int32_t t0 = __float_as_int(t.x), t1 = __float_as_int(t.y);
  s[0] = (t0 - kFixMagicBits + 31) >> 5;
  s[1] = (t1 - kFixMagicBits + 31) >> 5;
  v[0] = sm.tab_fix[t0 & 31] + static_cast<uint32_t>(__float2int_rn(sm.tab_scaled[t0 & 31] * g.x));
  v[1] = sm.tab_fix[t1 & 31] + static_cast<uint32_t>(__float2int_rn(sm.tab_scaled[t1 & 31] * g.y));
}

// The weight from v and s: in 32 bits if it is below 2^-11 (s >= 12), in 64.
__device__ __forceinline__ int32_t small_weight(uint32_t v, int32_t s) {
  return static_cast<int32_t>(((v >> min(s - 12, 31)) + 1) >> 1);
}
__device__ __forceinline__ int64_t large_weight(uint32_t v, int32_t s) {
  return static_cast<int64_t>((((static_cast<uint64_t>(v) << 12) >> s) + 1) >> 1);
}

// az q in units of 2^-41, as hi 2^21 + lo.  A q above `top` (a NaN too) counts
// as that: az q is then more than any weight beside it.  One below 0 counts as
// 0: no weight grows, and the sums stay within 64 bits.  (In packed fp32, two
// tokens at a time, 64 chains took 77.6 us against 76.3.)
__device__ __forceinline__ void fixed_q(const WeightCtx &c, float q, float top, int32_t &hi, int32_t &lo) {
  q = fmaxf(fminf(q, top), 0.f);
  const float x = q * c.az_hi, l = fmaf(q, c.az_lo, fmaf(q, c.az_hi, -x));
  const float a = x + kFixMagic;
  const float b = fmaf((x - (a - kFixMagic)) + l, 0x1p21f, kFixMagic);
  hi = __float_as_int(a) - kFixMagicBits;
  lo = __float_as_int(b) - kFixMagicBits;
}

// m - l, with a row's infinities in order: l = m gives 0, less than m = +inf everything.
__device__ __forceinline__ float below(const WeightCtx &c, float l) { return l == c.m ? 0.f : c.m - l; }

// The weight of one token (any lane by itself).
__device__ __noinline__ int64_t token_weight(const WeightCtx &c, float l, bool probs, float q) {
  uint32_t v[2];
  int32_t s[2], hi, lo;
  weight_pair(c, make_float2(below(c, l), 0.f), v, s);
  const int64_t w = large_weight(v[0], s[0]);
  if (!probs) return w;
  fixed_q(c, q, c.q_any, hi, lo);
  return max(w - (static_cast<int64_t>(hi) << 21) - lo, static_cast<int64_t>(0));
}

// Weight of a vector (8 tokens, at x; q: their draft probabilities).  By all
// lanes of a warp (live: the lane has such a vector).
// The 8 weights are computed side by side and their sum in 32 bits a pair,
// unless one of the warp's 256 is 2^-11 or more.
template <bool PROBS>
__device__ __forceinline__ int64_t vector_weight(const WeightCtx &c, const uint4 *x, bool live, float4 qa, float4 qb) {
  const uint4 raw = live ? *x : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);   // -inf
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  const float q[8] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
  int64_t sum = 0;
  if (c.m < INFINITY) {
    uint32_t wv[8];
    int32_t ws[8];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      weight_pair(c, make_float2(c.m - bf16lo(w[e]), c.m - bf16hi(w[e])), wv + 2 * e, ws + 2 * e);
    const int least = min(min(min(ws[0], ws[1]), min(ws[2], ws[3])), min(min(ws[4], ws[5]), min(ws[6], ws[7])));
    if (__any_sync(0xffffffffu, least < 12)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        int64_t a = large_weight(wv[e], ws[e]);
        if (PROBS) {
          int32_t hi, lo;
          fixed_q(c, q[e], c.q_any, hi, lo);
          a = max(a - (static_cast<int64_t>(hi) << 21) - lo, static_cast<int64_t>(0));
        }
        sum += a;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        int32_t a[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          a[h] = small_weight(wv[e + h], ws[e + h]);
          if (PROBS) {
            int32_t hi, lo;
            fixed_q(c, q[e + h], c.q_small, hi, lo);
            a[h] = max(a[h] - (hi << 21) - lo, 0);
          }
        }
        sum += static_cast<uint32_t>(a[0]) + static_cast<uint32_t>(a[1]);
      }
    }
  } else {
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      const float lg = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(x)[e]);
      if (live) sum += token_weight(c, lg, PROBS, e < 4 ? (e < 2 ? (e ? qa.y : qa.x) : (e == 2 ? qa.z : qa.w)) : (e < 6 ? (e == 4 ? qb.x : qb.y) : (e == 6 ? qb.z : qb.w)));
    }
  }
  return sum;
}

// A thread's part of the row, and the state of the cluster's exchange.
struct Part {
  const uint4 *x;    // held vectors, kVerThreads apart
  int nk, nk_warp, v0;   // their number, the most of a lane, and the first one's place in the row (then every 32nd)
  int C, rank;
  int parity;        // exchange buffer of the next round
};

__device__ __forceinline__ float4 load_q(const float *qrow, int v) { return __ldg(reinterpret_cast<const float4 *>(qrow) + v); }

// Sums of the weights over each warp's part (sm.ws), the CTA's, and (from the
// exchange) the row's; the sum before this CTA's part goes to *before.  All
// threads of the cluster.  Out of line: it is called in four places.
template <bool PROBS>
__device__ __noinline__ int64_t weight_sums(Part &t, const WeightCtx &c, const float *qrow, int64_t *before) {
  __syncthreads();   // sm.ws has been read
  int64_t sum = 0;
  float4 qa = make_float4(0.f, 0.f, 0.f, 0.f), qb = qa;
  if (PROBS && t.nk > 0) qa = load_q(qrow, 2 * t.v0), qb = load_q(qrow, 2 * t.v0 + 1);
#pragma unroll 1
  for (int k = 0; k < t.nk_warp; ++k) {
    const int v = t.v0 + 32 * k;
    float4 na = qa, nb = qb;   // the next vector's draft probabilities, in flight meanwhile
    if (PROBS && k + 1 < t.nk) na = load_q(qrow, 2 * v + 64), nb = load_q(qrow, 2 * v + 65);
    sum += vector_weight<PROBS>(c, t.x + k * kVerThreads, k < t.nk, qa, qb);
    qa = na, qb = nb;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if ((threadIdx.x & 31) == 0) sm.ws[threadIdx.x >> 5] = sum;
  __syncthreads();
  int64_t mine = 0;
#pragma unroll
  for (int w = 0; w < kVerWarps; ++w) mine += sm.ws[w];
  *before = 0;
  if (t.C == 1) return mine;
  if (threadIdx.x < t.C) st_cluster64(&sm.ex.s[t.parity][t.rank], threadIdx.x, mine);
  cluster_sync();
  int64_t total = 0;
  for (int k = 0; k < t.C; ++k) {
    if (k == t.rank) *before = total;
    total += sm.ex.s[t.parity][k];
  }
  t.parity ^= 1;
  return total;
}

// The largest logit that the cluster's CTAs hold.  All threads.
__device__ __noinline__ float row_max(Part &t) {
  __syncthreads();   // sm.wm has been read
  uint32_t pm = 0xFF80FF80u;   // -inf (a NaN is passed over)
  for (int k = 0; k < t.nk; ++k) {
    const uint4 v = t.x[k * kVerThreads];
    pm = max_bf16x2(max_bf16x2(pm, v.x), max_bf16x2(v.y, max_bf16x2(v.z, v.w)));
  }
  float m = fmaxf(bf16lo(pm), bf16hi(pm));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if ((threadIdx.x & 31) == 0) sm.wm[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kVerWarps; ++w) m = fmaxf(m, sm.wm[w]);
  if (t.C == 1) return m;
  if (threadIdx.x < t.C) st_cluster32(&sm.ex.m[t.parity][t.rank], threadIdx.x, __float_as_uint(m));
  cluster_sync();
  for (int k = 0; k < t.C; ++k) m = fmaxf(m, sm.ex.m[t.parity][k]);
  t.parity ^= 1;
  return m;
}

__global__ void __launch_bounds__(kVerThreads, kVerPerSm) verify_kernel(const __grid_constant__ VerifyParams p) {
  extern __shared__ __align__(16) uint4 held[];   // vector k of thread t at k kVerThreads + t
  const int C = p.cluster;
  const uint32_t rank = C > 1 ? cluster_ctarank() : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    sm.tab_fix[threadIdx.x] = p.tab.fix[threadIdx.x];
    sm.tab_scaled[threadIdx.x] = p.tab.scaled[threadIdx.x];
  }
  pdl_wait();
  pdl_trigger();
  if (C > 1) cluster_sync();   // every CTA of the cluster runs before one writes into another
  const int r = blockIdx.x / C;
  const int t0 = p.qo_indptr[r], t1 = p.qo_indptr[r + 1];
  int32_t *path = p.path + static_cast<int64_t>(r) * p.max_path;
  const bool order = t0 >= 0 && t1 >= t0 && t1 <= p.T;   // (compared before they are subtracted: the words may be anything)
  const int n = order ? t1 - t0 : 0;
  const bool bad = !order || n > kMaxTreeNodes;
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
  // this CTA's vectors of a row, and this warp's part of them: lane l holds
  // vectors w0 + l + 32 k, so a warp's sums cover consecutive tokens
  const int nv = p.vocab / 8;
  const int c0 = static_cast<int>(static_cast<int64_t>(nv) * rank / C), c1 = static_cast<int>(static_cast<int64_t>(nv) * (rank + 1) / C);
  const int w0 = c0 + (c1 - c0) * warp / kVerWarps, w1 = c0 + (c1 - c0) * (warp + 1) / kVerWarps;
  const int nk = (w1 - w0 - lane + 31) / 32;       // this thread's vectors
  uint4 *x = held + threadIdx.x;
  auto load_row = [&](int node) {
    const uint4 *row = reinterpret_cast<const uint4 *>(p.logits + (static_cast<size_t>(t0) + node) * p.vocab);
    for (int k = 0; k < nk; ++k) cp_async16(x + k * kVerThreads, row + w0 + lane + 32 * k);
  };
  load_row(0);
  // The request's words, each thread's loads side by side.
  const float temp_in = p.temperature ? p.temperature[r] : 0.f;
  const int i = threadIdx.x;   // its node
  int up = -1, tok = 0;
  float u = 0.f, u_last = 0.f;
  if (i < n) {
    up = p.parent[t0 + i];
    if (i > 0) tok = p.tokens[t0 + i];
    if (i > 0 && p.temperature) u = p.u_accept[t0 + i];
  }
  if (threadIdx.x == kVerThreads - 1 && p.temperature) u_last = p.u_final[r];
  const bool temp_ok = temp_in >= 0.f;
  const float temp = temp_ok ? temp_in : 0.f;
  const bool greedy = temp == 0.f;
  if (threadIdx.x == kVerThreads - 1) {   // (FP64 is slow: one thread's work, of a warp without nodes)
    if (!temp_ok) atomicExch(p.err, kErrBounds);
    const double kd = greedy ? 0.0 : fmax(fmin(1.4426950408889634074 / static_cast<double>(temp), 1e30), 1e-30);
    sm.u_final = u_last;
    sm.kh = static_cast<float>(kd);
    sm.kl = static_cast<float>(kd - static_cast<double>(sm.kh));
  }
  static_assert(kMaxTreeNodes < kVerThreads, "one thread a node");
  if (i < n) {
    const bool bad_up = up < -1 || up >= i, bad_tok = tok < 0 || tok >= p.vocab;
    if (bad_up || bad_tok) atomicExch(p.err, kErrBounds);
    if (bad_up) up = -1;
    sm.parent[i] = static_cast<int16_t>(up);
    sm.token[i] = bad_tok ? -1 : tok;
    sm.u[i] = u;
    const size_t at = (static_cast<size_t>(t0) + max(up, 0)) * p.vocab + (bad_tok ? 0 : tok);
    sm.logit[i] = greedy ? 0.f : __bfloat162float(p.logits[at]);
    const float q = greedy || !p.probs ? 0.f : p.probs[at];
    sm.q[i] = q < 0.f ? 0.f : q;   // (a NaN stays one: the child is refused)
  }
  __syncthreads();

  const float kh = sm.kh, kl = sm.kl, d_max = fminf(48.f / fmaxf(kh, 1e-30f), 3e38f);
  Part part{x, nk, (w1 - w0 + 31) / 32, w0 + lane, C, static_cast<int>(rank), 0};

  // A row's maximum (and, greedy, the lowest index that has it) and the sum of
  // 2^((l - max) k) over this warp's part, to sm.wm, wz, wi.
  auto warp_part = [&]() {
    float bm = -INFINITY, z = 0.f;
    int bi = 0x7fffffff;
    cp_async_wait();
    uint32_t pm = 0xFF80FF80u;   // -inf
#pragma unroll 2
    for (int k = 0; k < nk; ++k) {
      const uint4 v = x[k * kVerThreads];   // (a NaN is passed over)
      pm = max_bf16x2(max_bf16x2(pm, v.x), max_bf16x2(v.y, max_bf16x2(v.z, v.w)));
    }
    bm = fmaxf(bf16lo(pm), bf16hi(pm));
    if (greedy) {
      for (int k = nk - 1; k >= 0; --k) {
        const uint4 v = x[k * kVerThreads];
#pragma unroll
        for (int e = 7; e >= 0; --e)
          if (bf16_of(v, e) == bm) bi = 8 * (w0 + lane + 32 * k) + e;
      }
      if (bm == -INFINITY) bi = 0x7fffffff;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, bm, off);
        const int oi = __shfl_xor_sync(0xffffffffu, bi, off);
        if (om > bm || (om == bm && oi < bi)) bm = om, bi = oi;
      }
    } else {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, off));
      // relative to the warp's maximum (finite, or -inf: then there is nothing, or +inf: they share)
      const float ref = fabsf(bm) == INFINITY ? 0.f : bm;
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int k = 0; k < nk; ++k) {
        const uint4 v = x[k * kVerThreads];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 y = __fmul2_rn(__fadd2_rn(make_float2(bf16lo(w[e]), bf16hi(w[e])), both(-ref)), both(kh));
          sum = __fadd2_rn(sum, make_float2(ex2_approx(y.x), ex2_approx(y.y)));
        }
      }
      z = sum.x + sum.y;
      if (z != z) {   // a NaN counts 0
        z = 0.f;
#pragma unroll 1
        for (int k = 0; k < 8 * nk; ++k) z += fmaxf(ex2_approx((bf16_of(x[(k >> 3) * kVerThreads], k & 7) - ref) * kh), 0.f);
      }
      if (fabsf(bm) == INFINITY) {
        z = 0.f;
        if (bm > 0.f)
          for (int k = 0; k < nk; ++k)
            for (int e = 0; e < 8; ++e) z += bf16_of(x[k * kVerThreads], e) == bm ? 1.f : 0.f;
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    }
    if (lane == 0) sm.wm[warp] = bm, sm.wz[warp] = z, sm.wi[warp] = bi;
  };
  // n (maximum, sum, index) triples, one per lane: of all together.
  auto join = [&](float &m, float &s, int &i, int n) {
    float top_m = m;
    for (int off = n >> 1; off > 0; off >>= 1) top_m = fmaxf(top_m, __shfl_xor_sync(0xffffffffu, top_m, off));
    s = m == top_m ? s : m == -INFINITY || top_m == INFINITY ? 0.f : s * ex2_approx((m - top_m) * kh);
    i = m == top_m ? i : 0x7fffffff;
    for (int off = n >> 1; off > 0; off >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, off);
      i = min(i, __shfl_xor_sync(0xffffffffu, i, off));
    }
    m = top_m;
  };

  // A test in fp32: a < e, `scale` the terms that a is the difference of.
  auto fast_test = [](float a, float scale, float e) {
    const bool near = fabsf(a - e) <= kNear * (scale + e) || (e == 0.f && a < 0x1p-100f);   // (e may have been flushed to 0)
    return near ? kNearBorder : a < e ? kPassed : kRefused;
  };
  // Refused tokens (from the from-th on) leave the held row.
  auto drop_gone = [&](int from, int to) {
    for (int g = from; g < to; ++g) {
      const int tok = sm.gone[g], at = (tok >> 3) - w0;   // the vector's place in the warp's part
      if (at >= 0 && at < w1 - w0 && (at & 31) == lane)
        reinterpret_cast<uint16_t *>(x + (at >> 5) * kVerThreads)[tok & 7] = 0xFF80u;   // -inf
    }
  };

  int cur = 0, len = 1;

  while (true) {
    warp_part();
    // its children, in index order
    if (warp == 0) {
      int n_child = 0;
      if (len < p.max_path)
        for (int b = 0; b < n; b += 32) {
          const bool is = b + lane < n && b + lane > 0 && sm.parent[b + lane] == cur;
          const uint32_t mask = __ballot_sync(0xffffffffu, is);
          if (is) sm.child[n_child + __popc(mask & ((1u << lane) - 1))] = static_cast<int16_t>(b + lane);
          n_child += __popc(mask);
        }
      if (lane == 0) sm.n_child = n_child;
    }
    __syncthreads();
    // the CTA's part for the others
    if (warp == 0) {
      float m = sm.wm[lane % kVerWarps], s = sm.wz[lane % kVerWarps];
      int i = sm.wi[lane % kVerWarps];
      join(m, s, i, kVerWarps);
      if (C == 1 && lane == 0) sm.ex.m[part.parity][0] = m, sm.ex.z[part.parity][0] = s, sm.ex.idx[part.parity][0] = i;
      if (C > 1 && lane < C) {
        st_cluster32(&sm.ex.m[part.parity][rank], lane, __float_as_uint(m));
        st_cluster32(&sm.ex.z[part.parity][rank], lane, __float_as_uint(s));
        st_cluster32(&sm.ex.idx[part.parity][rank], lane, static_cast<uint32_t>(i));
      }
      __syncwarp();
    }
    if (C > 1) cluster_arrive();
    const int n_child = sm.n_child;
    if (n_child > 0) {   // the next row is most likely the first child's: its part goes to L2 meanwhile
      const char *next = reinterpret_cast<const char *>(p.logits + (static_cast<size_t>(t0) + sm.child[0]) * p.vocab) + 16ll * w0;
      for (int b = 128 * lane; b < 16 * (w1 - w0); b += 128 * 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(next + b));
    }
    // the row's maximum, sum and argmax from the CTAs' (every warp for itself)
    if (C > 1)
      cluster_wait();
    else
      __syncthreads();
    float m = sm.ex.m[part.parity][lane % C], Z = sm.ex.z[part.parity][lane % C];
    int top = sm.ex.idx[part.parity][lane % C];
    join(m, Z, top, C);
    part.parity ^= 1;
    if (m == -INFINITY) top = 0;   // no token has a chance: token 0
    // warp 0's lanes hold 32 children's values, from `first` on
    int c_tok = -1;
    float c_u = 2.f, c_l = -INFINITY, c_q = 0.f;
    auto load_children = [&](int first) {
      c_tok = -1;
      if (first + lane < n_child) {
        const int node = sm.child[first + lane];
        c_tok = sm.token[node];
        c_u = sm.u[node];
        c_l = sm.logit[node];
        c_q = sm.q[node];
      }
    };
    if (warp == 0) load_children(0);
    // the children's tests, by warp 0: every CTA comes to the same answer
    int taken = -1;
    int64_t total = 0, before = 0;
    int n_gone = 0, n_summed = 0;   // refused tokens (no draft probabilities): all, and those left out of `total`
    bool low = false;               // what is left weighs less than the reference
    const float *qrow = nullptr;
    WeightCtx ctx{m, 32.f * kh, 32.f * kl, d_max, 0.f, 0.f, 0.f, 0.f};
    bool have_sums = false;
    if (rank == 0 && threadIdx.x == 0) path[len - 1] = cur;
    if (greedy) {
      if (warp == 0) {
        int state = -1;
        for (int first = 0; first < n_child && state < 0; first += 32) {
          if (first > 0) load_children(first);
          const uint32_t hit = __ballot_sync(0xffffffffu, c_tok == top);
          if (hit) state = sm.child[first + __ffs(hit) - 1];
        }
        if (lane == 0) sm.state = state;
      }
      __syncthreads();
      taken = sm.state;
    } else if (m != -INFINITY && !p.probs) {
      // The row's fp32 sum serves as long as it can tell; then the weights of the
      // tokens left are summed, and the ones refused after that leave the sum
      // (warp 0's `left`).  The weights' reference is the row's maximum, or, when
      // that was refused and less than its weight is left, the maximum of what is
      // left: the sum is at least one reference, so the roundings to 2^-41 of it
      // are as small a part of the sum as in a whole row.
      int64_t left = 0;
      float gone = 0.f;
      for (int k = 0; k < n_child;) {
        if (warp == 0) {
          int state = kRefused;
          for (; k < n_child; ++k) {
            if (k % 32 == 0) load_children(k);
            const int tok = __shfl_sync(0xffffffffu, c_tok, k % 32);
            const float l = __shfl_sync(0xffffffffu, c_l, k % 32), u = __shfl_sync(0xffffffffu, c_u, k % 32);
            bool dup = tok < 0;   // an invalid token: passed over; one refused before: it has no chance
            for (int g = lane; g < n_gone; g += 32) dup |= sm.gone[g] == tok;
            if (__any_sync(0xffffffffu, dup)) continue;
            int64_t w = 0;
            if (have_sums) {
              if (left > 0 && left < kFixOne) state = kNearBorder;
              if (state != kRefused) break;
              const double e = fix_exp(l, ctx.m, kh, kl, sm.tab_fix, sm.tab_scaled);
              state = left > 0 && static_cast<double>(u) * (static_cast<double>(left) * 0x1p-41) < e ? kPassed : kRefused;
              if (state != kRefused) break;
              w = token_weight(ctx, l, false, 0.f);
              left -= w;
            } else {
              const float e = l == m ? 1.f : fmaxf(ex2_approx((l - m) * kh), 0.f);
              state = fast_test(u * (Z - gone), u * Z, e);
              if (state != kRefused) break;
              gone += e;
            }
            if (lane == 0) sm.gone[n_gone] = tok, sm.gone_w[n_gone] = w;
            __syncwarp();
            ++n_gone;
          }
          if (lane == 0) {
            sm.state = state == kPassed ? sm.child[k] : state == kNearBorder ? kNearBorder : -1;
            sm.n_gone = n_gone;
            sm.at = k;
            sm.low = n_gone > 0 && (have_sums ? left < kFixOne : Z - gone < 0.99f);
          }
        }
        __syncthreads();
        const int state = sm.state;
        n_gone = sm.n_gone;
        low = sm.low;
        k = sm.at;
        if (state != kNearBorder) {
          taken = state;
          break;
        }
        drop_gone(n_summed, n_gone);
        if (low) ctx.m = row_max(part);
        left = total = ctx.m == -INFINITY ? 0 : weight_sums<false>(part, ctx, nullptr, &before);
        n_summed = n_gone;
        have_sums = true;
      }
    } else if (m != -INFINITY) {
      const float *q = p.probs + (static_cast<size_t>(t0) + cur) * p.vocab;
      // a, c and the row's sum z (c in units of z) are warp 0's
      double a = 0.0, c = 1.0, zd = 0.0;
      bool exact = false;   // z is known to full accuracy
      for (int k = 0; k < n_child;) {
        if (warp == 0) {
          if (k > 0 && k % 32 == 0) load_children(k);
          if (lane == k % 32) {
            int state = kRefused;
            if (c_tok < 0) {
              state = kNoToken;   // (it was not drawn from q: p stays as it is)
            } else if (!exact) {
              const float uqz = c_u * (c_q * Z);
              state = fast_test(uqz, uqz, c_l == m ? 1.f : fmaxf(ex2_approx((c_l - m) * kh), 0.f));
            } else {   // both sides times z
              const double ex = fix_exp(c_l, m, kh, kl, sm.tab_fix, sm.tab_scaled);
              const double qz = static_cast<double>(c_q) * zd;
              if (static_cast<double>(c_u) * c * qz < ex - a * qz) state = kPassed;
            }
            sm.state = state;
          }
        }
        __syncthreads();
        const int state = sm.state;
        if (state == kPassed) {
          taken = sm.child[k];
          break;
        }
        if (state == kNoToken) {
          ++k;
          __syncthreads();   // sm.state has been read
          continue;
        }
        if (!exact) {   // the first refusal, or too close: the row's sum to full accuracy
          for (int b = 32 * lane; b < 8 * (w1 - w0); b += 32 * 32)   // its draft probabilities go to L2 meanwhile
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 8 * w0 + b));
          const int64_t z = weight_sums<false>(part, ctx, nullptr, &before);
          if (warp == 0) zd = static_cast<double>(z) * 0x1p-41;
          exact = true;
        }
        if (state == kNearBorder) continue;   // (the same child again)
        ++k;
        qrow = q;
        if (warp == 0) {
          a += c;
          const double az = a * zd;
          if (lane == 0) {
            const float h = static_cast<float>(az);
            sm.az_hi = h * 0x1p20f;
            sm.az_lo = static_cast<float>(az - static_cast<double>(h)) * 0x1p20f;
          }
        }
        __syncthreads();
        ctx.az_hi = sm.az_hi;
        ctx.az_lo = sm.az_lo;
        ctx.q_small = 513.f / ctx.az_hi;      // (in units of 2^-20, and one more)
        ctx.q_any = 1048577.f / ctx.az_hi;
        total = weight_sums<true>(part, ctx, qrow, &before);
        if (warp == 0) c = static_cast<double>(total) * 0x1p-41 / zd;
        have_sums = true;
      }
    }
    if (taken >= 0) {
      cur = taken;
      ++len;
      load_row(cur);
      __syncthreads();   // what this node left in shared memory is read before the next node writes there
      continue;
    }
    if (greedy || m == -INFINITY) {
      if (rank == 0 && threadIdx.x == 0) p.next_token[r] = top;
      break;
    }
    // none accepted: one token of what is left
    drop_gone(n_summed, n_gone);
    if (have_sums && !low) {
      for (int g = n_summed; g < n_gone; ++g) total -= sm.gone_w[g];   // (those refused since)
    } else {
      if (low) ctx.m = row_max(part);
      total = ctx.m == -INFINITY ? 0 : weight_sums<false>(part, ctx, nullptr, &before);
      n_summed = n_gone;
    }
    if (total == 0) {    // the refusals left nothing: p itself
      load_row(cur);
      cp_async_wait();
      qrow = nullptr;
      ctx = {m, 32.f * kh, 32.f * kl, d_max, 0.f, 0.f, 0.f, 0.f};
      total = weight_sums<false>(part, ctx, nullptr, &before);
      n_summed = n_gone;
    }
    if (threadIdx.x == 0) {
      const double uf = static_cast<double>(sm.u_final);
      const int64_t at = uf > 0.0 ? static_cast<int64_t>(fmin(uf, 1.0) * static_cast<double>(total)) : 0;
      sm.pick = min(at, total - 1);
    }
    __syncthreads();
    const int64_t pick = sm.pick;
    // the first token whose cumulative weight is above pick
    int64_t at = before, own = sm.ws[warp];
    for (int w = 0; w < warp; ++w) at += sm.ws[w];
    for (int g = n_summed; g < n_gone; ++g) {
      const int v = sm.gone[g] >> 3;
      at -= v < w0 ? sm.gone_w[g] : 0;
      own -= v >= w0 && v < w1 ? sm.gone_w[g] : 0;
    }
    if (at <= pick && pick < at + own) {
      // (this warp alone) its vectors' weights, in token order; then 8 lanes'
      // worth each, the vector, the token
      const int v0 = w0 + lane, nvec = w1 - w0;
      const float4 qa0 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int k = 0; k < part.nk_warp; ++k) {
        const int v = v0 + 32 * k;
        if (qrow) {
          float4 qa = make_float4(0.f, 0.f, 0.f, 0.f), qb = qa;
          if (k < nk) qa = load_q(qrow, 2 * v), qb = load_q(qrow, 2 * v + 1);
          sm.vec[32 * k + lane] = vector_weight<true>(ctx, x + k * kVerThreads, k < nk, qa, qb);
        } else {
          sm.vec[32 * k + lane] = vector_weight<false>(ctx, x + k * kVerThreads, k < nk, qa0, qa0);
        }
      }
      __syncwarp();
      const int per = (nvec + 31) / 32, lo = min(nvec, lane * per), hi = min(nvec, lo + per);
      int64_t sum = 0;
      for (int i = lo; i < hi; ++i) sum += sm.vec[i];
      int64_t inc = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
      }
      int64_t run = at + inc - sum;
      int i = lo;
      const bool mine = run <= pick && pick < run + sum;
      if (mine)
        while (pick >= run + sm.vec[i]) run += sm.vec[i++];
      const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
      const int vec = min(__shfl_sync(0xffffffffu, i, from), nvec - 1);
      run = __shfl_sync(0xffffffffu, run, from);
      // its 8 tokens, one a lane
      const int tok = 8 * (w0 + vec) + (lane & 7);
      const uint4 *hv = held + (vec >> 5) * kVerThreads + 32 * warp + (vec & 31);
      const int64_t w = token_weight(ctx, __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(hv)[lane & 7]), qrow != nullptr,
                                     qrow ? qrow[tok] : 0.f);
      inc = w;
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, off, 8);
        if ((lane & 7) >= off) inc += o;
      }
      if (lane < 8 && run + inc - w <= pick && pick < run + inc) p.next_token[r] = tok;
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
  // CTAs per request: enough that a CTA holds at most 20,480 of the row's
  // logits (four such fit an SM; with more than 16 times that in the vocabulary
  // 16 hold up to 32,768, three an SM), then as many as still fit the GPU
  // together, with at least 2,048 logits each; 16 (beyond what every GPU takes)
  // with at least 4,096: one chain of 5, vocabulary 128,256, 29.8 us against
  // 36.0 with 8; 16 trees of 24, vocabulary 50,264, 24.2 us against 22.6.
  int cluster = 1;
  while (cluster < kMaxCluster && a.vocab > cluster * 20480) cluster *= 2;
  while (cluster < kMaxCluster && static_cast<int64_t>(a.n_reqs) * cluster * 2 <= kVerPerSm * device_sm_count() &&
         a.vocab >= cluster * 2 * (cluster < 8 ? 2048 : 4096))
    cluster *= 2;
  p.cluster = cluster;
  static const FixExpTable table = fix_exp_table();
  p.tab = table;
  p.err = a.err;
  // a warp holds an eighth of the CTA's part, rounded up
  const int per_cta = (a.vocab / 8 + cluster - 1) / cluster;
  const int per_thread = ((per_cta + kVerWarps - 1) / kVerWarps + 31) / 32;
  const int smem = per_thread * kVerThreads * 16;
  const cudaError_t e = ensure_max_smem(reinterpret_cast<const void *>(verify_kernel), kMaxHeld * kVerThreads * 16);
  if (e != cudaSuccess) return e;
  if (cluster > 8) {
    const cudaError_t e16 = cudaFuncSetAttribute(reinterpret_cast<const void *>(verify_kernel),
                                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e16 != cudaSuccess) return e16;
  }
  if (per_thread > kMaxHeld) return cudaErrorInvalidValue;
  return launch_pdl(verify_kernel, dim3(a.n_reqs * cluster), dim3(kVerThreads), smem, st, cluster, p);
}

}  // namespace mb
