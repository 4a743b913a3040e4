// The latent cache of a layer whose heads' keys and values are linear maps of
// one vector per token, and attention against it in its absorbed form.
//
// A cached token is a row of rank + 64 numbers: its vector c (normalised) and
// one rotated key k_r that all heads share.  Head h with key rows W_uk,h [hd]
// [rank] and value rows W_uv,h [hd][rank] attends by
//
//   s_j = scale (q_nope . (W_uk,h c_j) + q_rope . k_r,j),  p = softmax(s),  o = sum_j p_j W_uv,h c_j
//
// and, the maps being linear,
//
//   s_j = scale ((W_uk,h^T q_nope) . c_j + q_rope . k_r,j),  o = W_uv,h (sum_j p_j c_j):
//
// keys and values are the cached rows themselves.  A single token reads each
// row once for all heads; a chunk of many does with the expanded form
// (mb_latent_prefill.cu) what this one does with (2 rank + 64) / (2 hd + 64)
// times the operations.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "mb_latent.h"
#include "mb_latent_dev.cuh"
#include "mb_launch.cuh"
#include "mb_ptx.cuh"
#include "mb_spec.h"

namespace mb {
namespace {

using namespace dev;

// ---------------------------------------------------------------- append
// One CTA per token: its vector normalised, its key and the queries' last 64
// numbers rotated (pairs (i, i + 32), frequency theta^(-2 i / 64)), vector and
// key into the token's slot.  The angles are taken as in rope_append_kernel: a
// split frequency and a two-constant reduction modulo 2 pi.  Every byte is read and
// written once; a head's 128 bytes go as eight 16-byte vectors, four lanes to a
// head.  64 tokens of 32 heads take 2.5 us: the latency of one load and a store.  2,144
// of 40 heads, rank 512, 27 MB, take 5.9 to 6.4 (4.2 to 4.5 TB/s): 40 registers a thread
// leave room for 6 CTAs on an SM, so they are three waves of a load, a barrier and a store.
constexpr int kAppendThreads = 256;
constexpr float kTwoPiHi = 6.28318548202514648f;         // fp32(2 pi)
constexpr float kTwoPiLo = -1.7484556000744893e-07f;     // 2 pi - kTwoPiHi
constexpr int kRopeHalf = kLatentRope / 2;

struct AppendParams {
  const __nv_bfloat16 *ckv, *q, *gain;
  __nv_bfloat16 *pool, *q_rope;
  const int32_t *tok_pos, *tok_slot;
  int64_t ld;
  int num_pages, H, q_row, hd, rank;
  float eps;
  int *err;
  float f_hi[kRopeHalf], f_lo[kRopeHalf];
};

__device__ __forceinline__ void rotate8(uint4 &a, uint4 &b, const float *cs, const float *sn) {
  uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a0 = bf16lo(x[e]), a1 = bf16hi(x[e]), b0 = bf16lo(y[e]), b1 = bf16hi(y[e]);
    const float c0 = cs[2 * e], c1 = cs[2 * e + 1], s0 = sn[2 * e], s1 = sn[2 * e + 1];
    x[e] = pack_bf16x2(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
    y[e] = pack_bf16x2(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
  }
  a = make_uint4(x[0], x[1], x[2], x[3]);
  b = make_uint4(y[0], y[1], y[2], y[3]);
}

__global__ void __launch_bounds__(kAppendThreads) latent_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float cs[kRopeHalf], sn[kRopeHalf], red[kAppendThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, part = tid & 3;
  // Every load goes out at once: nothing of the token's depends on its place
  // and position but where it goes and its angles.
  const int slot = p.tok_slot[t], pos = p.tok_pos[t];
  const uint4 *src = reinterpret_cast<const uint4 *>(p.ckv + t * p.ld);
  const int nv = p.rank / 8;   // at most 64: two warps hold the vector
  uint4 x = make_uint4(0, 0, 0, 0), g = x, ra = x, rb = x;
  if (tid < nv) {
    x = src[tid];
    g = reinterpret_cast<const uint4 *>(p.gain)[tid];
  }
  // rotated rows: the queries' heads, then (index H) the key; four lanes a row
  auto row_of = [&](int h) {
    return h < p.H ? reinterpret_cast<const uint4 *>(p.q + (static_cast<int64_t>(t) * p.H + h) * p.q_row + p.hd) : src + nv;
  };
  int h = tid >> 2;
  if (h <= p.H) {
    const uint4 *s = row_of(h);
    ra = s[part];
    rb = s[part + 4];
  }
  if (slot == -1) return;   // a row behind the batch's last token
  if (slot < 0 || slot >= p.num_pages * static_cast<int64_t>(kPage) || pos < 0 || pos > (1 << 24)) {
    if (tid == 0) atomicExch(p.err, kErrBounds);
    return;
  }
  uint4 *dst = reinterpret_cast<uint4 *>(p.pool + static_cast<int64_t>(slot) * (p.rank + kLatentRope));
  float ss = 0.f;
  const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) ss += bf16lo(xw[e]) * bf16lo(xw[e]) + bf16hi(xw[e]) * bf16hi(xw[e]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  if (lane == 0) red[warp] = ss;
  if (warp == 7) {   // the angles, by a warp that holds none of the vector
    const int i = lane;
    const float fp = static_cast<float>(pos);
    const float hi = fp * p.f_hi[i];
    const float lo = fmaf(fp, p.f_hi[i], -hi) + fp * p.f_lo[i];
    const float k = rintf(hi * 0.15915494309189535f);
    float r = fmaf(-k, kTwoPiHi, hi);
    r = fmaf(-k, kTwoPiLo, r) + lo;
    float sv, cv;
    sincosf(r, &sv, &cv);
    cs[i] = cv;
    sn[i] = sv;
  }
  __syncthreads();
  if (tid < nv) {
    const float inv = rsqrtf((red[0] + red[1]) / static_cast<float>(p.rank) + p.eps);
    const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(bf16lo(xw[e]) * inv * bf16lo(gw[e]), bf16hi(xw[e]) * inv * bf16hi(gw[e]));
    dst[tid] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  while (h <= p.H) {
    uint4 *d = h < p.H ? reinterpret_cast<uint4 *>(p.q_rope + (static_cast<int64_t>(t) * p.H + h) * kLatentRope) : dst + nv;
    rotate8(ra, rb, cs + 8 * part, sn + 8 * part);
    d[part] = ra;
    d[part + 4] = rb;
    h += kAppendThreads / 4;
    if (h <= p.H) {
      const uint4 *s = row_of(h);
      ra = s[part];
      rb = s[part + 4];
    }
  }
}

// ------------------------------------------------------------- the queries
// qc[t][h][r] = sum_d q[t][h][d] W_uk,h[d][r] for every head, rounded to bf16 for
// the product with the cached rows.  One CTA makes TOK tokens x 128 columns of
// one head on tcgen05, A and B wholly in shared memory, one barrier per 64 of
// hd; the result leaves by TMA from where A was.  Heads' weights are read once per
// TOK tokens: for few tokens they (and the launch) are the time, for many the
// stores.  All T rows are multiplied, whoever has them (96 decodes of 40 heads in a step of
// 2,144 tokens take 133 us, 86 by themselves).  64 tokens of 32 heads 2.3 us from the kernel
// before's end, 16 of 128 heads
// (16 MB of weights) 4, 256 of 128 heads (and 34 MB of results) 14.
constexpr int kQueryN = 128;

template <int HD, int TOK>
struct QueryCfg {
  static constexpr int KC = HD / 64;
  static constexpr int A_CHUNK = TOK * 128;
  static constexpr int B_PART = 64 * 128;            // 64 of hd x 64 columns
  static constexpr int OFF_B = KC * A_CHUNK;         // [64 columns][hd][128 B]: W_uk is stored [d][r]
  static constexpr int OFF_CTRL = OFF_B + KC * (kQueryN / 64) * B_PART;
  static constexpr int SMEM = OFF_CTRL + 256;
  static constexpr uint32_t IDESC = idesc_bf16(TOK, kQueryN, true);
};

// What becomes of a token's row: its unit's pieces (0: no request's token, 1: oc
// holds it), the CTA with the first one, and its place in the unit.
struct TokRec {
  int32_t pieces, first, place, pad;
};

struct QueryParams {
  TokRec *tok;
  int T;
  int *err;
};

template <int HD, int TOK>
__global__ void __launch_bounds__(128) latent_query_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmW,
                                                           const __grid_constant__ CUtensorMap tmO, const QueryParams p) {
  using C = QueryCfg<HD, TOK>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_CTRL), *done = full + C::KC;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5;
  const int n0 = blockIdx.x * kQueryN, h = blockIdx.y, t0 = blockIdx.z * TOK;
  if (smem_u32(smem) & 1023u) {   // the swizzled layouts need a 1024-aligned base
    pdl_wait();
    if (tid == 0) atomicExch(p.err, kErrBounds);
    return;
  }
  if (tid == 0) {
    for (int c = 0; c < C::KC; ++c) mbar_init(&full[c], 1);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmW);
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, kQueryN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The call's first kernel: every other one starts only after all of this one's
  // CTAs have passed this, so what earlier kernels of the stream wrote is there
  // for them without a wait of their own.
  pdl_wait();
  pdl_trigger();
  if (tid == 0) {
    const uint64_t a0 = sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t b0 = sdesc_sw128(smem_u32(smem + C::OFF_B), C::KC * C::B_PART, 1024);
    for (int c = 0; c < C::KC; ++c) {
      mbar_arrive_expect_tx(&full[c], C::A_CHUNK + (kQueryN / 64) * C::B_PART);
      for (int j = 0; j < kQueryN / 64; ++j)
        tma_load_2d(smem + C::OFF_B + (j * C::KC + c) * C::B_PART, &tmW, &full[c], n0 + 64 * j, h * 2 * HD + 64 * c);
      tma_load_3d(smem + c * C::A_CHUNK, &tmQ, &full[c], 64 * c, h, t0);
    }
    for (int c = 0; c < C::KC; ++c) {
      if (!mbar_wait(&full[c], 0, abort_flag, p.err, kErrWaitMma)) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16(tmem, a0 + ((c * C::A_CHUNK + kk * 32) >> 4), b0 + ((c * C::B_PART + kk * 2048) >> 4), C::IDESC,
                 (c > 0 || kk > 0) ? 1u : 0u);
    }
    mma_commit(done);
    if (*abort_flag) {
      const uint64_t t_start = globaltimer();
      for (int c = 0; c < C::KC; ++c) drain(&full[c], 0, t_start);
      drain(done, 0, t_start);
    }
  } else if (blockIdx.x == 0 && h == 0) {
    // (thread 0's row is thread 1's to clear)
    if (tid < TOK && t0 + tid < p.T) p.tok[t0 + tid].pieces = 0;
    if (tid == 1) p.tok[t0].pieces = 0;
  }
  __syncwarp();
  bool ok = mbar_wait(done, 0, abort_flag, p.err, kErrWaitEpilogue);
  ok = __all_sync(0xffffffffu, ok) && !*abort_flag;
  if (ok) {
    tc_fence_after();
    // (with 64 tokens a quarter's rows are its first 16 lanes)
    const int lane = tid & 31, row = TOK == 128 ? tid : 16 * warp + lane;
    uint8_t *dst = smem + (row >> 3) * 1024 + (row & 7) * 128;   // [64 columns][tokens][128 B], swizzled
#pragma unroll
    for (int cc = 0; cc < kQueryN / 32; ++cc) {
      float v[32];
      tmem_ld32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + cc * 32, v);
      if (TOK == 128 || lane < 16)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4 *>(dst + (cc >> 1) * (TOK * 128) + ((((cc & 1) * 4 + k) ^ (row & 7)) * 16)) =
              make_uint4(pack_bf16x2(v[8 * k], v[8 * k + 1]), pack_bf16x2(v[8 * k + 2], v[8 * k + 3]),
                         pack_bf16x2(v[8 * k + 4], v[8 * k + 5]), pack_bf16x2(v[8 * k + 6], v[8 * k + 7]));
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kQueryN);
    // (tokens behind T are none of the map's)
    if (ok && tid == 0) {
      for (int j = 0; j < kQueryN / 64; ++j) tma_store_3d(&tmO, smem + j * (TOK * 128), n0 + 64 * j, h, t0);
      asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
    }
  }
}

// ------------------------------------------------------ absorbed attention
// A unit is a tile of tokens of a request with up to 64 (token, head) rows; a
// CTA streams its keys in blocks of 64 rows of the cache, each copied once by
// TMA (a page's 16 rows per copy) and used twice, as keys and as values:
//
//   S   = Q K^T     M = 64 rows, N = 64 keys, K = rank + 64: a row of S is one
//                   thread's, so its maximum and sum need no exchange
//   O^T += V^T P^T  M = 128 numbers of the vectors, N = rows, K = 64 keys,
//                   rank / 128 times: with the vectors on the M side the
//                   accumulators of 64 rows take rank / 2 of the 512 columns of
//                   TMEM, not all of them
//
// With more than 64 heads two CTAs side by side take half the heads each and
// the same keys at the same time.  The probabilities are rounded to bf16 for
// their product with V, as everywhere in this library; logits, maxima, sums and
// accumulators are fp32.
//
// All units lie on one line, weighted by their blocks, and CTA w of W takes the
// w-th of W equal parts, whatever the lengths; every CTA works its part out from
// the device descriptor.  Units that a border cuts leave partials.
//
// What bounds it: HBM up to 64 heads (a block's 72 KB are 3,280 cycles of an SM's
// share, S and P V with N = 64 take 1,920), shared memory with 128 (S reads 144 KB of
// it, P V 96, the copies write 72: 2,500 cycles at 128 bytes; a block takes 2,900).
// Measured, the whole call replayed in a graph (head 128, rank 512): 96 ragged requests
// of 1,024 to 8,192 keys, 40 heads 87 us (this kernel by itself, under the profiler, 74 for
// 390 MB: 5.3 TB/s); 16 x 8,192 keys, 128 heads 66; 64 x 1,125 keys, 32 heads 35; one
// request 16 to 18.
constexpr int kMaxCtas = 160;       // CTAs of a launch at most; sizes the workspace
// Floats of a slot: whole lines only (with m and l behind each row the stores and
// loads of a row began 16 bytes off a sector).
__host__ __device__ constexpr int64_t part_floats(int64_t rank) { return 64 * rank + 128; }
constexpr int kBlk = 64;            // keys of a block
constexpr int kCostUnit = 3;        // a unit's start and end, in blocks (1 to 4: within 5 %; short units like more, long ones less)

struct AbsParams {
  __nv_bfloat16 *oc;             // [T][H][rank]: sum_j p_j c_j, an operand of the product with W_uv (so bf16)
  const uint8_t *pool;
  const int32_t *qo_indptr, *kv_len, *bt_indptr, *bt;
  int n_reqs, T, H, Hc, HT, NT, N, num_pages;   // heads of a tile, head tiles, tokens of a tile, padded rows
  float scale_log2;
  TokRec *tok;                   // [T]
  float *part;                   // [2 slots per CTA]: o of 64 rows [64][rank], their m and l [64][2]
  int *err;
};

// Queries of a tile and of a single token (vectors, then rotated), the parts of the
// cache's pages.
struct AbsMaps {
  CUtensorMap q[2][2], k[2];
};

template <int RANK>
struct AbsCfg {
  static constexpr int NC = RANK / 64 + 1;          // 64-wide chunks of a cached row
  static constexpr int DT = RANK / 128;             // tiles of 128 numbers of the vectors
  // A stage holds a block in two parts, each [page][8 rows of 2][chunk][8 rows][128 B]:
  // half of the vectors, and the other half with the rotated keys.  Parts are
  // loaded, waited for and given back by themselves, so S begins when the first has
  // come (16 requests at 8,192 keys, 128 heads: 67 us; 72 with whole blocks given back
  // page by page; 86 with five parts, whose copies of 4 KB come at 18 bytes a cycle).
  static constexpr int C0 = DT, C1 = DT + 1;        // chunks of the parts
  static constexpr int PART0 = C0 * kBlk * 128, PART1 = C1 * kBlk * 128;
  static constexpr int STAGE = PART0 + PART1, PAGE_BYTES = STAGE / 4;
  static constexpr int NST = RANK == 512 ? 2 : 4;
  static constexpr int Q_CHUNK = 64 * 128;
  static constexpr int NSEG = 4;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + NC * Q_CHUNK;
  static constexpr int OFF_P = OFF_K + NST * STAGE;
  static constexpr int OFF_CTRL = OFF_P + 64 * 128;
  static constexpr int SMEM = OFF_CTRL + 2048;
  static constexpr int THREADS = 256;               // TMA, 2 MMA issuers, one idle, 4 softmax warps
  static constexpr uint32_t IDESC_S = idesc_bf16(64, kBlk, false);
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t O_COL = 128;            // S buffers at 0 and 64, O^T tile dt at 128 + 64 dt
};

// A piece of a unit, as the producer tells it to the other roles.
struct AbsSeg {
  int32_t nb, j0;        // blocks [j0, j0 + nb); nb 0: no more pieces
  int32_t t0, toks;      // the tile's first row of q, its tokens
  int32_t first;         // the last key that the tile's first token sees
  int32_t kv, slot;      // partial slot, -1: the unit is whole
  int32_t odd;           // the first key behind `first` whose vector holds an infinity or a NaN
};

struct AbsReq {
  int t0, n, kv, b0, nkb, tiles;
  int64_t unit, cost;    // of one unit, of all
};

template <int RANK>
struct AbsCtrl {
  using C = AbsCfg<RANK>;
  uint64_t q_full, q_empty;
  uint64_t k_full[C::NST][2], k_empty[C::NST][2];
  uint64_t s_full[2], s_empty[2], p_full, pv_done;
  uint64_t seg_full[C::NSEG], seg_empty[C::NSEG];
  uint64_t done;
  AbsSeg seg[C::NSEG];
  int64_t wsum[C::THREADS / 32];
  int64_t start_base;
  AbsReq start;
  int32_t start_req;
  uint32_t tmem;
  int abort;
  alignas(16) float col[64];   // one number per row: the rescaling, the reciprocal of its sum
};

__device__ __forceinline__ AbsReq abs_req(const AbsParams &p, const ReqWords w, bool *bad) {
  AbsReq q;
  *bad = !req_ok(w, p.T);
  q.t0 = w.q0;
  q.n = *bad ? 0 : w.q1 - w.q0;
  q.kv = w.kv;
  q.b0 = w.b0;
  q.nkb = q.n ? (w.kv + kBlk - 1) / kBlk : 0;
  q.tiles = (q.n + p.NT - 1) / p.NT;
  q.unit = kCostUnit + q.nkb;
  q.cost = q.unit * q.tiles;
  return q;
}

template <int RANK>
__global__ void __launch_bounds__(AbsCfg<RANK>::THREADS, 1)
    latent_attention_kernel(const __grid_constant__ AbsMaps maps, const __grid_constant__ AbsParams p) {
  using C = AbsCfg<RANK>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem + C::OFF_Q, *sK = smem + C::OFF_K, *sP = smem + C::OFF_P;
  static_assert(sizeof(AbsCtrl<RANK>) <= 2048, "control area");
  static_assert(C::SMEM <= 232448, "shared memory");
  AbsCtrl<RANK> &ct = *reinterpret_cast<AbsCtrl<RANK> *>(smem + C::OFF_CTRL);
  volatile int *abort_flag = &ct.abort;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // (known uniform)
  const int ht = blockIdx.x % p.HT, cta = blockIdx.x / p.HT, W_max = gridDim.x / p.HT;
  if (smem_u32(smem) & 1023u) {   // the swizzled layouts need a 1024-aligned base
    pdl_wait();
    if (threadIdx.x == 0) atomicExch(p.err, kErrBounds);
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(&ct.q_full, 1);
    mbar_init(&ct.q_empty, 1);
    for (int s = 0; s < C::NST; ++s) {
      for (int g = 0; g < 2; ++g) {
        mbar_init(&ct.k_full[s][g], 1);
        mbar_init(&ct.k_empty[s][g], 1);
      }
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ct.s_full[b], 1);
      mbar_init(&ct.s_empty[b], 4);
    }
    mbar_init(&ct.p_full, 128);
    mbar_init(&ct.pv_done, 1);
    for (int s = 0; s < C::NSEG; ++s) {
      mbar_init(&ct.seg_full[s], 1);
      mbar_init(&ct.seg_empty[s], 6);   // the 2 MMA issuers and the 4 softmax warps
    }
    mbar_init(&ct.done, 2);
    ct.abort = 0;
    ct.start_req = -1;
    fence_mbar_init();
    for (int i = 0; i < 2; ++i) {
      prefetch_tmap(&maps.k[i]);
      for (int k = 0; k < 2; ++k) prefetch_tmap(&maps.q[i][k]);
    }
  }
  if (warp == 1) {
    tmem_alloc(&ct.tmem, C::TMEM_COLS);
    tmem_relinquish();
  }
  // Of what earlier kernels of the stream write, only the queries' products come
  // from this call's first kernel; this one is launched once that one has seen
  // all others finished, so the descriptor and the cache are there.  The producer
  // waits before it loads queries.  (That kernel has nearly always ended by then: its
  // CTAs leave no room for this one's.)

  // ---- this CTA's part of the line: [x0, x1) of `total`
  const int per = (p.n_reqs + C::THREADS - 1) / C::THREADS;
  const int r_lo = min(p.n_reqs, static_cast<int>(threadIdx.x) * per), r_hi = min(p.n_reqs, r_lo + per);
  int64_t mine = 0;
  AbsReq last{};
  for (int r = r_lo; r < r_hi; ++r) {
    bool bad;
    last = abs_req(p, load_req(p.qo_indptr, p.kv_len, p.bt_indptr, r), &bad);
    mine += last.cost;
    if (bad && blockIdx.x == 0) atomicExch(p.err, kErrBounds);
  }
  int64_t inc = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) ct.wsum[warp] = inc;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ct.tmem, 0);
  int64_t total = 0, pre = inc - mine;
#pragma unroll
  for (int w = 0; w < C::THREADS / 32; ++w) {
    if (w < warp) pre += ct.wsum[w];
    total += ct.wsum[w];
  }
  const int64_t W = min(total, static_cast<int64_t>(W_max));
  const bool active = cta < W;
  const int64_t x0 = active ? div64(total * cta, W) : 0, x1 = active ? div64(total * (cta + 1), W) : 0;
  if (active && pre <= x0 && x0 < pre + mine) {
    for (int r = r_lo; r < r_hi; ++r) {
      bool bad;
      if (per > 1) last = abs_req(p, load_req(p.qo_indptr, p.kv_len, p.bt_indptr, r), &bad);
      if (x0 < pre + last.cost) {
        ct.start_req = r;
        ct.start = last;
        ct.start_base = pre;
        break;
      }
      pre += last.cost;
    }
  }
  __syncthreads();

  if (!active) {
    pdl_wait();   // (no CTA ends, and with it the grid, before the kernel before)
    pdl_trigger();
  } else if (warp == 0) {
    // ------------------------------------------------ schedule, TMA producer
    int r = ct.start_req;
    bool bad;
    AbsReq q = ct.start;
    ReqWords nx{};
    if (r + 1 < p.n_reqs) nx = load_req(p.qo_indptr, p.kv_len, p.bt_indptr, r + 1);
    int u = static_cast<int>(div64(x0 - ct.start_base, q.unit));   // the unit that x0 lies in
    int64_t base = ct.start_base + u * q.unit;
    int kcnt = 0, sent = 0, nseg = 0, quse = 0;   // sent: parts of blocks
    const int pl = lane & 3;   // a lane's page of a block
    bool ok = true, waited = false;
    while (ok && base < x1) {
      auto cut = [&](int64_t x) {   // blocks of the unit that lie before x
        const int64_t d = x - base - kCostUnit;
        return d <= 0 ? 0 : static_cast<int>(min(static_cast<int64_t>(q.nkb), d));
      };
      auto owner = [&](int j) {     // the CTA whose part holds block j: the last w with total w / W <= its place
        return static_cast<int>(div64((base + kCostUnit + j + 1) * W - 1, total));
      };
      const int j0 = cut(x0), j1 = cut(x1);
      if (j1 > j0) {
        const int i0 = u * p.NT, toks = min(p.NT, q.n - i0);
        const int32_t *table = p.bt + q.b0;
        const int n_pages = (q.kv + kPage - 1) / kPage;
        // Page ids, a lane's, of the block to be sent and the one behind it, which is
        // on its way to L2 while it waits for a stage.  (96 requests at 1,024 to
        // 8,192 keys 88 us; 90, 93 and 109 with one, two and four more blocks under
        // way, 93 with none.)  They are looked at when they are used: their loads
        // take as long as a product.
        auto page_of = [&](int blk) { return blk < j1 && 4 * blk + pl < n_pages ? table[4 * blk + pl] : -1; };
        int cur = page_of(j0), nxt = page_of(j0 + 1);
        int j = j0;
        auto send = [&]() {   // block j: lane 4 g + k copies part g of page k
          const int np = min(4, n_pages - 4 * j), st = kcnt % C::NST, part = lane >> 2;
          int page = pl < np ? cur : 0;
          if (page < 0 || page >= p.num_pages) {
            atomicExch(p.err, kErrBounds);
            page = 0;
          }
          auto bytes = [&](int g) { return np * ((g ? C::PART1 : C::PART0) / 4); };
          auto copy = [&](int g) {
            tma_load_5d(sK + st * C::STAGE + g * C::PART0 + pl * ((g ? C::PART1 : C::PART0) / 4), &maps.k[g], &ct.k_full[st][g], 0, 0,
                        g * C::C0, 0, page);
          };
          if (kcnt < C::NST) {   // nothing to wait for
            if (lane < 2) mbar_arrive_expect_tx(&ct.k_full[st][lane], bytes(lane));
            __syncwarp();
            if (part < 2 && pl < np) copy(part);
            sent += 2;
          } else {
#pragma unroll 1
            for (int g = 0; g < 2; ++g, ++sent) {
              ok = __all_sync(0xffffffffu, mbar_wait(&ct.k_empty[st][g], ((kcnt / C::NST) & 1) ^ 1, abort_flag, p.err, kErrWaitProducer));
              if (!ok) return;
              if (lane == 0) mbar_arrive_expect_tx(&ct.k_full[st][g], bytes(g));
              __syncwarp();
              if (part == g && pl < np) copy(g);
            }
          }
          cur = nxt;
          if (++kcnt >= C::NST && lane < 4 && cur >= 0 && cur < p.num_pages)
            l2_prefetch(p.pool + cur * static_cast<int64_t>(C::PAGE_BYTES), C::PAGE_BYTES);
          nxt = page_of(++j + 1);
        };
        if (!waited) {
          pdl_wait();
          pdl_trigger();
          waited = true;
        }
        // the query tile, a copy per lane.  (Before the first keys: behind two blocks
        // of them it came 2 us later, as all CTAs' first blocks are more than HBM
        // brings in that time.)
        ok = __all_sync(0xffffffffu, mbar_wait(&ct.q_empty, (quse & 1) ^ 1, abort_flag, p.err, kErrWaitProducer));
        if (!ok) break;
        const int one = toks == 1;
        if (lane == 0) mbar_arrive_expect_tx(&ct.q_full, C::NC * p.Hc * (one ? 1 : p.NT) * 128);
        __syncwarp();
        if (lane < C::NC)
          tma_load_3d(sQ + lane * C::Q_CHUNK, &maps.q[one][lane == C::NC - 1], &ct.q_full, lane < C::NC - 1 ? lane * 64 : 0, ht * p.Hc, q.t0 + i0);
        ++quse;
        while (j < j1 && kcnt < C::NST) send();
        const int first = owner(0), last_w = owner(q.nkb - 1);
        // the piece's record for the other roles
        const int ss = nseg % C::NSEG;
        if (lane == 0) {
          ok = mbar_wait(&ct.seg_empty[ss], ((nseg / C::NSEG) & 1) ^ 1, abort_flag, p.err, kErrWaitProducer);
          if (ok) {
            AbsSeg &sg = ct.seg[ss];
            sg.nb = j1 - j0;
            sg.j0 = j0;
            sg.t0 = q.t0 + i0;
            sg.toks = toks;
            sg.first = q.kv - q.n + i0;
            sg.kv = q.kv;
            sg.slot = first == last_w ? -1 : 2 * static_cast<int>(blockIdx.x) + (cta == first ? 1 : 0);
            sg.odd = INT32_MAX;
            mbar_arrive(&ct.seg_full[ss]);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        ++nseg;
        if (cta == first && ht == 0)
          for (int i = lane; i < toks; i += 32) p.tok[q.t0 + i0 + i] = {last_w - first + 1, first, i, 0};
        while (ok && j < j1) send();
      }
      // the next unit on the line
      base += q.unit;
      if (++u == q.tiles) {
        u = 0;
        do {
          ++r;
          if (r >= p.n_reqs) break;
          q = abs_req(p, nx, &bad);
          if (r + 1 < p.n_reqs) nx = load_req(p.qo_indptr, p.kv_len, p.bt_indptr, r + 1);
        } while (q.n == 0);
        if (r >= p.n_reqs) break;
      }
    }
    if (!waited) pdl_wait();
    if (lane == 0) {
      if (ok) {
        const int ss = nseg % C::NSEG;
        if (mbar_wait(&ct.seg_empty[ss], ((nseg / C::NSEG) & 1) ^ 1, abort_flag, p.err, kErrWaitProducer)) {
          ct.seg[ss].nb = 0;
          mbar_arrive(&ct.seg_full[ss]);
        }
      }
      // after an abort, let copies in flight land before the CTA exits (bounded)
      if (!ok || *abort_flag) {
        const uint64_t t_start = globaltimer();
        for (int i = max(0, sent - 2 * C::NST); i < sent; ++i) drain(&ct.k_full[i / 2 % C::NST][i % 2], i / 2 / C::NST, t_start);
        if (quse > 0) drain(&ct.q_full, quse - 1, t_start);
      }
    }
  } else if (warp <= 2) {
    // --------------------------------------------------------- MMA issuers
    // Warp 1 issues S, a block ahead of the softmax (two buffers) and on into the
    // next piece, warp 2 the products with V: neither's commits and waits hold
    // up the other.  Each warp keeps the books, in step, and one elected lane issues
    // (the descriptors stay in uniform registers).
    auto wait = [&](uint64_t *bar, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, p.err, kErrWaitMma)) != 0;
    };
    const uint64_t kd0 = sdesc_sw128(smem_u32(sK), 16, C::C0 * 1024), kd1 = sdesc_sw128(smem_u32(sK + C::PART0), 16, C::C1 * 1024);
    const uint64_t qd0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t vd0 = sdesc_sw128(smem_u32(sK), 1024, C::C0 * 1024), vd1 = sdesc_sw128(smem_u32(sK + C::PART0), 1024, C::C1 * 1024);
    const uint64_t pd0 = sdesc_sw128(smem_u32(sP), 16, 1024);
    const uint32_t idesc_pv = idesc_bf16_ab(128, p.N, true, false);
    int nseg = 0, item = 0;
    bool ok = true;
    while (ok) {
      const int ss = nseg % C::NSEG;
      ok = wait(&ct.seg_full[ss], (nseg / C::NSEG) & 1);
      if (!ok) break;
      const int nb = __shfl_sync(0xffffffffu, ct.seg[ss].nb, 0);
      if (nb == 0) break;
      if (warp == 1) ok = wait(&ct.q_full, nseg & 1);
      for (int lb = 0; lb < nb && ok; ++lb, ++item) {
        const int st = item % C::NST;
        if (warp == 1) {
          ok = wait(&ct.s_empty[item & 1], ((item >> 1) & 1) ^ 1);
          const uint32_t d = tmem + 64 * (item & 1);
          const uint64_t at = static_cast<uint64_t>((st * C::STAGE) >> 4);
#pragma unroll
          for (int g = 0; g < 2; ++g) {   // the parts, as they come
            ok = ok && wait(&ct.k_full[st][g], (item / C::NST) & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t kd = (g ? kd1 : kd0) + at;
#pragma unroll
              for (int ch = 0; ch < (g ? C::C1 : C::C0); ++ch)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_bf16(d, qd0 + (((g * C::C0 + ch) * C::Q_CHUNK + kk * 32) >> 4), kd + ((ch * 1024 + kk * 32) >> 4), C::IDESC_S,
                           (g > 0 || ch > 0 || kk > 0) ? 1u : 0u);
              if (g == 1) {
                mma_commit(&ct.s_full[item & 1]);
                if (lb + 1 == nb) mma_commit(&ct.q_empty);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
        } else {
          ok = wait(&ct.p_full, item & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t at = static_cast<uint64_t>((st * C::STAGE) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int dt = 0; dt < C::DT; ++dt) {
              const int g = dt >= C::DT / 2, cc = g ? C::C1 : C::C0;   // the tile's part, and its chunks
              const uint64_t vd = (g ? vd1 : vd0) + at + (((2 * dt - g * C::C0) * 1024) >> 4);
#pragma unroll
              for (int ks = 0; ks < kBlk / 16; ++ks)   // 16 keys (a page) per MMA
                mma_bf16(tmem + C::O_COL + 64 * dt, vd + ((ks * 2 * cc * 1024) >> 4), pd0 + ((ks * 32) >> 4), idesc_pv,
                         (lb > 0 || ks > 0) ? 1u : 0u);
              if (dt % (C::DT / 2) == C::DT / 2 - 1) mma_commit(&ct.k_empty[st][g]);
            }
            mma_commit(&ct.pv_done);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      ++nseg;
      if (lane == 0) mbar_arrive(&ct.seg_empty[ss]);
    }
    // every MMA issued above has completed before TMEM is freed
    if (elect_one()) mma_commit(&ct.done);
    __syncwarp();
    drain(&ct.done, 0, globaltimer());
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------- softmax / epilogue
    const int qu = warp & 3;                     // TMEM lane quarter: rows 16 qu .. 16 qu + 15 of S in its first 16 lanes
    const int row = qu * 16 + (lane & 15);
    const int tid = (warp - 4) * 32 + lane;      // of the 128
    const uint32_t lane_base = static_cast<uint32_t>(qu * 32) << 16;
    constexpr float kRescaleAbove = 8.f;         // log2 units
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    const int row_tok = row / p.Hc, row_head = ht * p.Hc + row % p.Hc;
    int nseg = 0, item = 0;
    // The four warps meet in barriers, which have no limit: a warp whose wait
    // ran out goes on to the next one with `fail` set, and all leave together.
    bool fail = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (!fail) fail = !__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.err, kErrWaitSoftmax));
    };
    while (true) {
      const int ss = nseg % C::NSEG;
      wait(&ct.seg_full[ss], (nseg / C::NSEG) & 1);
      if (named_bar_or(1, 128, fail)) break;
      AbsSeg &sg = ct.seg[ss];
      const int nb = sg.nb;
      if (nb == 0) break;
      const int j0 = sg.j0, first = sg.first, kv = sg.kv;
      const bool live = lane < 16 && row_tok < sg.toks && row_head < p.H;
      const int limit = first + row_tok;          // the last key that the row sees
      float m_ref = -INFINITY, l = 0.f;
      bool stop = false;
      for (int lb = 0; lb < nb; ++lb, ++item) {
        const int key0 = kBlk * (j0 + lb);
        wait(&ct.s_full[item & 1], (item >> 1) & 1);
        float sv[64];
        float mx = -INFINITY;
        if (!fail) {
          tc_fence_after();
          tmem_ld64(tmem + lane_base + 64 * (item & 1), sv);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ct.s_empty[item & 1]);
          const int vis = limit - key0;
          if (vis < kBlk - 1)
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (e > vis) sv[e] = -INFINITY;
          float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
          for (int e = 0; e < 64; e += 8) {
            m0 = max3f(m0, sv[e], sv[e + 1]);
            m1 = max3f(m1, sv[e + 2], sv[e + 3]);
            m2 = max3f(m2, sv[e + 4], sv[e + 5]);
            m3 = max3f(m3, sv[e + 6], sv[e + 7]);
          }
          mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * p.scale_log2;
          if (!live) mx = -INFINITY;
          if (lb == 0) m_ref = mx;
        }
        // O^T holds a row as a column, in every warp's lanes: if a row rose
        // more than 2^8 above its reference, all four warps scale it
        const bool grow = mx > m_ref + kRescaleAbove;
        if (named_bar_or(1, 128, grow || fail)) {
          if (item > 0) wait(&ct.pv_done, (item - 1) & 1);   // O^T holds the blocks before
          if (named_bar_or(1, 128, fail)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const float alpha = grow ? ex2_approx(m_ref - mx) : 1.f;
          if (lane < 16) ct.col[row] = alpha;
          named_bar_sync(1, 128);
#pragma unroll 1
          for (int cc = 0; cc < C::DT * 64; cc += 32) {
            if ((cc & 63) >= p.N) continue;
            float v[32];
            tmem_ld32(tmem + lane_base + C::O_COL + cc, v);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] *= ct.col[(cc & 63) + k];
            tmem_st32(tmem + lane_base + C::O_COL + cc, v);
          }
          if (grow) {
            l *= alpha;
            m_ref = mx;
          }
        }
        const float negm = m_ref == -INFINITY ? 0.f : -m_ref;   // a row that has seen nothing yet
        uint32_t pk[32];
        float2 sum = make_float2(0.f, 0.f);
        probs<64>(sv, sc2, negm, pk, sum);
        l += sum.x + sum.y;
        if (item > 0) wait(&ct.pv_done, (item - 1) & 1);   // P of the block before is read
        if (live) {
          uint8_t *prow = sP + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4 *>(prow + ((k ^ (row & 7)) * 16)) = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        }
        if (key0 + kBlk - 1 > first && tid < kBlk) {
          // Keys that some row does not see: P is 0 there, but 0 times an
          // infinity or a NaN is not.  Rows past the request's last key hold
          // anything: zeroed.  So are those of the tile's own tokens with a value
          // that is not finite; the rows that see one become NaN at the end.
          const int key = key0 + tid;
          if (key > first) {
            uint8_t *stage = sK + (item % C::NST) * C::STAGE, *row0 = stage + (tid >> 3) * (C::C0 * 1024) + (tid & 7) * 128,
                    *row1 = stage + C::PART0 + (tid >> 3) * (C::C1 * 1024) + (tid & 7) * 128;
            if (wipe_row<C::DT>(row0, row1, key >= kv)) atomicMin(&sg.odd, key);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&ct.p_full);
      }
      if (stop) break;
      // ---- the piece is done: sum_j p_j c_j of its rows, or its partial
      wait(&ct.pv_done, (item - 1) & 1);
      if (named_bar_or(1, 128, fail)) break;
      tc_fence_after();
      // (the rows of a tile are one after another in oc as in a partial: more
      // than one token only if the tile has all heads)
      const int slot = sg.slot, rows = min(sg.toks * p.Hc, p.H - ht * p.Hc + (sg.toks - 1) * p.Hc);
      if (lane < 16) {
        if (live && sg.odd <= limit) l = NAN;
        ct.col[row] = 1.f / l;
        if (live && slot >= 0)
          *reinterpret_cast<float2 *>(p.part + slot * part_floats(RANK) + 64 * RANK + 2 * row) = make_float2(m_ref, l);
      }
      named_bar_sync(1, 128);
#pragma unroll 1
      for (int cc = 0; cc < C::DT * 64; cc += 32) {
        const int r0 = cc & 63, n = (cc >> 6) * 128 + qu * 32 + lane;   // rows from r0 on, number n of their vectors
        if (r0 >= rows) continue;
        float v[32];
        tmem_ld32(tmem + lane_base + C::O_COL + cc, v);
        if (slot < 0) {
          __nv_bfloat16 *dst = p.oc + (static_cast<int64_t>(sg.t0) * p.H + ht * p.Hc + r0) * RANK + n;
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 c = *reinterpret_cast<const float4 *>(ct.col + r0 + k);
            store_if(r0 + k < rows, dst + k * RANK, __float2bfloat16_rn(v[k] * c.x));
            store_if(r0 + k + 1 < rows, dst + (k + 1) * RANK, __float2bfloat16_rn(v[k + 1] * c.y));
            store_if(r0 + k + 2 < rows, dst + (k + 2) * RANK, __float2bfloat16_rn(v[k + 2] * c.z));
            store_if(r0 + k + 3 < rows, dst + (k + 3) * RANK, __float2bfloat16_rn(v[k + 3] * c.w));
          }
        } else {
          float *dst = p.part + slot * part_floats(RANK) + r0 * RANK + n;
#pragma unroll
          for (int k = 0; k < 32; ++k) store_if(r0 + k < rows, dst + k * RANK, v[k]);
        }
      }
      tc_fence_before();
      ++nseg;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ct.seg_empty[ss]);
    }
    tc_fence_before();
  }

  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ----------------------------------------------------------- cut units' rows
// oc[t][h] = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,  M = max_s m_s, for the
// tokens whose unit was cut.  A kernel of its own, with little shared memory:
// beside 200 KB of it L1 has room for so few lines on their way that bringing the
// pieces in within the next kernel took 5 to 14 us (3 here).  A warp takes a
// row; where there are few rows, and each may have a hundred pieces, the CTA's
// eight warps take every eighth piece of one.
template <int RANK, int WARPS>
__global__ void __launch_bounds__(256) latent_merge_kernel(const AbsParams p) {
  constexpr int PER = RANK / 128, AHEAD = 16 / PER;   // vectors of a lane; pieces in flight
  __shared__ float sh_acc[WARPS == 1 ? 1 : WARPS][WARPS == 1 ? 1 : RANK], sh_m[WARPS], sh_l[WARPS];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = WARPS == 1 ? 0 : warp;
  const int64_t slot = part_floats(RANK), rows = static_cast<int64_t>(p.T) * p.H;
  auto merge = [&](int64_t row, const TokRec rec) {
    const int pieces = rec.pieces, h = static_cast<int>(row % p.H);
    // (whole, or no request's; or, where requests of a bad descriptor overlap, the
    // words of two records)
    if (pieces <= 1 || (rec.first + pieces) * p.HT > kMaxCtas) return;
    // piece 0 in slot 2 x0 + 1, piece s > 0 in slot 2 (x0 + s HT)
    const int x0 = rec.first * p.HT + h / p.Hc;
    const int place = rec.place * p.Hc + h % p.Hc;
    const float *base = p.part + (2 * x0 + 1) * slot;
    auto src = [&](int s) { return base + (s == 0 ? 0 : (2 * s * p.HT - 1) * slot); };
    float2 ml[AHEAD];
    float4 v[AHEAD][PER];
    auto fetch = [&](int s0) {
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) {
        ml[s] = make_float2(-INFINITY, 0.f);
        if (s0 + s * WARPS < pieces) {
          ml[s] = *reinterpret_cast<const float2 *>(src(s0 + s * WARPS) + 64 * RANK + 2 * place);
#pragma unroll
          for (int k = 0; k < PER; ++k)
            v[s][k] = *reinterpret_cast<const float4 *>(src(s0 + s * WARPS) + place * RANK + 4 * lane + 128 * k);
        }
      }
    };
    fetch(share);
    float M = -INFINITY, L = 0.f;
    float4 acc[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = share; s0 < pieces; s0 += AHEAD * WARPS) {
      float top = M;
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) top = fmaxf(top, ml[s].x);
      const float old = M == -INFINITY ? 0.f : ex2_approx(M - top);
      // (a sum that is NaN says that the row saw one; a piece of which it saw
      // nothing has a sum of 0, and so has one with logits of minus infinity only)
      L = M == -INFINITY ? L : L * old;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        acc[k].x *= old;
        acc[k].y *= old;
        acc[k].z *= old;
        acc[k].w *= old;
      }
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) {
        const float w = ml[s].x == -INFINITY ? 0.f : ex2_approx(ml[s].x - top);
        L += ml[s].x == -INFINITY ? ml[s].y : w * ml[s].y;
        if (s0 + s * WARPS < pieces)   // (with a weight of 0 too: a vector that is not finite leaves NaN there)
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            acc[k].x = fmaf(w, v[s][k].x, acc[k].x);
            acc[k].y = fmaf(w, v[s][k].y, acc[k].y);
            acc[k].z = fmaf(w, v[s][k].z, acc[k].z);
            acc[k].w = fmaf(w, v[s][k].w, acc[k].w);
          }
      }
      M = top;
      if (s0 + AHEAD * WARPS < pieces) fetch(s0 + AHEAD * WARPS);
    }
    if (WARPS == 1) {
      const float inv = 1.f / L;
      uint2 *dst = reinterpret_cast<uint2 *>(p.oc + row * RANK + 4 * lane);
#pragma unroll
      for (int k = 0; k < PER; ++k)
        dst[32 * k] = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
      return;
    }
    // the warps' shares, two columns a thread
    if (lane == 0) sh_m[share] = M, sh_l[share] = L;
#pragma unroll
    for (int k = 0; k < PER; ++k) *reinterpret_cast<float4 *>(&sh_acc[share][4 * lane + 128 * k]) = acc[k];
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, sh_m[w]);
    float2 sum = make_float2(0.f, 0.f);
    L = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float a = sh_m[w] == -INFINITY ? 0.f : ex2_approx(sh_m[w] - top);
      L += sh_m[w] == -INFINITY ? sh_l[w] : a * sh_l[w];
      if (2 * threadIdx.x < RANK) {   // (a warp without pieces has zeros; as above, whatever the weight)
        const float2 x = *reinterpret_cast<const float2 *>(&sh_acc[w][2 * threadIdx.x]);
        sum.x = fmaf(a, x.x, sum.x);
        sum.y = fmaf(a, x.y, sum.y);
      }
    }
    if (2 * threadIdx.x < RANK)
      reinterpret_cast<uint32_t *>(p.oc + row * RANK)[threadIdx.x] = pack_bf16x2(sum.x / L, sum.y / L);
  };
  if (WARPS > 1) {   // (a CTA per row)
    if (blockIdx.x < rows) merge(blockIdx.x, p.tok[blockIdx.x / p.H]);
    return;
  }
  // the records of a warp's next 32 rows at once: most rows are whole
  const int64_t step = gridDim.x * 8;
  for (int64_t row0 = blockIdx.x * 8 + warp; row0 < rows; row0 += 32 * step) {
    const int64_t row = row0 + lane * step;
    TokRec rec = {0, 0, 0, 0};
    if (row < rows) rec = p.tok[row / p.H];
    for (uint32_t left = __ballot_sync(0xffffffffu, rec.pieces > 1); left; left &= left - 1) {
      const int i = __ffs(left) - 1;
      merge(row0 + i * step, {__shfl_sync(0xffffffffu, rec.pieces, i), __shfl_sync(0xffffffffu, rec.first, i),
                              __shfl_sync(0xffffffffu, rec.place, i), 0});
    }
  }
}

// ------------------------------------------------------------- the outputs
// o[t][h] = W_uv,h oc[t][h], K = rank, in one of two shapes:
//  * 32 or 64 tokens a CTA, D = W_uv (M = hd) times the tokens' rows (N), all of it in
//    shared memory; W_uv is loaded before the wait for the rows.  What bounds it is
//    latency: 3 us from the merge's end (the rows' copies 2), for 64 tokens as for 16.
//  * 128 tokens a CTA, D = the tokens' rows (M = 128) times W_uv^T (N = hd), in a ring of
//    64 of rank a stage, two CTAs an SM, so that one's loads and stores run beside the
//    other's products, and W_uv is read once per 128 tokens.
template <int HD, int RANK, int TR>
struct OutCfg {
  static constexpr bool TILE = TR == 128;           // the tokens on the M side
  static constexpr int KC = RANK / 64, NST = TILE ? (HD == 128 ? 3 : 4) : KC;
  static constexpr int W_CHUNK = HD * 128, STAGE = W_CHUNK + TR * 128;
  static constexpr int OFF_CTRL = NST * STAGE;
  static constexpr int SMEM = OFF_CTRL + 256;
  static constexpr int COLS = TILE ? HD : TR;       // of the accumulator
  static constexpr uint32_t IDESC = TILE ? idesc_bf16(128, HD, false) : idesc_bf16(HD, TR, false);
};

struct OutParams {
  const TokRec *tok;
  __nv_bfloat16 *o;
  int T, H;
  int *err;
};

template <int HD, int RANK, int TR>
__global__ void __launch_bounds__(128)
    latent_out_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const OutParams p) {
  using C = OutCfg<HD, RANK, TR>;
  extern __shared__ __align__(1024) uint8_t smem[];
  static_assert(C::SMEM <= 232448 && (2 * C::NST + 1) * 8 + 8 <= 256, "shared memory");
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_CTRL), *empty = full + C::NST, *done = empty + C::NST;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x, t0 = blockIdx.y * TR;
  auto load_w = [&](int c) {
    mbar_arrive_expect_tx(&full[c % C::NST], C::STAGE);
    tma_load_2d(smem + c % C::NST * C::STAGE, &tmW, &full[c % C::NST], 64 * c, (2 * h + 1) * HD);
  };
  auto load_x = [&](int c) { tma_load_3d(smem + c % C::NST * C::STAGE + C::W_CHUNK, &tmX, &full[c % C::NST], 64 * c, h, t0); };
  if (smem_u32(smem) & 1023u) {   // the swizzled layouts need a 1024-aligned base
    pdl_wait();
    if (tid == 0) atomicExch(p.err, kErrBounds);
    return;
  }
  if (tid == 0) {
    for (int c = 0; c < C::NST; ++c) {
      mbar_init(&full[c], 1);
      mbar_init(&empty[c], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int c = 0; c < C::NST; ++c) load_w(c);
    prefetch_tmap(&tmX);
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();   // the rows are the kernel before's
  pdl_trigger();
  if (tid == 0)
    for (int c = 0; c < C::NST; ++c) load_x(c);
  __syncwarp();
  // tokens that are a request's: the thread's own, or a bit for each of the tile's
  bool mine = false;
  uint32_t live[2] = {0, 0};
  if (C::TILE) mine = t0 + tid < p.T && p.tok[t0 + tid].pieces > 0;
  else
#pragma unroll
    for (int k = 0; k < TR / 32; ++k) {
      const int t = t0 + 32 * k + lane;
      live[k] = __ballot_sync(0xffffffffu, t < p.T && p.tok[t].pieces > 0);
    }
  if (tid == 0) {
    const uint64_t w0 = sdesc_sw128(smem_u32(smem), 16, 1024), x0 = sdesc_sw128(smem_u32(smem + C::W_CHUNK), 16, 1024);
    int sent = C::NST;
    bool ok = true;
#pragma unroll 1
    for (int c = 0; c < C::KC; ++c) {
      const int st = c % C::NST;
      ok = mbar_wait(&full[st], (c / C::NST) & 1, abort_flag, p.err, kErrWaitMma);
      if (!ok) break;
      tc_fence_after();
      const uint64_t w = w0 + static_cast<uint64_t>((st * C::STAGE) >> 4), x = x0 + static_cast<uint64_t>((st * C::STAGE) >> 4);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16(tmem, (C::TILE ? x : w) + ((kk * 32) >> 4), (C::TILE ? w : x) + ((kk * 32) >> 4), C::IDESC, (c > 0 || kk > 0) ? 1u : 0u);
      if (C::NST < C::KC) {
        mma_commit(&empty[st]);
        if (c > 0 && sent < C::KC) {   // the stage of the chunk before
          ok = mbar_wait(&empty[(c - 1) % C::NST], ((c - 1) / C::NST) & 1, abort_flag, p.err, kErrWaitProducer);
          if (!ok) break;
          load_w(sent);
          load_x(sent++);
        }
      }
    }
    mma_commit(done);
    if (!ok) {
      const uint64_t t_start = globaltimer();
      for (int c = sent - C::NST; c < sent; ++c) drain(&full[c % C::NST], c / C::NST, t_start);
      drain(done, 0, t_start);
    }
  }
  __syncthreads();
  bool ok = mbar_wait(done, 0, abort_flag, p.err, kErrWaitEpilogue);
  ok = __all_sync(0xffffffffu, ok) && !*abort_flag;
  if (ok) {
    tc_fence_after();
    // (with M = 64 a quarter's rows are its first 16 lanes)
    const int dim = HD == 128 ? warp * 32 + lane : warp * 16 + lane;
    const int64_t step = static_cast<int64_t>(p.H) * HD;
#pragma unroll
    for (int c0 = 0; c0 < C::COLS; c0 += 32) {
      float v[32];
      tmem_ld32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c0, v);
      if (C::TILE) {
        if (!mine) continue;
        uint32_t x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
        __nv_bfloat16 *dst = p.o + (t0 + tid) * step + h * HD + c0;
        store_out(dst, x);
        store_out(dst + 16, x + 8);
      } else if (HD == 128 || lane < 16) {
        __nv_bfloat16 *dst = p.o + (t0 + c0) * step + h * HD + dim;
#pragma unroll
        for (int k = 0; k < 32; ++k) store_if((live[(c0 / 32) & 1] >> k) & 1, dst + k * step, __float2bfloat16_rn(v[k]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <int HD, int TOK>
cudaError_t launch_query(const LatentArgs &a, void *qc, const QueryParams &p, cudaStream_t st) {
  using C = QueryCfg<HD, TOK>;
  static_assert(2 * TOK * 128 <= C::OFF_CTRL, "shared memory");
  CUtensorMap tq, tw, to;
  const uint64_t H = a.H, W = HD + kLatentRope, R = a.rank, T = a.T;
  const uint64_t dq[3] = {W, H, T}, sq[2] = {W * 2, W * 2 * H}, dc[3] = {R, H, T}, sc[2] = {R * 2, R * 2 * H};
  const uint32_t box[3] = {64, 1, TOK};
  cudaError_t e = encode_tmap(&tq, a.q, 3, dq, sq, box);
  if (e == cudaSuccess) e = encode_tmap(&to, qc, 3, dc, sc, box);
  if (e == cudaSuccess) e = encode_tmap_2d(&tw, a.w_kv, R, H * 2 * HD, R * 2, 64, 64);
  if (e == cudaSuccess) e = ensure_max_smem(reinterpret_cast<const void *>(latent_query_kernel<HD, TOK>), C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_query_kernel<HD, TOK>, dim3(a.rank / kQueryN, a.H, (a.T + TOK - 1) / TOK), dim3(128), C::SMEM, st, 1, tq, tw, to, p);
}

template <int HD>
cudaError_t launch_query(const LatentArgs &a, void *qc, const QueryParams &p, cudaStream_t st) {
  return a.T <= 64 ? launch_query<HD, 64>(a, qc, p, st) : launch_query<HD, 128>(a, qc, p, st);
}

template <int HD, int RANK, int TR>
cudaError_t launch_out(const LatentArgs &a, const void *oc, const OutParams &p, cudaStream_t st) {
  using C = OutCfg<HD, RANK, TR>;
  CUtensorMap tw, tx;
  const uint64_t H = a.H;
  const uint64_t dx[3] = {RANK, H, static_cast<uint64_t>(a.T)}, sx[2] = {RANK * 2, RANK * 2 * H};
  const uint32_t bx[3] = {64, 1, TR};
  cudaError_t e = encode_tmap_2d(&tw, a.w_kv, RANK, H * 2 * HD, RANK * 2, 64, HD);
  if (e == cudaSuccess) e = encode_tmap(&tx, oc, 3, dx, sx, bx);
  if (e == cudaSuccess) e = ensure_max_smem(reinterpret_cast<const void *>(latent_out_kernel<HD, RANK, TR>), C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_out_kernel<HD, RANK, TR>, dim3(a.H, (a.T + TR - 1) / TR), dim3(128), C::SMEM, st, 1, tw, tx, p);
}

// Tiles of 32 tokens while their CTAs fit the SMs at once (96 requests, 40 heads: the
// call takes 86.8 us, 88.7 with tiles of 64), of 64 while those do (64 requests of 500
// keys, 128 heads: 42.1 us, 47.0 with tiles of 32, 44.5 with 128), else of 128 (140
// requests of 300 keys, 128 heads: 58.3 us, 64.0 with 64).
template <int HD, int RANK>
cudaError_t launch_out(const LatentArgs &a, const void *oc, const OutParams &p, cudaStream_t st) {
  const int64_t sms = device_sm_count(), H = a.H;
  if (H * ((a.T + 31) / 32) <= sms) return launch_out<HD, RANK, 32>(a, oc, p, st);
  return H * ((a.T + 63) / 64) <= sms ? launch_out<HD, RANK, 64>(a, oc, p, st) : launch_out<HD, RANK, 128>(a, oc, p, st);
}

template <int RANK>
cudaError_t launch_attention(const LatentArgs &a, AbsParams &p, const void *qc, cudaStream_t st) {
  using C = AbsCfg<RANK>;
  const uint64_t H = a.H, T = a.T, R = RANK, W = RANK + kLatentRope;
  AbsMaps m;
  const uint64_t dq[3] = {R, H, T}, sq[2] = {R * 2, R * 2 * H};
  const uint64_t dr[3] = {kLatentRope, H, T}, sr[2] = {kLatentRope * 2, kLatentRope * 2 * H};
  const uint64_t dk[5] = {64, 8, C::NC, kPage / 8, static_cast<uint64_t>(a.num_pages)};
  const uint64_t sk[4] = {W * 2, 128, 8 * W * 2, kPage * W * 2};
  cudaError_t e = cudaSuccess;
  for (uint32_t i = 0; i < 2 && e == cudaSuccess; ++i) {   // (q: i = 1, a single token)
    const uint32_t bq[3] = {64, static_cast<uint32_t>(p.Hc), i ? 1u : static_cast<uint32_t>(p.NT)};
    const uint32_t bk[5] = {64, 8, static_cast<uint32_t>(i ? C::C1 : C::C0), kPage / 8, 1};
    e = encode_tmap(&m.q[i][0], qc, 3, dq, sq, bq);
    if (e == cudaSuccess) e = encode_tmap(&m.q[i][1], a.q_rope, 3, dr, sr, bq);
    if (e == cudaSuccess) e = encode_tmap_5d(&m.k[i], a.pool, dk, sk, bk);
  }
  if (e == cudaSuccess) e = ensure_max_smem(reinterpret_cast<const void *>(latent_attention_kernel<RANK>), C::SMEM);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(device_sm_count(), kMaxCtas) / p.HT * p.HT;
  e = launch_pdl(latent_attention_kernel<RANK>, dim3(ctas), dim3(C::THREADS), C::SMEM, st, 1, m, p);
  if (e != cudaSuccess) return e;
  // a CTA a row where all fit the SMs at once, two an SM (9 requests of drafts, 8 heads:
  // the call takes 23.3 us, 29.8 with a warp a row), else a warp (64 requests, 32 heads:
  // 34.5 us, 43.7 with a CTA a row)
  const int64_t rows = static_cast<int64_t>(a.T) * a.H, room = 2ll * device_sm_count();
  if (rows <= room) return launch_pdl(latent_merge_kernel<RANK, 8>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, st, 1, p);
  return launch_pdl(latent_merge_kernel<RANK, 1>, dim3(static_cast<unsigned>(std::min((rows + 7) / 8, room))), dim3(256), 0, st, 1, p);
}

}  // namespace

cudaError_t latent_append_run(const LatentAppendArgs &a, cudaStream_t st) {
  AppendParams p;
  p.ckv = static_cast<const __nv_bfloat16 *>(a.ckv);
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.gain = static_cast<const __nv_bfloat16 *>(a.gain);
  p.pool = static_cast<__nv_bfloat16 *>(a.pool);
  p.q_rope = static_cast<__nv_bfloat16 *>(a.q_rope);
  p.tok_pos = a.tok_pos;
  p.tok_slot = a.tok_slot;
  p.ld = a.ld;
  p.num_pages = a.num_pages;
  p.H = a.H;
  p.q_row = a.hd + kLatentRope;
  p.hd = a.hd;
  p.rank = a.rank;
  p.eps = a.eps;
  p.err = a.err;
  const double step = -std::log2(static_cast<double>(a.theta)) * 2 / kLatentRope;
  for (int i = 0; i < kRopeHalf; ++i) {
    const double f = std::exp2(i * step);   // (good to 2^-46 at any theta)
    p.f_hi[i] = static_cast<float>(f);
    p.f_lo[i] = static_cast<float>(f - static_cast<double>(p.f_hi[i]));
  }
  return launch_pdl(latent_append_kernel, dim3(a.T), dim3(kAppendThreads), 0, st, 1, p);
}

// q through W_uk [T][H][rank], sum_j p_j c_j [T][H][rank], the tokens' records, the partials
size_t latent_attention_workspace_bytes(int64_t T, int64_t H, int64_t rank) {
  return 2 * align256(static_cast<size_t>(T) * H * rank * 2) + align256(static_cast<size_t>(T) * sizeof(TokRec)) +
         static_cast<size_t>(2) * kMaxCtas * part_floats(rank) * sizeof(float);
}

cudaError_t latent_attention_run(const LatentArgs &a, cudaStream_t st) {
  uint8_t *w = static_cast<uint8_t *>(a.workspace);
  const size_t rows = align256(static_cast<size_t>(a.T) * a.H * a.rank * 2);
  __nv_bfloat16 *qc = reinterpret_cast<__nv_bfloat16 *>(w), *oc = reinterpret_cast<__nv_bfloat16 *>(w + rows);
  TokRec *tok = reinterpret_cast<TokRec *>(w + 2 * rows);
  AbsParams p;
  p.oc = oc;
  p.pool = static_cast<const uint8_t *>(a.pool);
  p.qo_indptr = a.qo_indptr;
  p.kv_len = a.kv_len;
  p.bt_indptr = a.bt_indptr;
  p.bt = a.bt;
  p.n_reqs = a.n_reqs;
  p.T = a.T;
  p.H = a.H;
  p.HT = (a.H + 63) / 64;
  p.Hc = (a.H + p.HT - 1) / p.HT;
  p.NT = 64 / p.Hc;
  p.N = (p.NT * p.Hc + 15) / 16 * 16;
  p.num_pages = a.num_pages;
  p.scale_log2 = a.scale * kLog2e;
  p.tok = tok;
  p.part = reinterpret_cast<float *>(w + 2 * rows + align256(static_cast<size_t>(a.T) * sizeof(TokRec)));
  p.err = a.err;
  const QueryParams qp = {tok, a.T, a.err};
  cudaError_t e = a.hd == 128 ? launch_query<128>(a, qc, qp, st) : launch_query<64>(a, qc, qp, st);
  if (e == cudaSuccess) e = a.rank == 512 ? launch_attention<512>(a, p, qc, st) : launch_attention<256>(a, p, qc, st);
  if (e != cudaSuccess) return e;
  const OutParams op = {tok, static_cast<__nv_bfloat16 *>(a.o), a.T, a.H, a.err};
  if (a.hd == 128) return a.rank == 512 ? launch_out<128, 512>(a, oc, op, st) : launch_out<128, 256>(a, oc, op, st);
  return a.rank == 512 ? launch_out<64, 512>(a, oc, op, st) : launch_out<64, 256>(a, oc, op, st);
}

}  // namespace mb
