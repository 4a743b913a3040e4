// Latent attention of prompt chunks, in the expanded form: a cached token's
// keys and values are made for every head from its vector, once, and its
// request's tokens attend to them causally,
//
//   K_h = C W_uk,h^T,  V_h = C W_uv,h^T   (C: the request's vectors, kv x rank)
//   o_i = sum_{j <= c + i} p_ij V_h,j,    p_i = softmax_j (scale (q_nope,i . K_h,j + q_rope,i . k_j))
//
// Making a key and a value costs 4 hd rank operations, attending to them
// 2 (2 hd + 64) for each token that does, against 2 (2 rank + 64) in the
// absorbed form: from hd rank / (rank - hd) tokens on this form does less, 171 for 128
// and 512, 85 for 64 and 256.  Measured at 8,192 keys it is the faster one from fewer:
// 40 heads of 128, rank 512, 64 tokens 121 us against 109, 96 tokens 113 against 132;
// 32 heads of 64, rank 256, 51 against 43 and 51 against 56.
//
// What bounds it: the tensor cores, and beside them the chain of product,
// softmax, product.  Keys and values of a head are 4 hd bytes a token, written once
// and read by every tile of queries.  Measured, replayed in a graph: 2,048 tokens at
// 8,192 keys, 40 heads of 128, rank 512 308 us, 1.50 PFLOP/s (expansion 57, attention
// 240); 512 tokens of 32 heads 28 us: three launches and the chain of two blocks.
//
// Two kernels, and a merge (per group of heads, if all heads' keys and values would
// take more than 512 MB):
//  * expand: 2 x 128 cached rows (8 pages a CTA, copied once by TMA) stay in shared
//    memory as the A operand of a CTA pair while the heads' weights stream past:
//    M = 256 keys, N = 2 hd (a head's key and value rows), K = rank.
//  * attention: a unit is 256 tokens of a request and one head, as two 128-row
//    query tiles that share the staged keys and values; S = Q K^T with K = hd +
//    64, softmax with one thread per row, O += P V with P in TMEM.  Two groups of
//    four softmax warps take turns, one per tile (with one tile: its even and its
//    odd blocks), so products run during the other group's softmax.
//  * merge: units cut by the schedule's borders, by log-sum-exp.
//
// The schedule: all units lie on one line, weighted by their blocks, and CTA w
// of W takes the w-th of W equal parts, whatever the lengths.  Warps of the
// expansion that have nothing else to do work it out from the device descriptor.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mb_latent.h"
#include "mb_latent_dev.cuh"
#include "mb_launch.cuh"
#include "mb_ptx.cuh"
#include "mb_spec.h"

namespace mb {
namespace {

using namespace dev;

constexpr int kMaxCtas = 160;      // CTAs of an attention launch at most; sizes the workspace
constexpr int kRecBytes = 8192, kPartsBytes = 20480;   // workspace: a record of 8 ints and a PrePart per CTA
constexpr int kBlk = 128;          // keys of a block
__host__ __device__ constexpr int64_t part_floats(int64_t hd) { return 256 * (hd + 2); }   // of a slot
// Keys and values of a group of heads at most (of one head, whatever it takes).
// Groups that fit L2 were slower: 2,048 tokens at 8,192 keys, 40 heads, took 413 us as
// one group of 168 MB, 448 as two, 517 as four (each starts and ends its kernels anew).
// 128 heads of 128, 2,048 tokens: at 8,064 keys, the last of one group, 1,000 us (1.30 of
// the operations' time), at 8,192, two groups of 64 heads, 1,019 (1.30).
constexpr int kGroupBytes = 512 << 20;
// The schedule's weights: a block of one query tile, a block of two, a unit's
// start and end, and the least a CTA takes (at least kCost2, so that no CTA
// between the first and the last of a unit is left without a block).
constexpr int kCost1 = 2, kCost2 = 3, kCostUnit = 5, kMinShare = 3;

struct PrePart;
struct PreParams {
  __nv_bfloat16 *kv;             // [heads of the group][rows][2 hd]: a head's keys and values
  __nv_bfloat16 *o;
  const __nv_bfloat16 *w_kv;
  const int32_t *qo_indptr, *kv_len, *bt_indptr, *bt;
  int n_reqs, T, H, h0, HG, num_pages;   // heads h0 .. h0 + HG - 1
  int cap_blocks;                // blocks of 128 rows that kv has room for
  float scale_log2;
  int32_t *rec;
  PrePart *parts;                // of the attention kernel's CTAs
  int ctas;
  float *part;                   // [2 slots per CTA]: o of 256 rows [hd][256], their m and l [256][2]
  int *err;
};

// A request's blocks of keys (none if it has no tokens, or breaks a rule).
__device__ __forceinline__ int key_blocks(const ReqWords &w, int T, bool *bad) {
  *bad = !req_ok(w, T);
  return *bad || w.q1 == w.q0 ? 0 : (w.kv + kBlk - 1) / kBlk;
}

// Sums over the threads of WARPS warps (named barrier BAR): this thread's exclusive
// prefix, and the total.
template <int WARPS, int BAR>
__device__ __forceinline__ int64_t warps_scan(int64_t mine, int warp, int64_t *sums, int64_t *total) {
  const int lane = threadIdx.x & 31;
  int64_t inc = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) sums[warp] = inc;
  named_bar_sync(BAR, 32 * WARPS);
  int64_t pre = inc - mine, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) pre += sums[w];
    all += sums[w];
  }
  *total = all;
  return pre;
}

// ------------------------------------------------------------ the schedule
struct PreReq {
  int t0, n, c, row_blk;   // first row of q, tokens, cached tokens, first block of the workspace
  int full, rem, a;        // units of 256 rows, rows of the last one if it is smaller, blocks of the cached tokens
  int64_t head;            // cost of one head
};

// Cost of the first u units of 256 rows of a request and head: unit k has a +
// 2 (k + 1) blocks.
__device__ __forceinline__ int64_t units_cost(int a, int64_t u) {
  return u * (kCostUnit + static_cast<int64_t>(kCost2) * a) + kCost2 * u * (u + 1);
}
__device__ __forceinline__ int tail_blocks(const PreReq &q) { return (q.c + q.n + kBlk - 1) / kBlk; }

__device__ __forceinline__ PreReq pre_req(const PreParams &p, const ReqWords &w, int64_t row_blk) {
  PreReq q;
  bool bad;
  const int blocks = key_blocks(w, p.T, &bad);
  q.t0 = w.q0;
  q.n = blocks > 0 && row_blk + blocks <= p.cap_blocks ? w.q1 - w.q0 : 0;
  q.c = w.kv - q.n;
  q.row_blk = static_cast<int>(row_blk);
  q.full = q.n / 256;
  q.rem = q.n % 256;
  q.a = (q.c + kBlk - 1) / kBlk;
  q.head = q.n == 0 ? 0 : units_cost(q.a, q.full) + (q.rem ? kCostUnit + (q.rem > 128 ? kCost2 : kCost1) * static_cast<int64_t>(tail_blocks(q)) : 0);
  return q;
}

// Where a CTA's part of the line begins: the request, head of the group and unit, and
// the unit's place on the line.
struct __align__(16) PrePart {
  int64_t total, base, x0, x1;   // of the line; the unit's; the part
  int32_t req, hg, u;            // req -1: the CTA has no part
  PreReq q;
};

// Works out where the parts w0, w0 + step, ... of W_max begin: by 128 threads (warps
// from `warp0` on), each for the parts that begin in its requests.  sums: 8 numbers.
__device__ __forceinline__ void line_parts(const PreParams &p, PrePart *parts, int W_max, int w0, int step, int warp0, int64_t *sums) {
  const int tid = threadIdx.x - 32 * warp0, per = (p.n_reqs + 127) / 128;
  const int r_lo = min(p.n_reqs, tid * per), r_hi = min(p.n_reqs, r_lo + per);
  bool bad;
  int64_t mine = 0, total;
  for (int r = r_lo; r < r_hi; ++r) mine += key_blocks(load_req(p.qo_indptr, p.kv_len, p.bt_indptr, r), p.T, &bad);
  const int64_t blk0 = warps_scan<4, 1>(mine, tid >> 5, sums, &total);
  int64_t at = blk0;
  mine = 0;
  for (int r = r_lo; r < r_hi; ++r) {
    const ReqWords w = load_req(p.qo_indptr, p.kv_len, p.bt_indptr, r);
    mine += pre_req(p, w, at).head * p.HG;
    at += key_blocks(w, p.T, &bad);
  }
  const int64_t pre = warps_scan<4, 1>(mine, tid >> 5, sums + 4, &total);
  const int64_t W = min(max(total / kMinShare, static_cast<int64_t>(total > 0)), static_cast<int64_t>(W_max));
  for (int w = w0; w < W_max; w += step) {
    if (w >= W) {
      if (tid == 0) parts[w].req = -1;
      continue;
    }
    PrePart o;
    o.total = total;
    o.x0 = div64(total * w, W);
    o.x1 = div64(total * (w + 1), W);
    if (o.x0 < pre || o.x0 >= pre + mine) continue;
    o.base = pre;
    o.req = r_lo;
    at = blk0;
    for (;; ++o.req) {
      const ReqWords q = load_req(p.qo_indptr, p.kv_len, p.bt_indptr, o.req);
      o.q = pre_req(p, q, at);
      if (o.x0 < o.base + o.q.head * p.HG) break;
      o.base += o.q.head * p.HG;
      at += key_blocks(q, p.T, &bad);
    }
    o.hg = static_cast<int>(div64(o.x0 - o.base, o.q.head));
    o.base += o.hg * o.q.head;
    int lo = 0, hi = o.q.full + (o.q.rem ? 1 : 0);   // the unit that x0 lies in: the last one that does not begin behind it
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (units_cost(o.q.a, mid) <= o.x0 - o.base) lo = mid;
      else hi = mid;
    }
    o.u = lo;
    o.base += units_cost(o.q.a, lo);
    parts[w] = o;
  }
}

// ------------------------------------------------------------------ expand
// Over pairs of CTAs (cta_group::2): each has its own 128 cached rows as its half
// of A and of the accumulators, and half of a head's weights as its half of B, so
// a CTA takes in 32 bytes of weights a cycle instead of 64 (a CTA by itself took
// three times as long: two stages of 32 KB did not cover a load's latency).  Four
// more warps meanwhile work out where the parts of the next kernel's CTAs begin.
// An item, 2 x 128 keys and a head of 128 at rank 512, takes 2.7 us (2.1 by the
// products' cycles; 2.5 without its loads).
template <int HD, int RANK>
struct ExpCfg {
  static constexpr int NC = RANK / 64 + 1;
  static constexpr int ATOM = NC * 1024;
  static constexpr int PAGE_BYTES = 2 * ATOM;
  static constexpr int A_BYTES = (kBlk / 8) * ATOM;
  static constexpr int N = 2 * HD;
  static constexpr int B_STAGE = HD * 128;            // this CTA's half of the head's rows, 64 of rank
  static constexpr int KC = RANK / 64;
  static constexpr int NB = (HD == 128 ? 1 : 2) * (RANK == 512 ? 5 : 8);
  static constexpr int OFF_B = A_BYTES;
  static constexpr int OFF_CTRL = OFF_B + NB * B_STAGE;
  static constexpr int SMEM = OFF_CTRL + 512;
  static constexpr int WARPS = 6, THREADS = 320;      // TMA, MMA, 4 epilogue warps; and 4 for the schedule
  static constexpr uint32_t IDESC = idesc_bf16(256, N, false);
};

template <int HD, int RANK>
struct ExpCtrl {
  using C = ExpCfg<HD, RANK>;
  uint64_t a_full, a_peer, a_empty;   // this CTA's rows; the other's (in rank 0); both CTAs' products with them done
  uint64_t b_full[C::NB], b_empty[C::NB], t_full[2], t_empty[2], done;   // b_full, t_empty: rank 0's count for both
  int64_t sums[C::WARPS], line_sums[8];
  int64_t start_base;
  int32_t start_req;
  uint32_t tmem;
  int abort;
};

// The pair's form of a 5D tile load: counted on an mbarrier of either CTA.
__device__ __forceinline__ void tma_load_5d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int32_t x0, int32_t x4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %4, %4, %5}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(x0), "r"(0), "r"(x4)
      : "memory");
}

// 64 fp32 columns of 16 TMEM lanes (16x256b shape, x8), waited on before returning:
// thread t gets columns 8 i + 2 (t % 4) and the next one of lane t / 4 in v[0][2 i]
// and v[0][2 i + 1], of lane t / 4 + 8 in v[1].
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float (&v)[2][16]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k >> 1][2 * i + (k & 1)] = __uint_as_float(r[4 * i + k]);
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(smem_u32(src)),
               "r"(x), "r"(y)
               : "memory");
}

template <int HD, int RANK>
__global__ void __launch_bounds__(ExpCfg<HD, RANK>::THREADS, 1)
    latent_expand_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ CUtensorMap tmR, const __grid_constant__ PreParams p) {
  using C = ExpCfg<HD, RANK>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sA = smem, *sB = smem + C::OFF_B;
  static_assert(sizeof(ExpCtrl<HD, RANK>) <= 512 && C::SMEM <= 232448, "shared memory");
  ExpCtrl<HD, RANK> &ct = *reinterpret_cast<ExpCtrl<HD, RANK> *>(smem + C::OFF_CTRL);
  volatile int *abort_flag = &ct.abort;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // (known uniform)
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (smem_u32(smem) & 1023u) {   // the swizzled layouts need a 1024-aligned base (the same in both CTAs)
    pdl_wait();
    if (threadIdx.x == 0) {
      atomicExch(p.err, kErrBounds);
      for (int w = blockIdx.x; w < p.ctas; w += gridDim.x) p.parts[w].req = -1;
    }
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(&ct.a_full, 1);
    mbar_init(&ct.a_peer, 1);
    mbar_init(&ct.a_empty, 1);
    for (int s = 0; s < C::NB; ++s) {
      mbar_init(&ct.b_full[s], 1);
      mbar_init(&ct.b_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ct.t_full[b], 1);
      mbar_init(&ct.t_empty[b], 8);   // the epilogue warps of both CTAs
    }
    mbar_init(&ct.done, 1);
    ct.abort = 0;
    ct.start_req = -1;
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmR);
  }
  if (warp == 1) {
    tmem_alloc_pair(&ct.tmem, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // (both CTAs' barriers are set up, and TMEM's address is there)
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ct.tmem, 0);
  pdl_wait();   // descriptor, cache, weights and workspace belong to earlier kernels of the stream
  pdl_trigger();
  if (threadIdx.x == 32 * C::WARPS) {
    // The group's weights on their way to L2, a part by each CTA: all pairs ask
    // for the same chunk at about the same time, and each would wait for HBM.
    const uint32_t lines = static_cast<uint32_t>(p.HG) * (2 * HD * RANK * 2 / 128), part = (lines + gridDim.x - 1) / gridDim.x;
    const uint32_t from = part * blockIdx.x;
    if (from < lines)
      l2_prefetch(reinterpret_cast<const uint8_t *>(p.w_kv + static_cast<int64_t>(p.h0) * 2 * HD * RANK) + from * 128ll,
                  min(part, lines - from) * 128);
  }

  // ---- this pair's items: (two blocks of 128 keys, head), heads fastest
  constexpr int SCAN = 32 * C::WARPS;
  const int per = (p.n_reqs + SCAN - 1) / SCAN;
  const int r_lo = warp < C::WARPS ? min(p.n_reqs, static_cast<int>(threadIdx.x) * per) : 0;
  const int r_hi = warp < C::WARPS ? min(p.n_reqs, r_lo + per) : 0;
  int64_t mine = 0, total = 0, pre = 0;
  for (int r = r_lo; r < r_hi; ++r) {
    bool bad;
    mine += key_blocks(load_req(p.qo_indptr, p.kv_len, p.bt_indptr, r), p.T, &bad);
    if (bad && blockIdx.x == 0) atomicExch(p.err, kErrBounds);
  }
  if (warp < C::WARPS) pre = warps_scan<C::WARPS, 2>(mine, warp, ct.sums, &total);
  if (total > p.cap_blocks) {
    // the caller's room is too small for the requests behind: they are left alone
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicExch(p.err, kErrBounds);
    total = p.cap_blocks;
  }
  const int64_t items = (total + 1) / 2 * p.HG, W = min(static_cast<int64_t>(pairs), items);
  const bool active = pair < W;
  const int64_t x0 = active ? div64(items * pair, W) : 0, x1 = active ? div64(items * (pair + 1), W) : 0;
  const int64_t p0 = active ? div64(x0, p.HG) : 0;   // the first pair of blocks
  const int64_t b0 = min(2 * p0 + rank, total - 1);  // this CTA's first block (none: a stand-in)
  if (active && pre <= b0 && b0 < pre + mine) {
    for (int r = r_lo; r < r_hi; ++r) {
      bool bad;
      const int b = key_blocks(load_req(p.qo_indptr, p.kv_len, p.bt_indptr, r), p.T, &bad);
      if (b0 < pre + b) {
        ct.start_req = r;
        ct.start_base = pre;
        break;
      }
      pre += b;
    }
  }
  if (warp < C::WARPS) named_bar_sync(2, SCAN);
  // Walks this CTA's blocks: the request of a block and where it starts.
  struct Walk {
    int r;
    int64_t base;   // the request's first block
    ReqWords w;
    int blocks;
  };
  auto start = [&]() {
    Walk k;
    bool bad;
    k.r = ct.start_req;
    k.base = ct.start_base;
    k.w = load_req(p.qo_indptr, p.kv_len, p.bt_indptr, k.r);
    k.blocks = key_blocks(k.w, p.T, &bad);
    return k;
  };
  auto reach = [&](Walk &k, int64_t blk) {
    bool bad;
    while (blk >= k.base + k.blocks && k.r + 1 < p.n_reqs) {
      k.base += k.blocks;
      k.w = load_req(p.qo_indptr, p.kv_len, p.bt_indptr, ++k.r);
      k.blocks = key_blocks(k.w, p.T, &bad);
    }
  };
  const int hg0 = static_cast<int>(x0 - p0 * p.HG);

  if (warp >= C::WARPS) {
    line_parts(p, p.parts, p.ctas, blockIdx.x, gridDim.x, C::WARPS, ct.line_sums);
  } else if (!active) {
  } else if (warp == 0) {
    // -------------------------------------------------------- TMA producer
    Walk k = start();
    int ause = 0, bcnt = 0;
    bool ok = true;
    int64_t blk = 2 * p0 + rank;
    int hg = hg0;
    const uint32_t peer_bar = mapa_shared(smem_u32(&ct.a_peer), 0);
    for (int64_t i = x0; i < x1 && ok; ++i) {
      const bool have = blk < total;   // (the last pair of blocks may be one)
      if (i == x0 || hg == 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ct.a_empty, (ause & 1) ^ 1, abort_flag, p.err, kErrWaitProducer));
        if (!ok) break;
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the keys' copies below have left the stage
        __syncwarp();
        if (have) {
          reach(k, blk);
          const int j = static_cast<int>(blk - k.base), n_pages = (k.w.kv + kPage - 1) / kPage, np = min(8, n_pages - 8 * j);
          int page = lane < np ? p.bt[k.w.b0 + 8 * j + lane] : 0;
          if (lane < np && (page < 0 || page >= p.num_pages)) {
            atomicExch(p.err, kErrBounds);
            page = 0;
          }
          if (lane == 0) mbar_arrive_expect_tx(&ct.a_full, np * C::PAGE_BYTES);
          __syncwarp();
          if (lane < np) tma_load_5d(sA + lane * C::PAGE_BYTES, &tmK, &ct.a_full, 0, 0, 0, 0, page);
        } else if (lane == 0) {
          mbar_arrive(&ct.a_full);
        }
        ++ause;
      }
      bool told = rank == 0 || (i > x0 && hg != 0);   // rank 0 knows that this CTA's rows are there
      for (int c = 0; c < C::KC && ok; ++c, ++bcnt) {
        const int st = bcnt % C::NB;
        if (lane == 0) {
          ok = mbar_wait(&ct.b_empty[st], ((bcnt / C::NB) & 1) ^ 1, abort_flag, p.err, kErrWaitProducer);
          if (ok) {
            if (rank == 0) mbar_arrive_expect_tx(&ct.b_full[st], 2 * C::B_STAGE);
            tma_load_5d_pair(sB + st * C::B_STAGE, &tmW, mapa_shared(smem_u32(&ct.b_full[st]), 0), 64 * c,
                             ((p.h0 + hg) * 2 + static_cast<int>(rank)) * (HD / 64));
          }
          // (after the first weights, which go out while the rows are on their way)
          if (ok && !told && (c == C::NB - 1 || c == C::KC - 1)) {
            ok = mbar_wait(&ct.a_full, (ause - 1) & 1, abort_flag, p.err, kErrWaitProducer);
            if (ok) mbar_arrive_remote(peer_bar);
            told = true;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
      }
      if (ok && have && p.h0 + hg == 0) {
        // the rotated keys, once per call, as one row of 64 per token (what lies
        // behind the request's last key is never attended to)
        ok = __all_sync(0xffffffffu, mbar_wait(&ct.a_full, (ause - 1) & 1, abort_flag, p.err, kErrWaitProducer));
        if (ok && lane < kBlk / 8) tma_store_2d(&tmR, sA + lane * C::ATOM + C::KC * 1024, 0, static_cast<int>(blk) * kBlk + 8 * lane);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      if (++hg == p.HG) {
        hg = 0;
        blk += 2;
      }
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok || *abort_flag) {   // let copies in flight land before the CTA exits (bounded)
      const uint64_t t_start = globaltimer();
      if (lane == 0) {
        if (rank == 0)
          for (int b = max(0, bcnt - C::NB); b < bcnt; ++b) drain(&ct.b_full[b % C::NB], b / C::NB, t_start);
        else
          while (bcnt > 0 && globaltimer() - t_start < kWaitLimitNs / 100) {   // (its weights count in rank 0: 20 ms)
          }
        if (ause > 0) drain(&ct.a_full, ause - 1, t_start);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // (the warp keeps the books, in step, and one elected lane issues: the
    // descriptors stay in uniform registers)
    if (rank == 0) {
      const uint64_t ad0 = sdesc_sw128(smem_u32(sA), 16, C::ATOM);
      const uint64_t bd0 = sdesc_sw128(smem_u32(sB), 16, 1024);
      auto wait = [&](uint64_t *bar, uint32_t par) {
        return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, p.err, kErrWaitMma)) != 0;
      };
      int ause = 0, bcnt = 0, acc = 0, hg = hg0;
      bool ok = true;
      for (int64_t i = x0; i < x1 && ok; ++i, ++acc) {
        if (i == x0 || hg == 0) {
          ok = wait(&ct.a_full, ause & 1) && wait(&ct.a_peer, ause & 1);
          ++ause;
        }
        ok = ok && wait(&ct.t_empty[acc & 1], ((acc >> 1) & 1) ^ 1);
        const bool last = ++hg == p.HG;
        if (last) hg = 0;
        const uint32_t d = tmem + 256 * (acc & 1);
#pragma unroll
        for (int c = 0; c < C::KC; ++c, ++bcnt) {
          const int st = bcnt % C::NB;
          ok = ok && wait(&ct.b_full[st], (bcnt / C::NB) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bd = bd0 + static_cast<uint64_t>((st * C::B_STAGE) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_pair(d, ad0 + ((c * 1024 + kk * 32) >> 4), bd + ((kk * 32) >> 4), C::IDESC, (c > 0 || kk > 0) ? 1u : 0u);
            mma_commit_pair(&ct.b_empty[st], 3);
            if (c == C::KC - 1) {
              mma_commit_pair(&ct.t_full[acc & 1], 3);
              if (last) mma_commit_pair(&ct.a_empty, 3);
            }
          }
          __syncwarp();
        }
      }
      // every MMA issued above has completed before TMEM is freed
      if (elect_one()) mma_commit_pair(&ct.done, 1);
      drain(&ct.done, 0, globaltimer());
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    // Keys and values are rounded to bf16 here: they are operands of the attention's
    // products, which take 16 bits, and half the bytes on their way.
    // Four threads per key, 16 of each 64 numbers a thread: the weights' rows are
    // loaded in the order that makes them neighbours (row 8 i + 2 q + e of 64 is
    // 16 q + 2 i + e), so a key's 128 bytes go out together.  (One thread per key
    // stored single sectors, 2,048 an item, which took 2.2 us and kept the weights'
    // loads waiting: 4.4 us an item.)  A value that is not finite would reach, times a
    // probability of 0, tokens that do not see the key: such a value row is
    // stored as zeros and the key as NaN, which the tokens that do see it get.
    const int qu = warp & 3, quad = lane & 3;
    const uint32_t lane_base = static_cast<uint32_t>(qu * 32) << 16;
    Walk k = start();
    int64_t blk = 2 * p0 + rank;
    int hg = hg0, acc = 0;
    const uint32_t empty0 = mapa_shared(smem_u32(&ct.t_empty[0]), 0), empty1 = mapa_shared(smem_u32(&ct.t_empty[1]), 0);
    for (int64_t i = x0; i < x1; ++i, ++acc) {
      if (blk < total && (i == x0 || hg == 0)) reach(k, blk);
      const bool fail = !mbar_wait(&ct.t_full[acc & 1], (acc >> 1) & 1, abort_flag, p.err, kErrWaitEpilogue);
      if (__any_sync(0xffffffffu, fail)) break;   // tcgen05.ld below is warp-collective
      tc_fence_after();
      if (blk < total) {
        const int key0 = static_cast<int>(blk - k.base) * kBlk;
        uint8_t *kv = reinterpret_cast<uint8_t *>(p.kv + (static_cast<int64_t>(hg) * p.cap_blocks + blk) * kBlk * (2 * HD));
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {   // 16 keys of the warp's 32: a thread has keys row and row + 8
          const uint32_t t = tmem + lane_base + (static_cast<uint32_t>(half * 16) << 16) + 256 * (acc & 1);
          const int row = qu * 32 + half * 16 + (lane >> 2);
          uint8_t *dst = kv + row * (4 * HD) + 32 * quad;
          uint32_t pk[2][HD / 8];
          float odd[2] = {0.f, 0.f};   // NaN if a value is not finite
          bool stale[2], wipe[2];
#pragma unroll
          for (int b = 0; b < HD / 64; ++b) {
            float v[2][16];
            tmem_ld_rows(t + HD + 64 * b, v);
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t x = pack_bf16x2(v[r][2 * e], v[r][2 * e + 1]);
                pk[r][8 * b + e] = x;
                odd[r] = fmaf(bf16lo(x), 0.f, odd[r]);
                odd[r] = fmaf(bf16hi(x), 0.f, odd[r]);
              }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            odd[r] += __shfl_xor_sync(0xffffffffu, odd[r], 1);
            odd[r] += __shfl_xor_sync(0xffffffffu, odd[r], 2);
            stale[r] = key0 + row + 8 * r >= k.w.kv;
            wipe[r] = stale[r] || odd[r] != 0.f;
#pragma unroll
            for (int b = 0; b < HD / 64; ++b) {
              if (wipe[r])
#pragma unroll
                for (int e = 0; e < 8; ++e) pk[r][8 * b + e] = 0;
              store32(dst + r * 8 * (4 * HD) + 2 * HD + 128 * b, pk[r] + 8 * b);
            }
          }
#pragma unroll
          for (int b = 0; b < HD / 64; ++b) {
            float v[2][16];
            tmem_ld_rows(t + 64 * b, v);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              uint32_t x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = wipe[r] ? (stale[r] ? 0u : 0x7FC07FC0u) : pack_bf16x2(v[r][2 * e], v[r][2 * e + 1]);
              store32(dst + r * 8 * (4 * HD) + 128 * b, x);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(acc & 1 ? empty1 : empty0);
      if (++hg == p.HG) {
        hg = 0;
        blk += 2;
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();   // (neither CTA's shared memory or TMEM goes while the pair's products use it)
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// --------------------------------------------------------------- attention
template <int HD>
struct PreCfg {
  static constexpr int UNIT = 128 * 128;              // [128 rows][64 bf16]: what the stages are made of
  static constexpr int KU = HD / 64 + 1;              // of a block of keys (the last: their rotated part), of a query tile
  static constexpr int VU = HD / 64;                  // of a block of values
  static constexpr int QT_BYTES = KU * UNIT;
  // One ring for keys and values, in the order they are used (K of a block, then
  // its V): 128 KB hold 1.6 blocks, where rings of their own would leave values
  // a single stage.  K of block b takes the places of K and V of blocks b - KB
  // and b - VB and of what lies between, V of block b those of K of block b - VK.
  static constexpr int NU = HD == 128 ? 8 : 10;
  static constexpr int KB = HD == 128 ? 2 : 3, VB = HD == 128 ? 2 : 4, VK = HD == 128 ? 1 : 3;
  static constexpr int NB = 4;                        // barriers per kind, by block
  static constexpr int NSEG = 4;
  static constexpr int OFF_R = 2 * QT_BYTES;
  static constexpr int OFF_CTRL = OFF_R + NU * UNIT;
  static constexpr int OFF_ML = OFF_CTRL + 1024;      // (m, l) of 128 rows, from one warp group to the other
  static constexpr int SMEM = OFF_ML + 1024;
  static constexpr int THREADS = 384;                 // TMA, 2 MMA issuers, one idle, 2 x 4 softmax warps
  static constexpr uint32_t IDESC_S = idesc_bf16(128, 128, false);
  static constexpr uint32_t IDESC_PV = idesc_bf16(128, HD, true);
  static constexpr uint32_t TMEM_COLS = 512;          // S/P buffers at 0 and 128, O of the two groups from 256
  static constexpr uint32_t O_COL = 256;
};

// A piece of a unit, as the producer tells it to the other roles.
struct PreSeg {
  int32_t nb, j0, qt;    // blocks [j0, j0 + nb), query tiles; nb 0: no more pieces
  int32_t t0, rows;      // first row of q, rows
  int32_t h, first;      // head; the last key that the unit's first row sees
  int32_t slot, qb;      // partial slot, -1: the unit is whole; Q buffer of tile 0 (tile 1: the other one)
};

template <int HD>
struct PreCtrl {
  using C = PreCfg<HD>;
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[C::NB], k_empty[C::NB], v_full[C::NB], v_empty[C::NB];   // by block; empty: both groups are done with it
  uint64_t s_full[2], p_half[2], p_full[2], h_full[2], o_full[2];   // by warp group: S; P of half the keys, of all; P V of them
  uint64_t ml_full[2];    // the group's (m, l) are in shared memory
  uint64_t ml_empty[2];   // the other group has read them and this group's O
  uint64_t seg_full[C::NSEG], seg_empty[C::NSEG];
  uint64_t turn[2];       // the other group's products are issued
  uint64_t done;
  PreSeg seg[C::NSEG];
  uint32_t tmem;
  int abort;
};

// Takes the keys behind `vis` out of a row's block of S (to -inf, in TMEM): a
// pass of its own, for the few blocks on the diagonal.
__device__ __forceinline__ void mask_block(uint32_t s_col, int vis) {
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    float v[32];
    tmem_ld32(s_col + 32 * k, v);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (32 * k + e > vis) v[e] = -INFINITY;
    tmem_st32(s_col + 32 * k, v);
  }
}

template <int HD>
__global__ void __launch_bounds__(PreCfg<HD>::THREADS, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQR,
                          const __grid_constant__ CUtensorMap tmKV, const __grid_constant__ CUtensorMap tmR,
                          const __grid_constant__ PreParams p) {
  using C = PreCfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem, *sR = smem + C::OFF_R;
  static_assert(sizeof(PreCtrl<HD>) <= 1024 && C::SMEM <= 232448, "shared memory");
  PreCtrl<HD> &ct = *reinterpret_cast<PreCtrl<HD> *>(smem + C::OFF_CTRL);
  volatile int *abort_flag = &ct.abort;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // (known uniform)
  if (smem_u32(smem) & 1023u) {   // the swizzled layouts need a 1024-aligned base
    pdl_wait();
    if (threadIdx.x == 0) {
      atomicExch(p.err, kErrBounds);
      p.rec[blockIdx.x * 8] = 0;
    }
    return;
  }
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ct.q_full[b], 1);
      mbar_init(&ct.q_empty[b], 2);
      mbar_init(&ct.s_full[b], 1);
      mbar_init(&ct.p_half[b], 128);
      mbar_init(&ct.p_full[b], 128);
      mbar_init(&ct.h_full[b], 1);
      mbar_init(&ct.o_full[b], 1);
      mbar_init(&ct.ml_full[b], 128);
      mbar_init(&ct.ml_empty[b], 128);
    }
    for (int s = 0; s < C::NB; ++s) {
      mbar_init(&ct.k_full[s], 1);
      mbar_init(&ct.k_empty[s], 2);
      mbar_init(&ct.v_full[s], 1);
      mbar_init(&ct.v_empty[s], 2);
    }
    for (int s = 0; s < C::NSEG; ++s) {
      mbar_init(&ct.seg_full[s], 1);
      mbar_init(&ct.seg_empty[s], 10);   // the 2 MMA issuers and the 8 softmax warps
    }
    for (int b = 0; b < 2; ++b) mbar_init(&ct.turn[b], 1);
    mbar_init(&ct.done, 2);
    ct.abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmQR);
    prefetch_tmap(&tmKV);
    prefetch_tmap(&tmR);
  }
  if (warp == 1) {
    tmem_alloc(&ct.tmem, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ct.tmem, 0);
  const int cta = blockIdx.x;

  if (warp == 0) {
    // ------------------------------------------------ schedule, TMA producer
    // (Only this thread waits for the kernel before: the other roles read what its
    // copies bring and what it tells them.)
    if (lane == 0) {
      pdl_wait();
      pdl_trigger();
      const PrePart part = p.parts[cta];
      int32_t rec[4] = {0, 0, 0, 0};
      int r = part.req, hg = part.hg, u = part.u;
      PreReq q = part.q;
      const int64_t total = part.total, x0 = part.x0, x1 = r >= 0 ? part.x1 : 0;
      const int64_t W = min(max(total / kMinShare, static_cast<int64_t>(total > 0)), static_cast<int64_t>(p.ctas));
      int64_t base = r >= 0 ? part.base : 0;
      ReqWords w{};
      if (r >= 0) w = load_req(p.qo_indptr, p.kv_len, p.bt_indptr, r);
      int blk = 0, nseg = 0, quse[2] = {0, 0}, qsel = 0;
      bool ok = true, k_sent = false;
      auto freed = [&](uint64_t *empty, int b) {   // block b (if there is one) of a kind has been used
        return b < 0 || mbar_wait(&empty[b % C::NB], (b / C::NB) & 1, abort_flag, p.err, kErrWaitProducer);
      };
      // 128 x 64 parts of keys or values: columns x .. x + 63 of row y of `map` to place u of the ring
      auto tile = [&](int u, const CUtensorMap *map, uint64_t *full, int x, int y) {
        tma_load_2d(sR + (u % C::NU) * C::UNIT, map, full, x, y);
      };
      while (ok && base < x1) {
        // the unit (hg, u) of request r, on the line from `base`
        const int rows = u < q.full ? 256 : q.rem, qt = rows > 128 ? 2 : 1, b = qt == 2 ? kCost2 : kCost1;
        const int nkb = u < q.full ? q.a + 2 * (u + 1) : tail_blocks(q);
        const int64_t cost = kCostUnit + static_cast<int64_t>(b) * nkb;
        auto cut = [&](int64_t x) {   // blocks of the unit that lie before x
          const int64_t d = x - base - kCostUnit;
          if (d <= 0) return 0;
          const int64_t n = qt == 2 ? (d + kCost2 - 1) / kCost2 : (d + kCost1 - 1) / kCost1;
          return static_cast<int>(min(static_cast<int64_t>(nkb), n));
        };
        auto owner = [&](int j) {     // the CTA whose part holds block j: the last w with total w / W <= its place
          return static_cast<int>(div64((base + kCostUnit + static_cast<int64_t>(b) * j + 1) * W - 1, total));
        };
        const int j0 = cut(x0), j1 = cut(x1);
        if (j1 > j0) {
          const int i0 = 256 * u, h = p.h0 + hg;
          const int krow = (hg * p.cap_blocks + q.row_blk) * kBlk, rrow = q.row_blk * kBlk;
          for (int t = 0; t < qt && ok; ++t) {
            const int qb = qsel ^ t;
            ok = mbar_wait(&ct.q_empty[qb], (quse[qb] & 1) ^ 1, abort_flag, p.err, kErrWaitProducer);
            if (!ok) break;
            mbar_arrive_expect_tx(&ct.q_full[qb], C::QT_BYTES);
            for (int ch = 0; ch < C::KU - 1; ++ch)
              tma_load_3d(sQ + qb * C::QT_BYTES + ch * C::UNIT, &tmQ, &ct.q_full[qb], ch * 64, h, q.t0 + i0 + 128 * t);
            tma_load_3d(sQ + qb * C::QT_BYTES + (C::KU - 1) * C::UNIT, &tmQR, &ct.q_full[qb], 0, h, q.t0 + i0 + 128 * t);
            ++quse[qb];
          }
          auto send = [&](int j) {   // block j
            const int u0 = blk * (C::KU + C::VU), sb = blk % C::NB;
            ok = freed(ct.k_empty, blk - C::KB) && freed(ct.v_empty, blk - C::VB);
            if (!ok) return;
            mbar_arrive_expect_tx(&ct.k_full[sb], C::KU * C::UNIT);
            for (int ch = 0; ch < C::KU - 1; ++ch) tile(u0 + ch, &tmKV, &ct.k_full[sb], 64 * ch, krow + kBlk * j);
            tile(u0 + C::KU - 1, &tmR, &ct.k_full[sb], 0, rrow + kBlk * j);
            k_sent = true;
            ok = freed(ct.k_empty, blk - C::VK);
            if (!ok) return;
            mbar_arrive_expect_tx(&ct.v_full[sb], C::VU * C::UNIT);
            for (int ch = 0; ch < C::VU; ++ch) tile(u0 + C::KU + ch, &tmKV, &ct.v_full[sb], HD + 64 * ch, krow + kBlk * j);
            ++blk;
            k_sent = false;
          };
          if (!ok) break;
          int j = j0;
          if (blk == 0) send(j++);   // (nothing to wait for: on its way before the books are kept)
          const int first = owner(0), last = owner(nkb - 1);
          const int ss = nseg % C::NSEG;
          ok = ok && mbar_wait(&ct.seg_empty[ss], ((nseg / C::NSEG) & 1) ^ 1, abort_flag, p.err, kErrWaitProducer);
          if (!ok) break;
          PreSeg &sg = ct.seg[ss];
          sg.nb = j1 - j0;
          sg.j0 = j0;
          sg.qt = qt;
          sg.t0 = q.t0 + i0;
          sg.rows = rows;
          sg.h = h;
          sg.first = q.c + i0;
          sg.slot = first == last ? -1 : 2 * cta + (cta == first ? 1 : 0);
          sg.qb = qsel;
          mbar_arrive(&ct.seg_full[ss]);
          ++nseg;
          if (first != last && cta == first) {
            rec[0] = last - first + 1;
            rec[1] = q.t0 + i0;
            rec[2] = h;
            rec[3] = rows;
          }
          if (qt == 1) qsel ^= 1;
          while (ok && j < j1) send(j++);
        }
        // the next unit on the line
        base += cost;
        if (++u == q.full + (q.rem ? 1 : 0)) {
          u = 0;
          if (++hg == p.HG) {
            hg = 0;
            int64_t row_blk = q.row_blk;
            do {
              bool bad;
              row_blk += key_blocks(w, p.T, &bad);
              if (++r >= p.n_reqs) break;
              w = load_req(p.qo_indptr, p.kv_len, p.bt_indptr, r);
              q = pre_req(p, w, row_blk);
            } while (q.n == 0);
            if (r >= p.n_reqs) break;
          }
        }
      }
      if (ok) {
        const int ss = nseg % C::NSEG;
        if (mbar_wait(&ct.seg_empty[ss], ((nseg / C::NSEG) & 1) ^ 1, abort_flag, p.err, kErrWaitProducer)) {
          ct.seg[ss].nb = 0;
          mbar_arrive(&ct.seg_full[ss]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) p.rec[cta * 8 + k] = rec[k];
      // after an abort, let copies in flight land before the CTA exits (bounded)
      if (!ok || *abort_flag) {
        const uint64_t t_start = globaltimer();
        for (int b = max(0, blk - C::NB); b < blk; ++b) {
          drain(&ct.k_full[b % C::NB], b / C::NB, t_start);
          drain(&ct.v_full[b % C::NB], b / C::NB, t_start);
        }
        if (!ok && k_sent) drain(&ct.k_full[blk % C::NB], blk / C::NB, t_start);
        for (int b = 0; b < 2; ++b)
          if (quse[b] > 0) drain(&ct.q_full[b], quse[b] - 1, t_start);
      }
    }
    __syncwarp();
  } else if (warp <= 2) {
    // -------------------------------------------------------- MMA issuers
    // One per group, strictly in turn: P V of the group's item, then S of its next
    // one (P lies over S, so not before), while the other group is at its
    // softmax.  Side by side without turns, both groups' products finished
    // together and left both at their softmax together (4,900 cycles a block
    // of two tiles); by one warp, its waits and commits lay between the products
    // (4,250).  The whole warp keeps the books, in step, and one elected lane issues
    // (the descriptors stay in uniform registers).
    const int w = warp - 1;
    const uint32_t sr = smem_u32(sR);
    const uint64_t qd0 = sdesc_sw128(smem_u32(sQ), 16, 1024), rd0 = sdesc_sw128(sr, 16, 1024);
    const uint32_t s_col = tmem + 128 * w, o_col = tmem + C::O_COL + HD * w;
    auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    auto wait = [&](uint64_t *bar, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, p.err, kErrWaitMma)) != 0;
    };
    int nseg = 0, item0 = 0, blk0 = 0, nb = 0, qt = 0, qb0 = 0, li = 0, items = 0;   // the piece, the place in it
    int quse0 = 0, quse1 = 0, slot = 0;
    int v_seg = -1, v_sb = 0, v_u = 0, v_ph = 0, v_par = 0;   // the item whose P V comes next (v_seg: the piece it ends, -1: none)
    bool in = false, end = false, v_have = false, v_first = false, v_twice = false, ok = true;
    while (ok) {
      if (v_have) ok = wait(&ct.p_half[w], v_par) && wait(&ct.v_full[v_sb], v_ph);
      if (ok && (w == 1 || slot > 0)) ok = wait(&ct.turn[w], (w == 1 ? slot : slot - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      if (v_have) {
        // P V, the first 64 keys while the softmax may be at the others; hd as 64
        // and 64 where the ring's end lies between its halves
        const bool side = C::VU == 1 || v_u + 1 < C::NU;
        const uint64_t vd = side ? sdesc_sw128(sr + v_u * C::UNIT, C::UNIT, 1024) : rd0 + static_cast<uint64_t>((v_u * C::UNIT) >> 4);
        constexpr uint32_t IDESC_64 = idesc_bf16(128, 64, true);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half == 1) ok = wait(&ct.p_full[w], v_par);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (side) {
#pragma unroll
              for (int ks = 4 * half; ks < 4 * half + 4; ++ks)   // 16 keys (two atoms) per MMA
                mma_bf16_ts(o_col, s_col + ks * 8, vd + ((ks * 2048) >> 4), C::IDESC_PV, (!v_first || ks > 0) ? 1u : 0u);
            } else {
#pragma unroll
              for (int ch = 0; ch < C::VU; ++ch)
#pragma unroll
                for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
                  mma_bf16_ts(o_col + 64 * ch, s_col + ks * 8, (ch ? rd0 : vd) + ((ks * 2048) >> 4), IDESC_64, (!v_first || ks > 0) ? 1u : 0u);
            }
            mma_commit(half ? &ct.o_full[w] : &ct.h_full[w]);
            if (half == 1) {
              mma_commit(&ct.v_empty[v_sb]);
              if (v_twice) mma_commit(&ct.v_empty[v_sb]);   // (for the other group, which does not take this block)
              if (v_seg >= 0) mbar_arrive(&ct.seg_empty[v_seg % C::NSEG]);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      // the group's next item
      while (ok && !end && !in) {
        ok = wait(&ct.seg_full[nseg % C::NSEG], (nseg / C::NSEG) & 1);
        if (!ok) break;
        const PreSeg &sg = ct.seg[nseg % C::NSEG];
        nb = uni(sg.nb);
        qt = uni(sg.qt);
        qb0 = uni(sg.qb);
        if (nb == 0) {
          end = true;
          break;
        }
        items = nb * qt;
        li = (item0 & 1) ^ w;
        in = li < items;
        if (!in) {   // (one block, and it is the other group's)
          if (lane == 0) mbar_arrive(&ct.seg_empty[nseg % C::NSEG]);
          ++quse0, quse0 -= qb0, quse1 += qb0;
          item0 += items;
          blk0 += nb;
          ++nseg;
        }
      }
      if (!ok) break;
      v_have = in;
      if (in) {
        const int blk = blk0 + (qt == 2 ? li >> 1 : li), sb = blk % C::NB, u0 = blk * (C::KU + C::VU);
        const int qb = qt == 2 ? qb0 ^ (li & 1) : qb0;
        if (li < 2) ok = wait(&ct.q_full[qb], (qb ? quse1 : quse0) & 1);
        ok = ok && wait(&ct.k_full[sb], (blk / C::NB) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t qd = qd0 + static_cast<uint64_t>((qb * C::QT_BYTES) >> 4);
        const bool last = li + 2 >= items, lone = qt == 2 || items == 1;   // lone: the tile's only user
        if (elect_one()) {
#pragma unroll
          for (int ch = 0; ch < C::KU; ++ch) {
            const uint64_t kd = rd0 + static_cast<uint64_t>((((u0 + ch) % C::NU) * C::UNIT) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16(s_col, qd + ((ch * C::UNIT + kk * 32) >> 4), kd + ((kk * 32) >> 4), C::IDESC_S, (ch > 0 || kk > 0) ? 1u : 0u);
          }
          mbar_arrive(&ct.turn[w ^ 1]);
          mma_commit(&ct.s_full[w]);
          mma_commit(&ct.k_empty[sb]);
          if (qt == 1) mma_commit(&ct.k_empty[sb]);
          if (last) {
            mma_commit(&ct.q_empty[qb]);
            if (lone) mma_commit(&ct.q_empty[qb]);
          }
        }
        __syncwarp();
        v_first = li < 2;
        v_twice = qt == 1;
        v_sb = sb;
        v_ph = (blk / C::NB) & 1;
        v_u = (u0 + C::KU) % C::NU;
        v_par = ((item0 + li) >> 1) & 1;
        v_seg = last ? nseg : -1;
        li += 2;
        if (last) {
          // (both groups count a tile's uses, whoever they are)
          if (qt == 2) ++quse0, ++quse1;
          else ++quse0, quse0 -= qb0, quse1 += qb0;
          item0 += items;
          blk0 += nb;
          ++nseg;
          in = false;
        }
      } else {
        if (elect_one()) mbar_arrive(&ct.turn[w ^ 1]);
        __syncwarp();
      }
      ++slot;
      if (end && !v_have) break;
    }
    // every MMA issued above has completed before TMEM is freed
    if (elect_one()) mma_commit(&ct.done);
    __syncwarp();
    drain(&ct.done, 0, globaltimer());
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------- softmax / epilogue
    const int w = (warp - 4) >> 2;          // warp group: it takes every second item
    const int qu = warp & 3;                // TMEM lane quarter
    const int row = qu * 32 + lane;         // row of the tile
    const uint32_t lane_base = static_cast<uint32_t>(qu * 32) << 16;
    const uint32_t s_col = tmem + lane_base + 128 * w;
    const uint32_t o_col = tmem + lane_base + C::O_COL + HD * w;
    const uint32_t o_other = tmem + lane_base + C::O_COL + HD * (w ^ 1);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    const float scale = p.scale_log2;
    const float2 sc2 = make_float2(scale, scale);
    int nseg = 0, item0 = 0;
    int lent[2] = {0, 0};     // times that group 0, 1 left its part of a piece to the other
    bool lending = false;     // the other group may still be reading this one's O and (m, l)
    bool ok = true;
    while (true) {
      const int ss = nseg % C::NSEG;
      bool fail = !mbar_wait(&ct.seg_full[ss], (nseg / C::NSEG) & 1, abort_flag, p.err, kErrWaitSoftmax);
      if (__any_sync(0xffffffffu, fail)) break;   // tcgen05.ld below is warp-collective
      const PreSeg &sg = ct.seg[ss];
      const int nb = sg.nb;
      if (nb == 0) break;
      const int qt = sg.qt, j0 = sg.j0;
      const int items = nb * qt;
      const int lb0 = (item0 & 1) ^ w;       // this group's first item of the piece
      const int t = qt == 2 ? lb0 : 0;       // its query tile
      if (lb0 >= items) {                    // one block, and it is the other group's
        ++item0;
        ++nseg;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.seg_empty[ss]);
        continue;
      }
      const int rows = min(sg.rows - 128 * t, 128);
      const bool idle = qu * 32 >= rows;     // no rows for this warp
      const int limit = sg.first + 128 * t + row;   // the last key that the row sees
      float m_ref = -INFINITY, l = 0.f;
      for (int li = lb0; li < items; li += 2) {
        const int item = item0 + li, lb = qt == 2 ? li >> 1 : li;
        const int key0 = kBlk * (j0 + lb);
        fail = !mbar_wait(&ct.s_full[w], (item >> 1) & 1, abort_flag, p.err, kErrWaitSoftmax);
        if (__any_sync(0xffffffffu, fail)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (!idle) {
          if (key0 + kBlk - 1 > sg.first + 128 * t + qu * 32) mask_block(s_col, limit - key0);
          // The group's first block of the piece sets each row's reference
          // maximum.
          if (li < 2) {
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              float sv[32];
              tmem_ld32(s_col + 32 * k, sv);
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                m0 = max3f(m0, sv[e], sv[e + 1]);
                m1 = max3f(m1, sv[e + 2], sv[e + 3]);
              }
            }
            m_ref = fmaxf(m0, m1) * scale;
          }
        }
        if (lending) {
          // P V of this item overwrites O: the other group must have read it
          fail = !mbar_wait(&ct.ml_empty[w], (lent[w] - 1) & 1, abort_flag, p.err, kErrWaitSoftmax);
          if (__any_sync(0xffffffffu, fail)) {
            ok = false;
            break;
          }
          lending = false;
        }
        // Half the keys at a time, so that P V of the first runs beside the
        // second.  No maximum is taken as long as the reference holds: a half
        // whose probabilities sum to more than 2^14 says that a logit rose above
        // it (P and the sums have room for far more); then the reference moves, O
        // is rescaled and the half is taken again from S, intact until its P is
        // stored.  P goes over S: keys 0-63 in columns 0-31, keys 64-127 in 32-63.
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
          if (!idle) {
            float sv[64];
            uint32_t pk[32];
            float2 sum = make_float2(0.f, 0.f);
            float negm = m_ref == -INFINITY ? 0.f : -m_ref;   // a row that has seen nothing yet
            tmem_ld64(s_col + 64 * hh, sv);
            probs<64>(sv, sc2, negm, pk, sum);
            // (a row that has seen nothing has no reference to hold)
            const bool grow = sum.x + sum.y > 16384.f || m_ref == -INFINITY;
            if (__any_sync(0xffffffffu, grow)) {
              // O holds the group's blocks before, and the half before: their P V must be done
              fail = false;
              if (hh == 1) fail = !mbar_wait(&ct.h_full[w], (item >> 1) & 1, abort_flag, p.err, kErrWaitSoftmax);
              else if (li >= 2) fail = !mbar_wait(&ct.o_full[w], ((item - 2) >> 1) & 1, abort_flag, p.err, kErrWaitSoftmax);
              if (__any_sync(0xffffffffu, fail)) {
                ok = false;
                break;
              }
              tc_fence_after();
              float mx = -INFINITY;
              tmem_ld64(s_col + 64 * hh, sv);
#pragma unroll
              for (int e = 0; e < 64; e += 2) mx = max3f(mx, sv[e], sv[e + 1]);
              mx *= scale;
              const bool up = grow && mx > m_ref;
              const float alpha = up ? ex2_approx(m_ref - mx) : 1.f;
              if (hh == 1 || li >= 2) {
#pragma unroll 1
                for (int cc = 0; cc < HD / 32; ++cc) {
                  float v[32];
                  tmem_ld32(o_col + cc * 32, v);
#pragma unroll
                  for (int k = 0; k < 32; ++k) v[k] *= alpha;
                  tmem_st32(o_col + cc * 32, v);
                }
              }
              if (up) {
                l *= alpha;
                m_ref = mx;
              }
              negm = m_ref == -INFINITY ? 0.f : -m_ref;
              sum = make_float2(0.f, 0.f);
              probs<64>(sv, sc2, negm, pk, sum);
            }
            tmem_st32u(s_col + 32 * hh, pk);
            l += sum.x + sum.y;
          }
          tc_fence_before();
          mbar_arrive(hh ? &ct.p_full[w] : &ct.p_half[w]);
        }
        if (!ok) break;
      }
      if (!ok) break;
      // ---- the piece is done: its output, or its partial
      const int last_item = item0 + items - 1;
      const bool joint = qt == 1 && nb > 1;         // both groups had blocks of the tile
      if (joint && (last_item & 1) != w) {
        // the other group has the last block: it gets this one's m and l
        ml[row] = make_float2(m_ref, l);
        ++lent[w];
        lending = true;
        tc_fence_before();
        mbar_arrive(&ct.ml_full[w]);
      } else {
        const int mine_last = qt == 2 ? item0 + items - 2 + lb0 : last_item;
        fail = !mbar_wait(&ct.o_full[w], (mine_last >> 1) & 1, abort_flag, p.err, kErrWaitSoftmax);
        float wa = 1.f, wb = 0.f;                     // weights of this group's O and the other's
        if (joint) {
          if (!fail) fail = !mbar_wait(&ct.ml_full[w ^ 1], lent[w ^ 1] & 1, abort_flag, p.err, kErrWaitSoftmax);
          ++lent[w ^ 1];
          if (!fail) fail = !mbar_wait(&ct.o_full[w ^ 1], ((last_item - 1) >> 1) & 1, abort_flag, p.err, kErrWaitSoftmax);
          const float2 o = ml[row];
          const float M = fmaxf(m_ref, o.x);
          wa = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - M);
          wb = o.x == -INFINITY ? 0.f : ex2_approx(o.x - M);
          // (a group whose part of the row is NaN has that in its sum too)
          l = (m_ref == -INFINITY ? l : wa * l) + (o.x == -INFINITY ? o.y : wb * o.y);
          m_ref = M;
        }
        if (__any_sync(0xffffffffu, fail)) break;
        tc_fence_after();
        if (!idle) {
          const bool valid = row < rows;
          const int tok = sg.t0 + 128 * t + row, slot = sg.slot;
          const float inv = 1.f / l;
          __nv_bfloat16 *dst = p.o + (static_cast<int64_t>(tok) * p.H + sg.h) * HD;
          float *part = p.part + max(slot, 0) * part_floats(HD) + 128 * t + row;
#pragma unroll 1
          for (int cc = 0; cc < HD / 32; ++cc) {
            float v[32];
            tmem_ld32(o_col + cc * 32, v);
            if (joint) {
              float x[32];
              tmem_ld32(o_other + cc * 32, x);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = wa * v[k] + wb * x[k];
            }
            if (valid && slot < 0) {
              uint32_t x[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = pack_bf16x2(v[2 * k] * inv, v[2 * k + 1] * inv);
              store_out(dst + cc * 32, x);
              store_out(dst + cc * 32 + 16, x + 8);
            } else if (slot >= 0) {
              // (column by column: a warp's stores fill whole lines; row by row they
              // took 5,000 cycles a piece.  Rows that are none have a place too.)
#pragma unroll
              for (int k = 0; k < 32; ++k) part[(cc * 32 + k) * 256] = v[k];
            }
          }
          if (slot >= 0) reinterpret_cast<float2 *>(part - row - 128 * t + 256 * HD)[128 * t + row] = make_float2(m_ref, l);
        }
        tc_fence_before();
        if (joint) mbar_arrive(&ct.ml_empty[w ^ 1]);
      }
      item0 += items;
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

// Merge of the units that were cut: CTA (w, y) takes rows 32 y .. 32 y + 31 of the
// unit whose first piece CTA w computed, a lane a row, a warp 8 columns.
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,   M = max_s m_s
template <int HD>
__global__ void __launch_bounds__(4 * HD) latent_prefill_merge_kernel(const __grid_constant__ PreParams p) {
  constexpr int COLS = 8;
  pdl_wait();
  pdl_trigger();
  const int w = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 rec = *reinterpret_cast<const int4 *>(p.rec + w * 8);
  const int pieces = rec.x, row = blockIdx.y * 32 + lane;
  if (pieces == 0 || static_cast<int>(blockIdx.y) * 32 >= rec.w) return;
  // piece 0 in slot 2 w + 1, piece s > 0 in slot 2 (w + s)
  auto src = [&](int s) { return p.part + (s == 0 ? 2 * w + 1 : 2 * (w + s)) * part_floats(HD); };
  float M = -INFINITY, L = 0.f, acc[COLS];
#pragma unroll
  for (int k = 0; k < COLS; ++k) acc[k] = 0.f;
#pragma unroll 4
  for (int s = 0; s < pieces; ++s) {
    const float *x = src(s);
    float v[COLS];
#pragma unroll
    for (int k = 0; k < COLS; ++k) v[k] = x[(warp * COLS + k) * 256 + row];
    const float2 ml = reinterpret_cast<const float2 *>(x + 256 * HD)[row];
    const float mn = fmaxf(M, ml.x);
    // (a piece of which the row saw nothing has a sum of 0, or NaN if it saw one)
    const float a = M == -INFINITY ? 0.f : ex2_approx(M - mn), b = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mn);
    L = (M == -INFINITY ? L : L * a) + (ml.x == -INFINITY ? ml.y : b * ml.y);
    M = mn;
#pragma unroll
    for (int k = 0; k < COLS; ++k) acc[k] = acc[k] * a + (b == 0.f ? 0.f : b * v[k]);
  }
  const float inv = 1.f / L;
  uint32_t x[COLS / 2];
#pragma unroll
  for (int k = 0; k < COLS / 2; ++k) x[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  // out row by row: HD / 8 threads a row
  __shared__ uint4 sh[32][HD / 8 + 1];
  sh[lane][warp] = make_uint4(x[0], x[1], x[2], x[3]);
  __syncthreads();
  const int r = threadIdx.x / (HD / 8), c = threadIdx.x % (HD / 8), out = blockIdx.y * 32 + r;
  if (out < rec.w)
    reinterpret_cast<uint4 *>(p.o + (static_cast<int64_t>(rec.y + out) * p.H + rec.z) * HD)[c] = sh[r][c];
}

// The workspace's keys: blocks of 128, each request's from a block of its own.
int64_t cap_blocks(int64_t kv_tokens, int64_t n_reqs) { return kv_tokens / kBlk + n_reqs; }

int64_t head_bytes(int64_t blocks, int64_t hd) { return blocks * kBlk * 4 * hd; }   // one head's keys and values

// Heads of a group: as many as keep its keys and values within kGroupBytes, evenly spread.
int group_heads(int64_t blocks, int64_t H, int64_t hd) {
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(H, kGroupBytes / std::max<int64_t>(1, head_bytes(blocks, hd))));
  const int64_t groups = (H + most - 1) / most;
  return static_cast<int>((H + groups - 1) / groups);
}

// Room for a group's keys and values: what all heads take, at most kGroupBytes, and
// one head's at least.  The even spread may need about half of that (just above
// kGroupBytes two groups have half the heads each), but a size that followed it
// would fall as a batch grows, and a workspace of the largest call has to do for
// every smaller one.
size_t kv_room(int64_t blocks, int64_t H, int64_t hd) {
  const int64_t one = head_bytes(blocks, hd);
  return std::max<int64_t>(one, std::min<int64_t>(H * one, kGroupBytes));
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <int HD, int RANK>
cudaError_t launch_expand(const CUtensorMap &tk, const CUtensorMap &tw, const CUtensorMap &tr, const PreParams &p, cudaStream_t st) {
  using C = ExpCfg<HD, RANK>;
  cudaError_t e = ensure_max_smem(reinterpret_cast<const void *>(latent_expand_kernel<HD, RANK>), C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_expand_kernel<HD, RANK>, dim3(device_sm_count() / 2 * 2), dim3(C::THREADS), C::SMEM, st, 2, tk, tw, tr, p);
}

template <int HD>
cudaError_t launch_prefill(const LatentArgs &a, PreParams &p, int group, __nv_bfloat16 *rope, cudaStream_t st) {
  using C = PreCfg<HD>;
  const uint64_t H = a.H, T = a.T, W = a.rank + kLatentRope, nc = a.rank / 64 + 1;
  const uint64_t rows = static_cast<uint64_t>(p.cap_blocks) * kBlk;
  CUtensorMap tq, tqr, tkv, tr, ts, tk, tw;
  const uint64_t dq[3] = {HD + kLatentRope, H, T}, sq[2] = {(HD + kLatentRope) * 2, (HD + kLatentRope) * 2 * H};
  const uint64_t dr[3] = {kLatentRope, H, T}, sr[2] = {kLatentRope * 2, kLatentRope * 2 * H};
  const uint32_t bq[3] = {64, 1, 128};
  const uint64_t dk[5] = {64, 8, nc, kPage / 8, static_cast<uint64_t>(a.num_pages)};
  const uint64_t sk[4] = {W * 2, 128, 8 * W * 2, kPage * W * 2};
  const uint32_t bk[5] = {64, 8, static_cast<uint32_t>(nc), kPage / 8, 1};
  cudaError_t e = encode_tmap(&tq, a.q, 3, dq, sq, bq);
  if (e == cudaSuccess) e = encode_tmap(&tqr, a.q_rope, 3, dr, sr, bq);
  if (e == cudaSuccess) e = encode_tmap_2d(&tkv, p.kv, 2 * HD, rows * group, 4 * HD, 64, kBlk);
  if (e == cudaSuccess) e = encode_tmap_2d(&tr, rope, kLatentRope, rows, kLatentRope * 2, 64, kBlk);
  if (e == cudaSuccess) e = encode_tmap_2d(&ts, rope, kLatentRope, rows, kLatentRope * 2, 64, 8);
  if (e == cudaSuccess) e = encode_tmap_5d(&tk, a.pool, dk, sk, bk);
  // the weights' rows, 64 at a time, in the order in which the expansion stores what they make
  const uint64_t R = a.rank, dw[5] = {R, 2, 4, 8, H * 2 * HD / 64}, sw[4] = {R * 2, 16 * R * 2, 2 * R * 2, 64 * R * 2};
  const uint32_t bw[5] = {64, 2, 4, 8, HD / 64};
  if (e == cudaSuccess) e = encode_tmap_5d(&tw, a.w_kv, dw, sw, bw);
  if (e == cudaSuccess) e = ensure_max_smem(reinterpret_cast<const void *>(latent_prefill_kernel<HD>), C::SMEM);
  const int ctas = p.ctas;
  for (p.h0 = 0; p.h0 < a.H && e == cudaSuccess; p.h0 += group) {
    p.HG = std::min(group, a.H - p.h0);
    e = a.rank == 512 ? launch_expand<HD, 512>(tk, tw, ts, p, st) : launch_expand<HD, 256>(tk, tw, ts, p, st);
    if (e == cudaSuccess) e = launch_pdl(latent_prefill_kernel<HD>, dim3(ctas), dim3(C::THREADS), C::SMEM, st, 1, tq, tqr, tkv, tr, p);
    if (e == cudaSuccess) e = launch_pdl(latent_prefill_merge_kernel<HD>, dim3(ctas, 8), dim3(4 * HD), 0, st, 1, p);
  }
  return e;
}

}  // namespace

// a group's keys and values, the rotated keys, the records and parts, the partials
size_t latent_prefill_workspace_bytes(int64_t kv_tokens, int64_t n_reqs, int64_t H, int64_t hd) {
  const int64_t blocks = cap_blocks(kv_tokens, n_reqs);
  return align256(kv_room(blocks, H, hd)) +
         align256(static_cast<size_t>(blocks) * kBlk * kLatentRope * 2) + kRecBytes + kPartsBytes +
         static_cast<size_t>(2) * kMaxCtas * part_floats(hd) * sizeof(float);
}

cudaError_t latent_prefill_run(const LatentArgs &a, cudaStream_t st) {
  const int64_t blocks = cap_blocks(a.kv_tokens, a.n_reqs);
  const int group = group_heads(blocks, a.H, a.hd);
  uint8_t *w = static_cast<uint8_t *>(a.workspace);
  const size_t kv_bytes = align256(kv_room(blocks, a.H, a.hd));
  const size_t rope_bytes = align256(static_cast<size_t>(blocks) * kBlk * kLatentRope * 2);
  PreParams p;
  p.kv = reinterpret_cast<__nv_bfloat16 *>(w);
  p.o = static_cast<__nv_bfloat16 *>(a.o);
  p.w_kv = static_cast<const __nv_bfloat16 *>(a.w_kv);
  p.qo_indptr = a.qo_indptr;
  p.kv_len = a.kv_len;
  p.bt_indptr = a.bt_indptr;
  p.bt = a.bt;
  p.n_reqs = a.n_reqs;
  p.T = a.T;
  p.H = a.H;
  p.h0 = 0;
  p.HG = group;
  p.num_pages = a.num_pages;
  p.cap_blocks = static_cast<int>(blocks);
  p.scale_log2 = a.scale * kLog2e;
  p.rec = reinterpret_cast<int32_t *>(w + kv_bytes + rope_bytes);
  static_assert(kMaxCtas * 32 <= kRecBytes && kMaxCtas * sizeof(PrePart) <= kPartsBytes, "workspace");
  p.parts = reinterpret_cast<PrePart *>(w + kv_bytes + rope_bytes + kRecBytes);
  p.ctas = std::min(device_sm_count(), kMaxCtas);
  p.part = reinterpret_cast<float *>(w + kv_bytes + rope_bytes + kRecBytes + kPartsBytes);
  p.err = a.err;
  __nv_bfloat16 *rope = reinterpret_cast<__nv_bfloat16 *>(w + kv_bytes);
  return a.hd == 128 ? launch_prefill<128>(a, p, group, rope, st) : launch_prefill<64>(a, p, group, rope, st);
}

}  // namespace mb
