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
// for every q-head; q-head h reads KV head h / G, G = Hq / Hkv.
//
// What bounds it: every key and value of the prefix is read once for all
// nodes and heads that share it, 4 hd bytes per key and KV head, against
// 4 hd n G operations: n G operations a byte.  The ratio of the measured
// tensor and copy rates is 285, so trees of up to about 285 / G nodes are
// bound by HBM and larger ones by the tensor cores and the softmax.
//
// Measured (head_dim 128, G = 4, 8 KV heads): 16 trees of 8 nodes at 8,192
// keys 91 us, 5.9 TB/s, 87 % of a copy's rate; 64 trees of 8 at 1,125 keys
// 59 us, 5.2 TB/s (a CTA has 3.4 units of 9 blocks each, and every unit's end
// waits for its last softmax and product); 16 trees of 64 nodes at 8,192 keys
// 131.5 us, 1.05 PFLOP/s of bf16, 54 % of a plain matrix product's rate, bound
// by the chain S, softmax, P V of the two warp groups (128 us with all keys in
// L2); one tree of 6 nodes at 1,125 keys 12 us, two launches and the chain of
// one block.
//
// Layout of the work.  The rows that share a KV head, (node, q-head of the
// group), row = node G + g, are the M side of the products: 128 / G nodes make
// a query tile of up to 128 rows, loaded by one 3-D copy per 64 columns.  A
// unit is one or two query tiles of a (request, KV head) and all of its
// 128-key blocks, staged once for both tiles:
//
//   S = Q K^T        tcgen05, M = 128 rows, N = 128 keys, K = hd, in TMEM
//   softmax          one thread per row: its maximum and sum need no exchange
//   O += P V         P (bf16, written over S) is the A operand from TMEM, V the
//                    MN-major B operand straight from its stage
//
// Two groups of four softmax warps take turns, each with an S buffer and an O
// accumulator of its own: with two tiles each has one of them, with one tile
// they take its even and odd blocks, as if each computed a piece, and the group
// of the last block joins the two (O of both is in the same TMEM lanes, m and
// l go through shared memory).  So products run during the other group's
// softmax, and one group's output during the other's next unit.
//
// Schedule.  All units of the batch lie on one line, weighted by their blocks
// (and a constant per unit); CTA w of W takes the w-th of W equal parts, so
// every SM streams the same amount whatever the lengths, and a unit cut by a
// border is computed in pieces: fp32 partials (o, m, l) in the workspace, two
// slots per CTA, merged by log-sum-exp in a second small kernel.  Every CTA
// works the parts out by itself from the device descriptor (a scan over the
// requests), so nothing is planned on the host and a captured call follows
// new contents.  The merge is a kernel of its own rather than the work of a
// tile's last CTA: one CTA would have to read up to 152 partials of 256 rows
// alone, and waiting for one another would tie the CTAs of concurrent calls.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "mb_launch.cuh"
#include "mb_ptx.cuh"
#include "mb_spec.h"

namespace mb {
namespace {

using namespace dev;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxTreeCtas = 160;   // CTAs of a launch at most (one per SM); sizes the workspace
constexpr int kRecBytes = 8192;     // workspace: one record of 8 ints per CTA, then the partials
// The schedule's weights: a block of one query tile, a block of two, a unit's
// start and end, and the least a CTA takes (at least kCost2, so that no CTA
// between the first and the last of a unit is left without a block).  A unit's
// start and end cost what 2.5 blocks do: weighted by 3, 96 trees of 13 nodes at
// 1,024 to 8,192 keys took 237 us, by 5 233, by 8 235; 64 at 1,125 keys 66.7, 66.8
// and 67.3.
constexpr int kCost1 = 2, kCost2 = 3, kCostUnit = 5, kMinShare = 3;

struct TreeParams {
  __nv_bfloat16 *o;
  const __nv_bfloat16 *q, *pool;
  const int32_t *qo_indptr, *kv_len, *bt_indptr, *bt, *parent, *is_tree;
  int n_reqs, T, Hq, Hkv, G, num_pages;
  float scale_log2;
  int32_t *rec;
  float *part;   // [2 slots per CTA][256 rows][hd + 4]: o, m, l, pad
  int *err;
};

template <int HD>
struct TreeCfg {
  static constexpr int NH = HD / 64;
  static constexpr int TILE_BYTES = 128 * 128;       // [128 rows][64 bf16]
  static constexpr int QT_BYTES = NH * TILE_BYTES;
  static constexpr int KV_BYTES = NH * TILE_BYTES;   // a block of K or of V, as [8-key group][hd half][8 keys][128 B]
  static constexpr int ATOM_STRIDE = NH * 1024;
  static constexpr int PAGE_BYTES = 2 * ATOM_STRIDE;
  // K runs one block ahead of V (S comes before P V).
  static constexpr int NK = HD == 128 ? 2 : 5;
  static constexpr int NV = HD == 128 ? 3 : 6;
  static constexpr int NSEG = 4;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * QT_BYTES;
  static constexpr int OFF_V = OFF_K + NK * KV_BYTES;
  static constexpr int OFF_CTRL = OFF_V + NV * KV_BYTES;
  static constexpr int OFF_ML = OFF_CTRL + 2048;     // (m, l) of 128 rows, from one warp group to the other
  static constexpr int SMEM = OFF_ML + 1024;
  static constexpr int THREADS = 320;                // TMA, MMA, 2 x 4 softmax warps
  static constexpr uint32_t IDESC_S = idesc_bf16(128, 128, false);
  static constexpr uint32_t IDESC_PV = idesc_bf16(128, HD, true);
  static constexpr uint32_t TMEM_COLS = 512;         // S/P buffers at 0 and 128, O of the two groups from 256
  static constexpr uint32_t O_COL = 256;
};

// A piece of a unit, as the producer tells it to the other roles.
struct Seg {
  int32_t nb;         // blocks [j0, j0 + nb); 0: no more pieces
  int32_t j0, qt;     // first block, query tiles
  int32_t t0, i0;     // the request's first row, the unit's first node
  int32_t hk, c, kv;
  int32_t nodes;      // of the unit
  int32_t slot;       // partial slot, -1: the unit is whole
  int32_t qb;         // Q buffer of tile 0 (tile 1: the other one)
  int32_t b0;         // the request's first block table entry
  uint32_t odd[4];    // nodes whose V row holds an infinity or a NaN (set by the softmax)
  uint8_t parent[kMaxTreeNodes];   // 0xFF: none
};

// What the schedule needs to know of a request.
struct Req {
  int t0, n, kv, b0, nkb;
  int full, rem;   // units of 2 NT nodes, and the nodes of the last one if it is smaller
  int64_t head;    // cost of one KV head
};

template <int HD>
struct Ctrl {
  using C = TreeCfg<HD>;
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[C::NK], k_empty[C::NK], v_full[C::NV], v_empty[C::NV];
  // By warp group.  (A group's next S waits for the P V of its last, so no
  // phase is passed before the group has seen the one before it.)
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t ml_full[2];    // the group's (m, l) are in shared memory
  uint64_t ml_empty[2];   // the other group has read them and this group's O
  uint64_t seg_full[C::NSEG], seg_empty[C::NSEG];
  uint64_t done;
  Seg seg[C::NSEG];
  int64_t wsum[C::THREADS / 32];
  int64_t start_base;
  Req start;
  int32_t start_req;
  uint32_t tmem;
  int abort;
};

// Its words of the descriptor (loaded well before they are worked on).
struct RawReq {
  int q0, q1, kv, b0, b1, tree;
};
__device__ __forceinline__ RawReq load_raw(const TreeParams &p, int r) {
  return {p.qo_indptr[r], p.qo_indptr[r + 1], p.kv_len[r], p.bt_indptr[r], p.bt_indptr[r + 1], p.is_tree ? p.is_tree[r] : 1};
}

// (an invalid request costs nothing: it is skipped and reported)
__device__ __forceinline__ Req make_req(const TreeParams &p, const RawReq x, bool *bad) {
  Req q;
  q.t0 = x.q0;
  q.kv = x.kv;
  q.b0 = x.b0;
  // (compared before they are subtracted: the words may be anything)
  const bool order = x.q0 >= 0 && x.q1 >= x.q0 && x.q1 <= p.T && x.b0 >= 0 && x.b1 >= x.b0;
  q.n = order ? x.q1 - x.q0 : 0;
  *bad = !order || q.n > kMaxTreeNodes || q.kv < q.n || q.kv > (1 << 24) || (q.kv + kPage - 1) / kPage > x.b1 - x.b0;
  *bad = *bad && x.tree;
  if (*bad || !x.tree) q.n = 0;
  q.nkb = (q.kv + 127) / 128;
  const int nt2 = 2 * (128 / p.G);
  q.full = q.n / nt2;
  q.rem = q.n % nt2;
  q.head = static_cast<int64_t>(q.full) * (kCostUnit + kCost2 * static_cast<int64_t>(q.nkb));
  if (q.rem) q.head += kCostUnit + (2 * q.rem > nt2 ? kCost2 : kCost1) * static_cast<int64_t>(q.nkb);
  if (q.n == 0) q.head = 0;
  return q;
}

// 32 columns at each of two addresses of this thread's TMEM lane, one wait.
__device__ __forceinline__ void tmem_ld32x2(uint32_t a, uint32_t b, float (&v)[32], float (&w)[32]) {
  uint32_t r[32], s[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3]), "=r"(s[4]), "=r"(s[5]), "=r"(s[6]), "=r"(s[7]), "=r"(s[8]), "=r"(s[9]), "=r"(s[10]), "=r"(s[11]), "=r"(s[12]), "=r"(s[13]), "=r"(s[14]), "=r"(s[15]), "=r"(s[16]), "=r"(s[17]), "=r"(s[18]), "=r"(s[19]), "=r"(s[20]), "=r"(s[21]), "=r"(s[22]), "=r"(s[23]), "=r"(s[24]), "=r"(s[25]), "=r"(s[26]), "=r"(s[27]), "=r"(s[28]), "=r"(s[29]), "=r"(s[30]), "=r"(s[31])
      : "r"(a), "r"(b)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = __uint_as_float(r[i]);
    w[i] = __uint_as_float(s[i]);
  }
}

// Store 16 consecutive 32-bit columns (raw bits) of this thread's TMEM lane, waited on.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// p = 2^(s scale + negm) of N logits, as bf16 pairs, added into `sum`.
template <int N>
__device__ __forceinline__ void probs(const float (&sv)[N], float2 sc2, float negm, uint32_t (&pk)[N / 2], float2 &sum) {
  const float2 nm = make_float2(negm, negm);
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 x = __ffma2_rn(make_float2(sv[c], sv[c + 1]), sc2, nm);
    const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
    sum = __fadd2_rn(sum, make_float2(p0, p1));
    pk[c / 2] = pack_bf16x2(p0, p1);
  }
}

// One lane of a converged warp (the same one each time).
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
  return is != 0;
}

__device__ __noinline__ int64_t div64(int64_t a, int64_t b) { return a / b; }

// Takes the logits of keys that a row does not see out of a block of S (to
// -inf, in TMEM): `first` is the node index of the block's first key (negative
// while it is a key of the prefix), `see` the nodes that the row's node sees.
// A pass of its own, for the one or two blocks of a unit that hold nodes: it
// keeps the loop over the prefix short.  (Inline: as a call, 256 trees of 8
// nodes at 300 keys took 142 us against 126, and 96 of 13 at up to 8,192 240
// against 234; add_odd, which almost no call reaches, is better out of line:
// inline, the 256 trees took 134 us.)
__device__ __forceinline__ void mask_block(uint32_t s_col, int first, const uint4 see) {
  const uint32_t w[4] = {see.x, see.y, see.z, see.w};
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const int f = first + 32 * k;   // node index of this word's first key
    uint32_t vis = 0;
    if (f <= -32) continue;         // prefix keys
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int sh = 32 * a - f;    // word a of `see` starts at this bit
      if (sh >= 0 && sh < 32) vis |= w[a] << sh;
      if (sh < 0 && sh > -32) vis |= w[a] >> -sh;
    }
    if (f < 0) vis |= (1u << -f) - 1u;
    float v[32];
    tmem_ld32(s_col + 32 * k, v);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((vis >> e) & 1u)) v[e] = -INFINITY;
    tmem_st32(s_col + 32 * k, v);
  }
}

// Adds to 32 columns of a row's o the parts p v of marked nodes (their V rows
// hold an infinity or a NaN and left the product) that the row sees, p from
// the same logit in fp32.  m: the reference that o is relative to.
template <int HD>
__device__ __noinline__ void add_odd(const TreeParams &p, const Seg &sg, uint4 see, int tok, int head, float m, int col,
                                     float *v) {
  const uint32_t w[4] = {sg.odd[0] & see.x, sg.odd[1] & see.y, sg.odd[2] & see.z, sg.odd[3] & see.w};
  for (int a = 0; a < kMaxTreeNodes; ++a) {
    if (!((w[a >> 5] >> (a & 31)) & 1u)) continue;
    const int pos = sg.c + a;
    int pg = p.bt[sg.b0 + pos / kPage];
    if (pg < 0 || pg >= p.num_pages) pg = 0;
    const __nv_bfloat16 *kr = p.pool + ((static_cast<size_t>(pg) * 2 * p.Hkv + sg.hk) * kPage + pos % kPage) * HD;
    const __nv_bfloat16 *vr = kr + static_cast<size_t>(p.Hkv) * kPage * HD;
    const __nv_bfloat16 *qr = p.q + (static_cast<size_t>(tok) * p.Hq + head) * HD;
    float s = 0.f;
    for (int k = 0; k < HD; ++k) s = fmaf(__bfloat162float(qr[k]), __bfloat162float(kr[k]), s);
    const float pr = ex2_approx(fmaf(s, p.scale_log2, m == -INFINITY ? 0.f : -m));
    for (int k = 0; k < 32; ++k) v[k] = fmaf(pr, __bfloat162float(vr[col + k]), v[k]);
  }
}

// What a warp's rows need on their way out of TMEM.
template <int HD>
struct Rows {
  const TreeParams *p;
  const Seg *sg;
  uint4 see;
  int tok, head;
  uint32_t o_col, o_other;   // this group's O, the other's
  bool joint, whole, cut;    // o = wa o + wb o_other; to o, or to a partial (neither: no row)
  float wa, wb, inv, m;
  uint4 *dst;
  float *part;
};

// The rows of a warp to o, or to a partial.  Rolled: the code of a unit's end is
// cold each time it is reached, and with four copies of the loop's body 256
// trees of 8 nodes at 300 keys took 121 us against 99.  (ODD, almost never, is
// out of line for the same reason.)
template <int HD, bool ODD>
__device__ __forceinline__ void write_rows(const Rows<HD> &r, bool odd) {
#pragma unroll 1
  for (int cc = 0; cc < HD / 32; ++cc) {
    float v[32];
    if (r.joint) {
      float x[32];
      tmem_ld32x2(r.o_col + cc * 32, r.o_other + cc * 32, v, x);
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = r.wa * v[k] + r.wb * x[k];
    } else {
      tmem_ld32(r.o_col + cc * 32, v);
    }
    if (ODD && odd) add_odd<HD>(*r.p, *r.sg, r.see, r.tok, r.head, r.m, cc * 32, v);
    if (r.whole) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        r.dst[cc * 4 + k] = make_uint4(pack_bf16x2(v[8 * k] * r.inv, v[8 * k + 1] * r.inv),
                                       pack_bf16x2(v[8 * k + 2] * r.inv, v[8 * k + 3] * r.inv),
                                       pack_bf16x2(v[8 * k + 4] * r.inv, v[8 * k + 5] * r.inv),
                                       pack_bf16x2(v[8 * k + 6] * r.inv, v[8 * k + 7] * r.inv));
    } else if (r.cut) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        reinterpret_cast<float4 *>(r.part + cc * 32)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
  }
}

template <int HD>
__device__ __noinline__ void write_odd(const Rows<HD> &r, bool odd) {
  write_rows<HD, true>(r, odd);
}

template <int HD>
__global__ void __launch_bounds__(TreeCfg<HD>::THREADS, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKV,
                const __grid_constant__ TreeParams p) {
  using C = TreeCfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem + C::OFF_Q;
  uint8_t *sK = smem + C::OFF_K;
  uint8_t *sV = smem + C::OFF_V;
  static_assert(sizeof(Ctrl<HD>) <= 2048, "control area");
  Ctrl<HD> &ct = *reinterpret_cast<Ctrl<HD> *>(smem + C::OFF_CTRL);
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
      mbar_init(&ct.q_empty[b], 1);
      mbar_init(&ct.s_full[b], 1);
      mbar_init(&ct.p_full[b], 128);
      mbar_init(&ct.o_full[b], 1);
      mbar_init(&ct.ml_full[b], 128);
      mbar_init(&ct.ml_empty[b], 128);
    }
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(&ct.k_full[s], 1);
      mbar_init(&ct.k_empty[s], 1);
    }
    for (int s = 0; s < C::NV; ++s) {
      mbar_init(&ct.v_full[s], 1);
      mbar_init(&ct.v_empty[s], 1);
    }
    for (int s = 0; s < C::NSEG; ++s) {
      mbar_init(&ct.seg_full[s], 1);
      mbar_init(&ct.seg_empty[s], 9);   // the MMA issuer and the 8 softmax warps
    }
    mbar_init(&ct.done, 1);
    ct.abort = 0;
    ct.start_req = -1;
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmKV);
  }
  if (warp == 1) {
    tmem_alloc(&ct.tmem, C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();   // the descriptor, q, the pool and o belong to earlier kernels of the stream
  pdl_trigger();

  // ---- this CTA's part of the line: [x0, x1) of `total`
  const int W_max = gridDim.x, cta = blockIdx.x;
  const int per = (p.n_reqs + C::THREADS - 1) / C::THREADS;
  const int r_lo = min(p.n_reqs, static_cast<int>(threadIdx.x) * per), r_hi = min(p.n_reqs, r_lo + per);
  int64_t mine = 0;
  Req last{};
  for (int r = r_lo; r < r_hi; ++r) {
    bool bad;
    last = make_req(p, load_raw(p, r), &bad);
    mine += last.head * p.Hkv;
    if (bad && cta == 0) atomicExch(p.err, kErrBounds);
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
  const int64_t W = total / kMinShare < 1 ? (total > 0 ? 1 : 0) : (total / kMinShare < W_max ? total / kMinShare : W_max);
  const bool active = cta < W;
  const int64_t x0 = active ? div64(total * cta, W) : 0, x1 = active ? div64(total * (cta + 1), W) : 0;
  if (active && pre <= x0 && x0 < pre + mine) {
    for (int r = r_lo; r < r_hi; ++r) {
      bool bad;
      if (per > 1) last = make_req(p, load_raw(p, r), &bad);
      const int64_t c = last.head * p.Hkv;
      if (x0 < pre + c) {
        ct.start_req = r;
        ct.start = last;
        ct.start_base = pre;
        break;
      }
      pre += c;
    }
  }
  __syncthreads();

  if (!active) {
    if (threadIdx.x == 0) p.rec[cta * 8] = 0;
  } else if (warp == 0) {
    // ------------------------------------------------ schedule, TMA producer
    // The whole warp: all lanes wait for each stage (waiting in one and telling
    // the others took 229 us against 222 for 96 trees of 13 nodes at 1,024 to
    // 8,192 keys), lane 0 arms it, a block's 8 pages go out as one copy per lane
    // (by one elected lane in turn: 225 us unrolled, 287 rolled).  The K of a
    // block goes out before the V of the block before it, as a rule; the page ids
    // of the next block are loaded a block ahead, the next request's descriptor
    // when its predecessor starts.
    const int G = p.G, NT = 128 / G;
    int32_t rec[5] = {0, 0, 0, 0, 0};
    int r = ct.start_req;
    int64_t base = ct.start_base;
    bool bad;
    Req q = ct.start;
    RawReq nx{};
    if (r + 1 < p.n_reqs) nx = load_raw(p, r + 1);
    // the unit that x0 lies in
    int64_t off = x0 - base;
    int hk = static_cast<int>(div64(off, q.head));
    base += hk * q.head;
    off -= hk * q.head;
    const int64_t big0 = kCostUnit + kCost2 * static_cast<int64_t>(q.nkb);
    int u = static_cast<int>(min(static_cast<int64_t>(q.full), div64(off, big0)));
    base += u * big0;
    int kcnt = 0, vcnt = 0, nseg = 0, quse[2] = {0, 0}, qsel = 0;
    bool ok = true;
    // the block whose V is still to be sent
    int pv_np = 0, pv_page = 0, pv_hk = 0;
    bool pv_have = false;
    auto send = [&](bool is_v, int np, int page, int h) -> bool {
      const int ns = is_v ? C::NV : C::NK;
      int &cnt = is_v ? vcnt : kcnt;
      const int st = cnt % ns;
      uint64_t *full = (is_v ? ct.v_full : ct.k_full) + st;
      uint64_t *empty = (is_v ? ct.v_empty : ct.k_empty) + st;
      if (!__all_sync(0xffffffffu, mbar_wait(empty, ((cnt / ns) & 1) ^ 1, abort_flag, p.err, kErrWaitProducer))) return false;
      if (lane < np && (page < 0 || page >= p.num_pages)) {
        atomicExch(p.err, kErrBounds);
        page = 0;
      }
      if (lane == 0) mbar_arrive_expect_tx(full, np * C::NH * 2048);
      __syncwarp();
      if (lane < np)
        tma_load_5d((is_v ? sV : sK) + st * C::KV_BYTES + lane * C::PAGE_BYTES, &tmKV, full, 0, 0, 0, 0,
                    (page * 2 + (is_v ? 1 : 0)) * p.Hkv + h);
      ++cnt;
      return true;
    };
    auto room = [&](bool is_v) {   // whether the next stage is free
      const int ns = is_v ? C::NV : C::NK, cnt = is_v ? vcnt : kcnt;
      uint64_t *empty = (is_v ? ct.v_empty : ct.k_empty) + cnt % ns;
      return __all_sync(0xffffffffu, mbar_test_wait(smem_u32(empty), ((cnt / ns) & 1) ^ 1)) != 0;
    };
    while (ok && base < x1) {
      // the unit (hk, u) of request r, on the line from `base`
      const int nodes = u < q.full ? 2 * NT : q.rem;
      const int qt = nodes > NT ? 2 : 1;
      const int b = qt == 2 ? kCost2 : kCost1;
      const int64_t cost = kCostUnit + static_cast<int64_t>(b) * q.nkb;
      auto cut = [&](int64_t x) {   // blocks of the unit that lie before x
        const int64_t d = x - base - kCostUnit;
        if (d <= 0) return 0;
        const int64_t n = qt == 2 ? (d + kCost2 - 1) / kCost2 : (d + kCost1 - 1) / kCost1;
        return static_cast<int>(min(static_cast<int64_t>(q.nkb), n));
      };
      auto owner = [&](int j) {     // the CTA whose part holds block j: the last w with total w / W <= its place
        return static_cast<int>(div64((base + kCostUnit + static_cast<int64_t>(b) * j + 1) * W - 1, total));
      };
      const int j0 = cut(x0), j1 = cut(x1);
      if (j1 > j0) {
        const int first = owner(0), last = owner(q.nkb - 1);
        const int i0 = u * 2 * NT;
        const int32_t *table = p.bt + q.b0;
        const int n_pages = (q.kv + kPage - 1) / kPage;
        auto page_of = [&](int blk) { return lane < 8 && 8 * blk + lane < n_pages ? table[8 * blk + lane] : 0; };
        int cur = page_of(j0), nxt = j0 + 1 < j1 ? page_of(j0 + 1) : 0;
        const bool tail = 128 * j1 > q.kv - q.n;   // some of the piece's keys are nodes
        int32_t par[4] = {-1, -1, -1, -1};
        if (tail)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (lane + 32 * k < q.n) par[k] = p.parent[q.t0 + lane + 32 * k];
        // what is left of the piece before
        if (pv_have) ok = send(true, pv_np, pv_page, pv_hk);
        pv_have = false;
        // the query tiles
        if (lane == 0)
          for (int t = 0; t < qt && ok; ++t) {
            const int qb = qsel ^ t;
            ok = mbar_wait(&ct.q_empty[qb], (quse[qb] & 1) ^ 1, abort_flag, p.err, kErrWaitProducer);
            if (!ok) break;
            mbar_arrive_expect_tx(&ct.q_full[qb], C::NH * G * NT * 128);
            for (int ch = 0; ch < C::NH; ++ch)
              tma_load_3d(sQ + qb * C::QT_BYTES + ch * C::TILE_BYTES, &tmQ, &ct.q_full[qb], ch * 64, hk * G,
                          q.t0 + i0 + t * NT);
            ++quse[qb];
          }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        // the first K, then the piece's record for the other roles
        const int np0 = min(8, n_pages - 8 * j0);
        if (ok) ok = send(false, np0, cur, hk);
        const int ss = nseg % C::NSEG;
        if (ok) {
          if (lane == 0) ok = mbar_wait(&ct.seg_empty[ss], ((nseg / C::NSEG) & 1) ^ 1, abort_flag, p.err, kErrWaitProducer);
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (!ok) break;
        Seg &sg = ct.seg[ss];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = lane + 32 * k;
          if (i < q.n && tail) {
            if (par[k] < -1 || par[k] >= i) {
              atomicExch(p.err, kErrBounds);
              par[k] = -1;
            }
            sg.parent[i] = static_cast<uint8_t>(par[k]);
          }
        }
        if (lane < 4) sg.odd[lane] = 0;
        if (lane == 0) {
          sg.nb = j1 - j0;
          sg.j0 = j0;
          sg.qt = qt;
          sg.t0 = q.t0;
          sg.i0 = i0;
          sg.hk = hk;
          sg.c = q.kv - q.n;
          sg.kv = q.kv;
          sg.nodes = nodes;
          sg.slot = first == last ? -1 : 2 * cta + (cta == first ? 1 : 0);
          sg.qb = qsel;
          sg.b0 = q.b0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.seg_full[ss]);
        ++nseg;
        if (first != last && cta == first) {
          rec[0] = last - first + 1;
          rec[1] = q.t0;
          rec[2] = i0;
          rec[3] = hk;
          rec[4] = nodes * G;
        }
        if (qt == 1) qsel ^= 1;
        pv_np = np0;
        pv_page = cur;
        pv_hk = hk;
        pv_have = true;
        cur = nxt;
        nxt = j0 + 2 < j1 ? page_of(j0 + 2) : 0;
        for (int j = j0 + 1; j < j1 && ok; ++j) {
          const int np = min(8, n_pages - 8 * j);
          const int after = j + 2 < j1 ? page_of(j + 2) : 0;
          // With two tiles K's stages are held for long: a V that has one free
          // does not wait for the K before it (16 trees of 64 nodes at 8,192
          // keys 132 us against 141; with one tile it gained nothing).
          const bool v_first = qt == 2 && pv_have && room(true) && !room(false);
          if (v_first) ok = send(true, pv_np, pv_page, pv_hk);
          if (ok) ok = send(false, np, cur, hk);
          if (ok && pv_have && !v_first) ok = send(true, pv_np, pv_page, pv_hk);
          pv_np = np;
          pv_page = cur;
          pv_hk = hk;
          pv_have = true;
          cur = nxt;
          nxt = after;
        }
      }
      // the next unit on the line
      base += cost;
      if (++u == q.full + (q.rem ? 1 : 0)) {
        u = 0;
        if (++hk == p.Hkv) {
          hk = 0;
          do {
            ++r;
            if (r >= p.n_reqs) break;
            q = make_req(p, nx, &bad);
            if (r + 1 < p.n_reqs) nx = load_raw(p, r + 1);
          } while (q.n == 0);
          if (r >= p.n_reqs) break;
        }
      }
    }
    if (ok && pv_have) ok = send(true, pv_np, pv_page, pv_hk);
    if (lane == 0) {
      if (ok) {
        const int ss = nseg % C::NSEG;
        if (mbar_wait(&ct.seg_empty[ss], ((nseg / C::NSEG) & 1) ^ 1, abort_flag, p.err, kErrWaitProducer)) {
          ct.seg[ss].nb = 0;
          mbar_arrive(&ct.seg_full[ss]);
        }
      }
#pragma unroll
      for (int k = 0; k < 5; ++k) p.rec[cta * 8 + k] = rec[k];
      // after an abort, let copies in flight land before the CTA exits (bounded)
      if (!ok || *abort_flag) {
        const uint64_t t_start = globaltimer();
        auto drain = [&](uint64_t *bar, int use) {
          while (!mbar_try_wait(smem_u32(bar), use & 1) && globaltimer() - t_start < kWaitLimitNs) {
          }
        };
        for (int i = max(0, kcnt - C::NK); i < kcnt; ++i) drain(&ct.k_full[i % C::NK], i / C::NK);
        for (int i = max(0, vcnt - C::NV); i < vcnt; ++i) drain(&ct.v_full[i % C::NV], i / C::NV);
        for (int b = 0; b < 2; ++b)
          if (quse[b] > 0) drain(&ct.q_full[b], quse[b] - 1);
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    // Items in order: block by block, tile by tile.  S of an item goes out
    // as soon as its K (and Q) landed and the P V before the last one is
    // issued (its S buffer is then free, in order); P V as soon as P is
    // written and V landed.  S runs on into the next piece.  The whole warp
    // keeps the books, in step, and one elected lane issues.
    const uint64_t qd0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t kd0 = sdesc_sw128(smem_u32(sK), 16, C::ATOM_STRIDE);
    const uint64_t vd0 = sdesc_sw128(smem_u32(sV), 1024, C::ATOM_STRIDE);
    struct Cursor {
      int seg, blk, item;      // pieces, blocks and items before it
      int nb, qt, qb, lb, t;   // the piece, and the place in it
      bool in;
    };
    Cursor s{0, 0, 0, 0, 0, 0, 0, 0, false}, v{0, 0, 0, 0, 0, 0, 0, 0, false};
    int quse[2] = {0, 0};
    bool s_end = false;
    uint64_t t_idle = 0;
    auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    auto ready = [](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_test_wait(smem_u32(bar), parity)) != 0;
    };
    auto enter = [&](Cursor &x) {
      const Seg &sg = ct.seg[x.seg % C::NSEG];
      x.nb = uni(sg.nb);
      x.qt = uni(sg.qt);
      x.qb = uni(sg.qb);
      x.lb = x.t = 0;
      x.in = true;
    };
    for (uint32_t spin = 1;; ++spin) {   // rounds without progress
      bool progress = false;
      if (!s_end && s.item < v.item + 2) {
        if (!s.in && ready(&ct.seg_full[s.seg % C::NSEG], (s.seg / C::NSEG) & 1)) {
          enter(s);
          if (s.nb == 0) s_end = true;
        }
        if (s.in && !s_end) {
          const int qb = s.qb ^ s.t, st = s.blk % C::NK;
          if ((s.lb > 0 || ready(&ct.q_full[qb], quse[qb] & 1)) && ready(&ct.k_full[st], (s.blk / C::NK) & 1)) {
            tc_fence_after();
            const uint32_t d = tmem + 128 * (s.item & 1);
            const uint64_t qd = qd0 + static_cast<uint64_t>((qb * C::QT_BYTES) >> 4);
            const uint64_t kd = kd0 + static_cast<uint64_t>((st * C::KV_BYTES) >> 4);
            const bool last = s.lb == s.nb - 1, k_done = s.t + 1 == s.qt;
            if (elect_one()) {
#pragma unroll
              for (int ch = 0; ch < C::NH; ++ch)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_bf16(d, qd + ((ch * C::TILE_BYTES + kk * 32) >> 4), kd + ((ch * 1024 + kk * 32) >> 4), C::IDESC_S,
                           (ch > 0 || kk > 0) ? 1u : 0u);
              mma_commit(&ct.s_full[s.item & 1]);
              if (last) mma_commit(&ct.q_empty[qb]);
              if (k_done) mma_commit(&ct.k_empty[st]);
            }
            __syncwarp();
            if (last) ++quse[qb];
            ++s.item;
            if (++s.t == s.qt) {
              s.t = 0;
              ++s.blk;
              if (++s.lb == s.nb) {
                s.in = false;
                ++s.seg;
              }
            }
            progress = true;
          }
        }
      }
      if (v.item < s.item) {
        if (!v.in) enter(v);   // S of the piece is out: its record is there
        const int st = v.blk % C::NV;
        if (ready(&ct.p_full[v.item & 1], (v.item >> 1) & 1) && ready(&ct.v_full[st], (v.blk / C::NV) & 1)) {
          tc_fence_after();
          const uint64_t vd = vd0 + static_cast<uint64_t>((st * C::KV_BYTES) >> 4);
          const int w = v.item & 1;               // warp group, S buffer, O accumulator
          const uint32_t pcol = tmem + 128 * w;
          const bool first = v.lb < (v.qt == 1 ? 2 : 1);   // the group's first block of the piece
          const bool v_done = v.t + 1 == v.qt, last = v_done && v.lb + 1 == v.nb;
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)   // 16 keys (two atoms) per MMA; hd halves 1 KB apart
              mma_bf16_ts(tmem + C::O_COL + HD * w, pcol + ks * 8, vd + ((ks * 2 * C::ATOM_STRIDE) >> 4), C::IDESC_PV,
                          (!first || ks > 0) ? 1u : 0u);
            mma_commit(&ct.o_full[w]);
            if (v_done) mma_commit(&ct.v_empty[st]);
            if (last) mbar_arrive(&ct.seg_empty[v.seg % C::NSEG]);
          }
          __syncwarp();
          ++v.item;
          if (++v.t == v.qt) {
            v.t = 0;
            ++v.blk;
            if (++v.lb == v.nb) {
              v.in = false;
              ++v.seg;
            }
          }
          progress = true;
        }
      }
      if (s_end && v.item == s.item) break;
      if (progress) {
        spin = 0;
        t_idle = 0;
      } else if ((spin & 255u) == 0) {
        if (t_idle == 0) t_idle = globaltimer();
        const bool late = globaltimer() - t_idle > kWaitLimitNs;
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
          if (__any_sync(0xffffffffu, late) && lane == 0) {
            *abort_flag = 1;
            atomicExch(p.err, kErrWaitMma);
          }
          break;
        }
      }
    }
    // every MMA issued above has completed before TMEM is freed
    if (elect_one()) mma_commit(&ct.done);
    __syncwarp();
    const uint64_t t_end = globaltimer();
    while (!mbar_try_wait(smem_u32(&ct.done), 0) && globaltimer() - t_end < kWaitLimitNs) {
    }
    __syncwarp();
  } else {
    // ------------------------------------------------- softmax / epilogue
    const int w = (warp - 2) >> 2;          // warp group: it takes every second item
    const int qu = warp & 3;                // TMEM lane quarter
    const int row = qu * 32 + lane;         // row of the tile; also the key of a block it looks after
    const uint32_t lane_base = static_cast<uint32_t>(qu * 32) << 16;
    const uint32_t s_col = tmem + lane_base + 128 * w;
    const uint32_t o_col = tmem + lane_base + C::O_COL + HD * w;
    const uint32_t o_other = tmem + lane_base + C::O_COL + HD * (w ^ 1);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    constexpr float kRescaleAbove = 8.f;    // log2 units
    const float scale = p.scale_log2;
    const float2 sc2 = make_float2(scale, scale);
    const int G = p.G, NT = 128 / G, row_node = row / G, row_head = row % G;
    int nseg = 0, item0 = 0, blk0 = 0;
    int lent[2] = {0, 0};     // times that group 0, 1 left its part of a piece to the other
    bool lending = false;     // the other group may still be reading this one's O and (m, l)
    bool ok = true;
    while (true) {
      const int ss = nseg % C::NSEG;
      bool fail = !mbar_wait(&ct.seg_full[ss], (nseg / C::NSEG) & 1, abort_flag, p.err, kErrWaitSoftmax);
      if (__any_sync(0xffffffffu, fail)) break;   // tcgen05.ld below is warp-collective
      Seg &sg = ct.seg[ss];
      const int nb = sg.nb;
      if (nb == 0) break;
      const int qt = sg.qt, j0 = sg.j0, c = sg.c, kv = sg.kv;
      const int items = nb * qt;
      const int lb0 = (item0 & 1) ^ w;       // this group's first item of the piece
      const int t = qt == 2 ? lb0 : 0;       // its query tile
      if (lb0 >= items) {                    // one block, and it is the other group's
        ++item0;
        ++blk0;
        ++nseg;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.seg_empty[ss]);
        continue;
      }
      const int rows = (t == 0 ? min(sg.nodes, NT) : sg.nodes - NT) * G;
      const bool idle = qu * 32 >= rows;     // no rows for this warp (it still looks after keys)
      const int node = sg.i0 + t * NT + row_node;
      // the nodes that this row's node sees
      uint4 see = make_uint4(0, 0, 0, 0);
      if (row < rows && 128 * (j0 + nb) > c)
        for (uint32_t x = node; x != 0xFF; x = sg.parent[x]) {
          const uint32_t bit = 1u << (x & 31), a = x >> 5;
          see.x |= a == 0 ? bit : 0;
          see.y |= a == 1 ? bit : 0;
          see.z |= a == 2 ? bit : 0;
          see.w |= a == 3 ? bit : 0;
        }
      float m_ref = -INFINITY, l = 0.f;
      for (int li = lb0; li < items; li += 2) {
        const int item = item0 + li, lb = qt == 2 ? li >> 1 : li;
        const int j = j0 + lb, key0 = 128 * j;
        fail = !mbar_wait(&ct.s_full[w], (item >> 1) & 1, abort_flag, p.err, kErrWaitSoftmax);
        if (__any_sync(0xffffffffu, fail)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool full = key0 + 128 <= c;   // only prefix keys: visible to every row
        if (!idle) {
          if (!full) mask_block(s_col, key0 - c, see);
          // The group's first block of the piece sets each row's reference
          // maximum.  From then on one pass over S while it holds; if a row of
          // the warp rose more than 2^8 above it, the reference moves, O is
          // rescaled and the probabilities are taken again from S, intact
          // until P is stored.
          uint32_t pk_lo[32], pk_hi[32];
          float2 lsum = make_float2(0.f, 0.f);
          float mq0 = -INFINITY, mq1 = -INFINITY, mq2 = -INFINITY, mq3 = -INFINITY;
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
          // (Always so.  As a condition it keeps the exponentials behind the
          // maxima: in one piece, 16 trees of 64 nodes took 145 us against 142.)
          const bool apart = nb > 0;
          float negm = m_ref == -INFINITY ? 0.f : -m_ref;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float sv[64];
            tmem_ld64(s_col + 64 * hh, sv);
#pragma unroll
            for (int e = 0; e < 64; e += 8) {
              mq0 = max3f(mq0, sv[e], sv[e + 1]);
              mq1 = max3f(mq1, sv[e + 2], sv[e + 3]);
              mq2 = max3f(mq2, sv[e + 4], sv[e + 5]);
              mq3 = max3f(mq3, sv[e + 6], sv[e + 7]);
            }
            if (apart) probs<64>(sv, sc2, negm, hh ? pk_hi : pk_lo, lsum);
          }
          const float mx = fmaxf(fmaxf(mq0, mq1), fmaxf(mq2, mq3)) * scale;
          const bool grow = mx > m_ref + kRescaleAbove;
          if (__any_sync(0xffffffffu, grow)) {
            if (li >= 2) {
              // O holds the group's blocks before: their P V must be done
              fail = !mbar_wait(&ct.o_full[w], ((item - 2) >> 1) & 1, abort_flag, p.err, kErrWaitSoftmax);
              if (__any_sync(0xffffffffu, fail)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const float alpha = grow ? ex2_approx(m_ref - mx) : 1.f;
#pragma unroll 1
              for (int cc = 0; cc < HD / 32; ++cc) {
                float v[32];
                tmem_ld32(o_col + cc * 32, v);
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] *= alpha;
                tmem_st32(o_col + cc * 32, v);
              }
              if (grow) l *= alpha;
            }
            if (grow) m_ref = mx;
            negm = m_ref == -INFINITY ? 0.f : -m_ref;   // a row that has seen nothing yet
            // P of 32 keys goes over 16 columns of S that have been read
            lsum = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              float sv[32];
              uint32_t pk[16];
              tmem_ld32(s_col + 32 * k, sv);
              probs<32>(sv, sc2, negm, pk, lsum);
              tmem_st16u(s_col + 16 * k, pk);
            }
          } else {
            // P over S: keys 0-63 in columns 0-31, keys 64-127 in 32-63
            tmem_st32u(s_col, pk_lo);
            tmem_st32u(s_col + 32, pk_hi);
          }
          l += lsum.x + lsum.y;
        }
        if (!full && t == 0) {
          // Keys that some row does not see: P is 0 there, but 0 times an
          // infinity or a NaN is not.  V rows past the request's last key hold
          // anything: zeroed.  A node's V row with a non-finite value is zeroed
          // too and the node marked; the rows that do see it add its part at the
          // end.  (Tile 0's warp group does it, before its P is ready; tile 1's
          // product with this block is issued after tile 0's.)
          const int vb = blk0 + lb;
          fail = !mbar_wait(&ct.v_full[vb % C::NV], (vb / C::NV) & 1, abort_flag, p.err, kErrWaitSoftmax);
          if (__any_sync(0xffffffffu, fail)) {
            ok = false;
            break;
          }
          const int key = key0 + row;
          uint8_t *vrow = sV + (vb % C::NV) * C::KV_BYTES + (row >> 3) * C::ATOM_STRIDE + (row & 7) * 128;
          bool wipe = key >= kv;
          if (key >= c && !wipe) {
            uint32_t special = 0;
#pragma unroll 1
            for (int ch = 0; ch < C::NH; ++ch)
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint4 x = *reinterpret_cast<const uint4 *>(vrow + ch * 1024 + ((k + lane) & 7) * 16);
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  special |= ((y[e] & 0x7F80u) == 0x7F80u || (y[e] & 0x7F800000u) == 0x7F800000u) ? 1u : 0u;
              }
            if (special) {
              wipe = true;
              atomicOr(&sg.odd[(key - c) >> 5], 1u << ((key - c) & 31));
            }
          }
          if (wipe) {
#pragma unroll
            for (int ch = 0; ch < C::NH; ++ch)
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4 *>(vrow + ch * 1024 + ((k + lane) & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
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
        tc_fence_before();
        mbar_arrive(&ct.p_full[w]);
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
          l = wa * l + wb * o.y;
          m_ref = M;
        }
        if (__any_sync(0xffffffffu, fail)) break;
        tc_fence_after();
        if (!idle) {
          const bool valid = row < rows;
          const bool odd = valid && ((sg.odd[0] & see.x) | (sg.odd[1] & see.y) | (sg.odd[2] & see.z) | (sg.odd[3] & see.w));
          const int tok = sg.t0 + node, head = sg.hk * G + row_head, slot = sg.slot;
          const float inv = 1.f / l;
          uint4 *dst = reinterpret_cast<uint4 *>(p.o + (static_cast<size_t>(tok) * p.Hq + head) * HD);
          // (partial rows in node order: tile 1's behind tile 0's)
          float *part = p.part + (static_cast<size_t>(max(slot, 0)) * 256 + t * NT * G + row) * (HD + 4);
          const Rows<HD> out{&p, &sg, see, tok, head, o_col, o_other, joint, valid && slot < 0, valid && slot >= 0,
                             wa, wb, inv, m_ref, dst, part};
          if (__any_sync(0xffffffffu, odd))
            write_odd<HD>(out, odd);
          else
            write_rows<HD, false>(out, false);
          if (valid && slot >= 0) *reinterpret_cast<float2 *>(part + HD) = make_float2(m_ref, l);
        }
        tc_fence_before();
        if (joint) mbar_arrive(&ct.ml_empty[w ^ 1]);
      }
      item0 += items;
      blk0 += nb;
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

// Merge of the units that were cut: CTA (w, y) takes every gridDim.y-th row
// group of the unit whose first piece CTA w computed.
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,   M = max_s m_s
// One warp takes a row, lane s holding piece s's (m, l); the first pieces' rows
// are loaded beside them, not after the weights are known (one tree of 6 nodes at
// 1,125 keys 12.5 us in all against 13.9, at 8,192 keys 16.5 against 18.8).
// Where there are many rows of few pieces, 8 lanes take a row and a warp four at
// a time (16 trees of 64 nodes at 8,192 keys, 256 rows a unit: 158 us in all
// against 165; one tree of 6 nodes, 24 rows of 8 pieces: 18 us against 13.6, so
// it is for more than 64 rows).
template <int HD>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  pdl_wait();
  pdl_trigger();
  const int w = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 rec = *reinterpret_cast<const int4 *>(p.rec + w * 8);
  const int rows = p.rec[w * 8 + 4];
  const int pieces = rec.x;
  if (pieces == 0) return;
  // piece 0 in slot 2 w + 1, piece s > 0 in slot 2 (w + s)
  auto src = [&](int s, int row) {
    return p.part + (static_cast<size_t>(s == 0 ? 2 * w + 1 : 2 * (w + s)) * 256 + row) * (HD + 4);
  };
  auto out = [&](int row) {
    const int tok = rec.y + rec.z + row / p.G, head = rec.w * p.G + row % p.G;
    return p.o + (static_cast<size_t>(tok) * p.Hq + head) * HD;
  };
  if (pieces <= 8 && rows > 64) {
    constexpr int PER = HD / 32;   // float4s of a lane: columns 4 (lane + 8 k)
    const int l8 = lane & 7;
    for (int row = (blockIdx.y * 8 + warp) * 4 + (lane >> 3); row < rows; row += gridDim.y * 32) {
      float M = -INFINITY, L = 0.f;
      float4 acc[PER];
#pragma unroll
      for (int k = 0; k < PER; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int s = 0; s < pieces; ++s) {
        const float *x = src(s, row);
        float4 v[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) v[k] = reinterpret_cast<const float4 *>(x)[l8 + 8 * k];
        const float2 ml = *reinterpret_cast<const float2 *>(x + HD);
        if (ml.x == -INFINITY) continue;   // the row saw nothing in this piece
        const float mn = fmaxf(M, ml.x);
        const float a = ex2_approx(M - mn), b = ex2_approx(ml.x - mn);
        M = mn;
        L = fmaf(L, a, b * ml.y);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          acc[k].x = fmaf(acc[k].x, a, b * v[k].x);
          acc[k].y = fmaf(acc[k].y, a, b * v[k].y);
          acc[k].z = fmaf(acc[k].z, a, b * v[k].z);
          acc[k].w = fmaf(acc[k].w, a, b * v[k].w);
        }
      }
      const float inv = 1.f / L;
      uint2 *dst = reinterpret_cast<uint2 *>(out(row));
#pragma unroll
      for (int k = 0; k < PER; ++k)
        dst[l8 + 8 * k] = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
    }
    return;
  }
  constexpr int PER = HD / 32;
  using Vec = typename std::conditional<HD == 128, float4, float2>::type;
  constexpr int AHEAD = 4;   // pieces whose rows are in flight together, from before their weights are known
  for (int row = blockIdx.y * 8 + warp; row < rows; row += gridDim.y * 8) {
    Vec x[AHEAD];
    auto fetch = [&](int s0) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (s0 + u < pieces) x[u] = reinterpret_cast<const Vec *>(src(s0 + u, row))[lane];
    };
    auto m_and_l = [&](int s) {
      return s < pieces ? *reinterpret_cast<const float2 *>(src(s, row) + HD) : make_float2(-INFINITY, 0.f);
    };
    float2 ml = m_and_l(lane);
    fetch(0);
    float M = ml.x;
    for (int s = lane + 32; s < pieces; s += 32) M = fmaxf(M, src(s, row)[HD]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float L = 0.f, acc[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[k] = 0.f;
    for (int s0 = 0; s0 < pieces; s0 += 32) {
      if (s0 > 0) ml = m_and_l(s0 + lane);
      const float wgt = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
      L = fmaf(wgt, ml.y, L);
      for (int s = 0; s < 32 && s0 + s < pieces; s += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const float ws = __shfl_sync(0xffffffffu, wgt, s + u);   // (0: no such piece, or the row saw nothing in it)
          const float *xf = reinterpret_cast<const float *>(&x[u]);
#pragma unroll
          for (int k = 0; k < PER; ++k) acc[k] = ws != 0.f ? fmaf(ws, xf[k], acc[k]) : acc[k];
        }
        fetch(s0 + s + AHEAD);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    const float inv = 1.f / L;
    uint32_t *dst = reinterpret_cast<uint32_t *>(out(row) + lane * PER);
#pragma unroll
    for (int k = 0; k < PER / 2; ++k) dst[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  }
}

template <int HD>
cudaError_t launch_tree(const CUtensorMap &tq, const CUtensorMap &tkv, const TreeParams &p, int ctas, cudaStream_t st) {
  using C = TreeCfg<HD>;
  cudaError_t e = ensure_max_smem(reinterpret_cast<const void *>(tree_kernel<HD>), C::SMEM);
  if (e == cudaSuccess) e = launch_pdl(tree_kernel<HD>, dim3(ctas), dim3(C::THREADS), C::SMEM, st, 1, tq, tkv, p);
  if (e == cudaSuccess) e = launch_pdl(tree_merge_kernel<HD>, dim3(ctas, 4), dim3(256), 0, st, 1, p);
  return e;
}

}  // namespace

size_t tree_workspace_bytes() {
  return kRecBytes + static_cast<size_t>(2) * kMaxTreeCtas * 256 * (128 + 4) * sizeof(float);
}

cudaError_t tree_attention_run(const TreeArgs &a, cudaStream_t st) {
  if (a.n_reqs <= 0 || a.T <= 0) return cudaSuccess;
  TreeParams p;
  p.o = static_cast<__nv_bfloat16 *>(a.o);
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.pool = static_cast<const __nv_bfloat16 *>(a.pool);
  p.qo_indptr = a.qo_indptr;
  p.kv_len = a.kv_len;
  p.bt_indptr = a.bt_indptr;
  p.bt = a.bt;
  p.parent = a.parent;
  p.is_tree = a.is_tree;
  p.n_reqs = a.n_reqs;
  p.T = a.T;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.num_pages = a.num_pages;
  p.scale_log2 = kLog2e / sqrtf(static_cast<float>(a.hd));
  p.rec = static_cast<int32_t *>(a.workspace);
  p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kRecBytes);
  p.err = a.err;
  CUtensorMap tq, tkv;
  const uint64_t hd = a.hd;
  const uint64_t dq[3] = {hd, static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.T)};
  const uint64_t sq[2] = {hd * 2, hd * 2 * a.Hq};
  const uint32_t bq[3] = {64, static_cast<uint32_t>(p.G), static_cast<uint32_t>(128 / p.G)};
  cudaError_t e = encode_tmap(&tq, a.q, 3, dq, sq, bq);
  if (e == cudaSuccess) e = encode_kv_tmap(&tkv, a.pool, static_cast<uint64_t>(a.num_pages) * 2 * a.Hkv, a.hd);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(device_sm_count(), kMaxTreeCtas);
  return a.hd == 128 ? launch_tree<128>(tq, tkv, p, ctas, st) : launch_tree<64>(tq, tkv, p, ctas, st);
}

}  // namespace mb
