// Device helpers shared by the latent-cache kernels.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "mb_kernels.h"
#include "mb_ptx.cuh"

namespace mb {
namespace dev {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxKeys = 1 << 24;   // keys of one request

// A request's words of the descriptor.
struct ReqWords {
  int q0, q1, kv, b0, b1;
};
__device__ __forceinline__ ReqWords load_req(const int32_t *qo_indptr, const int32_t *kv_len, const int32_t *bt_indptr, int r) {
  return {qo_indptr[r], qo_indptr[r + 1], kv_len[r], bt_indptr[r], bt_indptr[r + 1]};
}
// (compared before they are subtracted: the words may be anything)
__device__ __forceinline__ bool req_ok(const ReqWords &w, int T) {
  return w.q0 >= 0 && w.q1 >= w.q0 && w.q1 <= T && w.b0 >= 0 && w.b1 >= w.b0 && w.kv >= w.q1 - w.q0 && w.kv <= kMaxKeys &&
         (w.kv + kPage - 1) / kPage <= w.b1 - w.b0;
}

// max(a, b, c) in one instruction.
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

static __device__ __noinline__ int64_t div64_long(int64_t a, int64_t b) { return a / b; }
// a / b for a >= 0, b > 0: in 32 bits where both fit (a tenth of the time).
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : div64_long(a, b);
}

// After a wait that ran out: lets the copies or products that `bar` counts land, at
// most until the limit after t0, before the CTA exits.
__device__ __forceinline__ void drain(uint64_t *bar, int use, uint64_t t0) {
  while (!mbar_try_wait(smem_u32(bar), use & 1) && globaltimer() - t0 < kWaitLimitNs) {
  }
}

// Bytes from a 16-byte boundary (a multiple of 16), into L2.
__device__ __forceinline__ void l2_prefetch(const void *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ void store32(void *dst, const uint32_t *v) {   // 32 bytes from a boundary of them: a whole sector
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 32 bytes of an output, which need not begin on a boundary of them.
__device__ __forceinline__ void store_out(void *dst, const uint32_t *v) {
  if ((reinterpret_cast<uintptr_t>(dst) & 31u) == 0) {
    store32(dst, v);
  } else {
    reinterpret_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// Stores under a predicate.  (With an `if` each, stores of an unrolled loop became
// branches: 20 cycles a store of a warp instead of 16.)
__device__ __forceinline__ void store_if(bool yes, __nv_bfloat16 *dst, __nv_bfloat16 v) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.b16 [%0], %1;\n\t}" ::"l"(dst),
               "h"(__bfloat16_as_ushort(v)), "r"(static_cast<uint32_t>(yes))
               : "memory");
}
__device__ __forceinline__ void store_if(bool yes, float *dst, float v) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.f32 [%0], %1;\n\t}" ::"l"(dst), "f"(v),
               "r"(static_cast<uint32_t>(yes))
               : "memory");
}

// A tile of shared memory to global memory (part of the thread's current bulk group).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Zeroes a key's row, two parts of CHUNKS swizzled 128-byte chunks (1 KB apart), if
// `stale`, or if it holds an infinity or a NaN (then true).
template <int CHUNKS>
__device__ __noinline__ bool wipe_row(uint8_t *row0, uint8_t *row1, bool stale) {
  bool odd = false;
  if (!stale) {
    uint32_t special = 0;
#pragma unroll 1
    for (int c = 0; c < 2 * CHUNKS; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint8_t *at = (c < CHUNKS ? row0 : row1 - CHUNKS * 1024) + c * 1024;
        const uint4 x = *reinterpret_cast<const uint4 *>(at + ((k + threadIdx.x) & 7) * 16);
        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          special |= ((y[e] & 0x7F80u) == 0x7F80u || (y[e] & 0x7F800000u) == 0x7F800000u) ? 1u : 0u;
      }
    odd = special != 0;
  }
  if (stale || odd)
#pragma unroll 1
    for (int c = 0; c < 2 * CHUNKS; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint4 *>((c < CHUNKS ? row0 : row1 - CHUNKS * 1024) + c * 1024 + ((k + threadIdx.x) & 7) * 16) = make_uint4(0, 0, 0, 0);
  return odd;
}

}  // namespace dev
}  // namespace mb
