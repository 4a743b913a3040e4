// Exponentials for sampling, accurate far beyond fp32, as fixed-point integers.
//
// The token that a random number picks from a distribution is the first whose
// cumulative weight passes it, so an error in the weights moves the borders
// between tokens, and a sum whose order depends on the launch moves them
// differently each time.  Here a weight 2^((l - m) k) (l <= m) is computed
// with a relative error of about 2^-30 and rounded to a multiple of 2^-41;
// sums of such integers are exact, so every split of a row over threads, warps
// and CTAs gives the same cumulative weights.
//
// Method: table-driven exponential (P. T. P. Tang, "Table-driven
// implementation of the exponential function in IEEE floating-point
// arithmetic", 1989): y = (l - m) k = n / 32 + f with |f| <= 1/64 (y as a sum
// of two floats); 2^(n/32) from a 32-entry table (built on the host in double
// precision; one entry per shared-memory bank, so lookups do not conflict),
// 2^f - 1 from the first four terms of its Taylor series in fp32: it is below
// 0.011, so its rounding is 2^-31 of the result.  The product is an integer
// from the table's entry on.
#pragma once

#include <cmath>
#include <cstdint>

namespace mb {

constexpr int kFixBits = 41;

struct FixExpTable {
  uint32_t fix[32];   // 2^(i/32) in units of 2^-30
  float scaled[32];   // the same, as a float
};

inline FixExpTable fix_exp_table() {
  FixExpTable t;
  for (int i = 0; i < 32; ++i) {
    const double v = std::exp2(i / 32.0) * 0x1p30;
    t.fix[i] = static_cast<uint32_t>(std::lround(v));
    t.scaled[i] = static_cast<float>(v);
  }
  return t;
}

// 2^((l - m) k) in units of 2^-41, rounded to nearest; k = kh + kl >= 0, l <=
// m.  0 for a NaN or -inf logit; l == m gives exactly 1 (m = +inf too).  (l - m
// is a float; it is exact for bf16 logits unless |l| is below about 2^-16 m.)
__host__ __device__ __forceinline__ int64_t fix_exp(float l, float m, float kh, float kl, const uint32_t *tab_fix,
                                                    const float *tab_scaled) {
  constexpr float kMagic = 12582912.f;   // 1.5 2^23: a sum with it has its integer part in the low bits
  constexpr int32_t kMagicBits = 0x4B400000;
  constexpr float kC1 = 0.6931471806f, kC2 = 0.2402265070f, kC3 = 0.0555041087f, kC4 = 0.0096181291f;   // ln(2)^i / i!
  const float d = l - m;
  const float yh = fmaxf(d * kh, -48.f);   // (a NaN too: 2^-48 rounds to 0)
  const float yl = fmaf(d, kl, fmaf(d, kh, -yh));
  union {
    float f;
    int32_t i;
  } t;
  t.f = fmaf(yh, 32.f, kMagic);
  const float f = fmaf(t.f - kMagic, -0.03125f, yh) + (yh > -48.f ? yl : 0.f);
  const float g = f * fmaf(f, fmaf(f, fmaf(f, kC4, kC3), kC2), kC1);
  const int32_t i = t.i & 31, s = (kMagicBits - t.i + 31) >> 5;   // y = i / 32 - s + f, s >= 0
#ifdef __CUDA_ARCH__
  const int32_t add = __float2int_rn(tab_scaled[i] * g);
#else
  const int32_t add = static_cast<int32_t>(std::lrint(tab_scaled[i] * g));
#endif
  // units of 2^-42, then rounded to 2^-41
  const uint64_t w = static_cast<uint64_t>(tab_fix[i] + static_cast<uint32_t>(add)) << 12;
  return l == m ? int64_t{1} << kFixBits : static_cast<int64_t>(((w >> s) + 1) >> 1);
}

// hi + lo (hi in [0, 2]) in units of 2^-41, rounded to nearest.
__host__ __device__ __forceinline__ int64_t to_fix(float hi, float lo) {
  constexpr float kMagic = 12582912.f;
  constexpr int32_t kMagicBits = 0x4B400000;
  union {
    float f;
    int32_t i;
  } a, b;
  const float x = hi * 0x1p20f;
  a.f = x + kMagic;
  const float rem = (x - (a.f - kMagic)) + lo * 0x1p20f;
  b.f = fmaf(rem, 0x1p21f, kMagic);
  return (static_cast<int64_t>(a.i - kMagicBits) << 21) + (b.i - kMagicBits);
}

}  // namespace mb
