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
// arithmetic", 1989): 32 (m - l) k = n - f with n the nearest integer (k is the
// sum of two floats; fused multiply-adds leave f without the product's
// rounding); 2^(-n/32) from a 32-entry table (built on the host in double
// precision; one entry per shared-memory bank, so lookups do not conflict),
// 2^(f/32) - 1 from the first four terms of its Taylor series in fp32: it is
// below 0.011, so its rounding is 2^-31 of the result.  The product is an
// integer from the table's entry on.
#pragma once

#include <cmath>
#include <cstdint>

namespace mb {

constexpr int64_t kFixOne = int64_t{1} << 41;   // a weight of 1

struct FixExpTable {
  uint32_t fix[32];   // 2^(-i/32 + (i > 0)), in [1, 2), in units of 2^-30
  float scaled[32];   // the same, as a float
};

inline FixExpTable fix_exp_table() {
  FixExpTable t;
  for (int i = 0; i < 32; ++i) {
    const double v = std::exp2((32 - i) % 32 / 32.0) * 0x1p30;
    t.fix[i] = static_cast<uint32_t>(std::lround(v));
    t.scaled[i] = static_cast<float>(v);
  }
  return t;
}

constexpr float kFixMagic = 12582912.f;   // 1.5 2^23: a sum with it has its integer part in the low bits
constexpr int32_t kFixMagicBits = 0x4B400000;
// (ln(2) / 32)^i / i!
constexpr float kFixC1 = static_cast<float>(0.69314718055994531 / 32), kFixC2 = static_cast<float>(0.24022650695910071 / 0x1p10),
                kFixC3 = static_cast<float>(0.055504108664821580 / 0x1p15),
                kFixC4 = static_cast<float>(0.0096181291076284772 / 0x1p20);

// 2^((l - m) k) to the same accuracy, before it is rounded to a multiple of
// 2^-41; k = kh + kl >= 0, l <= m.  0 for a NaN or -inf logit and below 2^-960;
// l == m gives exactly 1 (m = +inf too).  (l - m is a float; it is exact for
// bf16 logits unless |l| is below about 2^-16 m.)
__device__ __forceinline__ double fix_exp(float l, float m, float kh, float kl, const uint32_t *tab_fix,
                                          const float *tab_scaled) {
  if (l == m) return 1.0;
  const float d = m - l;
  if (!(d < fminf(960.f / fmaxf(kh, 1e-30f), 3e38f))) return 0.0;
  const float t = fmaf(d, 32.f * kh, kFixMagic);
  const float f = fmaf(d, -32.f * kl, fmaf(d, -32.f * kh, t - kFixMagic));
  const float g = f * fmaf(f, fmaf(f, fmaf(f, kFixC4, kFixC3), kFixC2), kFixC1);
  const int32_t n = __float_as_int(t), i = n & 31, s = (n - kFixMagicBits + 31) >> 5;   // the exponent: -s, and the table's
  const uint32_t v = tab_fix[i] + static_cast<uint32_t>(__float2int_rn(tab_scaled[i] * g));   // 2^30 2^(s + ...)
  return static_cast<double>(v) * __hiloint2double((1023 - 30 - s) << 20, 0);
}

}  // namespace mb
