// Exponentials for sampling, accurate far beyond fp32, as fixed-point integers.
//
// The token that a random number picks from a distribution is the first whose
// cumulative weight passes it, so an error in the weights moves the borders
// between tokens, and a sum whose order depends on the launch moves them
// differently each time.  Here a weight 2^((l - m) k) (l <= m) is computed as
// a pair of floats hi + lo with relative error about 1e-11 and rounded to a
// multiple of 2^-40; sums of such integers are exact, so every split of a row
// over threads, warps and CTAs gives the same cumulative weights.
//
// Method: table-driven exponential (P. T. P. Tang, "Table-driven
// implementation of the exponential function in IEEE floating-point
// arithmetic", 1989): y = (l - m) k = n / 32 + f with |f| <= 1/64; 2^(n/32)
// from a 32-entry table (built on the host in double precision), 2^f - 1 from
// the first terms of its Taylor series, products and sums that matter carried
// with their rounding errors (T. J. Dekker, "A floating-point technique for
// extending the available precision", 1971).
#pragma once

#include <cmath>
#include <cstdint>

namespace mb {

constexpr int kFixBits = 40;

struct FixExpTable {
  float hi[32], lo[32];   // 2^(i/32)
};

inline FixExpTable fix_exp_table() {
  FixExpTable t;
  for (int i = 0; i < 32; ++i) {
    const double v = std::exp2(i / 32.0);
    t.hi[i] = static_cast<float>(v);
    t.lo[i] = static_cast<float>(v - static_cast<double>(t.hi[i]));
  }
  return t;
}

// 2^((l - m) k) as hi + lo, k = kh + kl >= 0, l <= m.  0 for a NaN or -inf
// logit and below 2^-48; l == m gives exactly 1 (m = +inf too).
__host__ __device__ __forceinline__ void fix_exp(float l, float m, float kh, float kl, const float *tab_hi,
                                                 const float *tab_lo, float *hi, float *lo) {
  constexpr float kLn2Hi = static_cast<float>(0.693147180559945309417);
  constexpr float kLn2Lo = static_cast<float>(0.693147180559945309417 - static_cast<double>(kLn2Hi));
  if (l == m) {
    *hi = 1.f;
    *lo = 0.f;
    return;
  }
  const float d = l - m;
  const float yh = d * kh;
  if (!(yh > -48.f)) {
    *hi = *lo = 0.f;
    return;
  }
  const float bb = d - l;
  const float de = (l - (d - bb)) - (m + bb);   // d + de = l - m exactly
  const float yl = fmaf(d, kh, -yh) + fmaf(d, kl, de * kh);
  const float n = rintf(yh * 32.f);
  const float f = fmaf(n, -0.03125f, yh);       // exact
  const float ph = f * kLn2Hi;
  const float r = f * f * fmaf(f, fmaf(f, fmaf(f, 1.33335581e-3f, 9.61812911e-3f), 5.55041087e-2f), 2.40226507e-1f);
  const float w = yl * kLn2Hi;                  // 2^(f + yl) = 2^f (1 + yl ln 2)
  const float pl = fmaf(f, kLn2Hi, -ph) + fmaf(f, kLn2Lo, fmaf(w, ph + r, w));
  const float q = pl + r;
  const float mh = ph + q;
  const float ml = (ph - mh) + q;
  const int ni = static_cast<int>(n);
  const float th = tab_hi[ni & 31], tl = tab_lo[ni & 31];
  const float gh = th * mh;
  const float gl = fmaf(th, mh, -gh) + fmaf(th, ml, fmaf(tl, mh, tl));
  const float h = th + gh;
  const float e = ((th - h) + gh) + gl;
  union {
    int32_t i;
    float f;
  } sc;
  sc.i = (127 + (ni >> 5)) << 23;
  *hi = h * sc.f;
  *lo = e * sc.f;
}

// hi + lo (in [0, 2^10)) as a multiple of 2^-40, rounded to nearest.
__host__ __device__ __forceinline__ int64_t to_fix(float hi, float lo) {
  const float a = hi * 1048576.f;
  const float fl = floorf(a);
  const float rem = (a - fl) + lo * 1048576.f;
  return (static_cast<int64_t>(fl) << 20) + static_cast<int64_t>(static_cast<int32_t>(rintf(rem * 1048576.f)));
}

}  // namespace mb
