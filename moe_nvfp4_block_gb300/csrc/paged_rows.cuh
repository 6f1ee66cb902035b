// paged_rows.cuh -- what the appends share: a row's sequence, and two-float
// arithmetic on bf16 pairs.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

// A sequence's rows [s0, s1) that are none of a call's T rows (no rows: anywhere).
__device__ __forceinline__ bool wrong_rows(int s0, int s1, int T) { return s0 != s1 && (s0 < 0 || s1 < s0 || s1 > T); }

// Row t's sequence: the last b with start[b] <= t, or -1.  With `wrong` rows
// somewhere the starts need not rise: the last right sequence that has t.
__device__ __forceinline__ int seq_of(const int* start, int n, int t, int T, bool wrong) {
  if (wrong) {
    for (int b = n - 1; b >= 0; --b)
      if (!wrong_rows(start[b], start[b + 1], T) && start[b] <= t && t < start[b + 1]) return b;
    return -1;
  }
  int lo = 0, hi = n + 1;  // start[lo - 1] <= t < start[hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1 < n ? lo - 1 : -1;
}

// Two floats, and two correctly rounded operations at a time.
typedef unsigned long long f2;
__device__ __forceinline__ f2 make_f2(float x, float y) {
  f2 p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ f2 unpack2(uint32_t w) { return make_f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ uint32_t pack2(f2 p) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
  return pack_bf16(x, y);
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// Cosine and sine of p f, each to little more than half an ulp and what the
// product's rounding moves the angle by (2^-53 of it: 1.5e-11 at 131,072, which
// counts only near a zero, and 2.4e-7 at 2^31), so that E4M3 codes are as far off
// as their rounding alone: the angle less its multiple of
// pi / 2 in double, as hi + lo in FP32; the Taylor series of sin and cos up to
// hi^9 and hi^10 (|hi| <= pi / 4: what follows is below 2^-28), their leading
// terms' rounding errors kept apart until the last sum; lo to first order.
__device__ __forceinline__ void rope_cs_fine(int p, double f, float& c, float& s) {
  const double th = (double)p * f;
  const double k = rint(th * 0.6366197723675814);  // 2 / pi
  double r = fma(-k, 1.5707963267948966, th);
  r = fma(-k, 6.123233995736766e-17, r);
  const float hi = (float)r, lo = (float)(r - (double)hi);
  const float z = __fmul_rn(hi, hi), ze = __fmaf_rn(hi, hi, -z), h = 0.5f * z;
  const float w = __fsub_rn(1.f, h), we = __fsub_rn(__fsub_rn(1.f, w), h);  // 1 - z / 2 = w + we
  float sp = __fmaf_rn(z, 1.f / 362880.f, -1.f / 5040.f);
  sp = __fmaf_rn(z, sp, 1.f / 120.f);
  sp = __fmaf_rn(z, sp, -1.f / 6.f);
  float cp = __fmaf_rn(z, -1.f / 3628800.f, 1.f / 40320.f);
  cp = __fmaf_rn(z, cp, -1.f / 720.f);
  cp = __fmaf_rn(z, cp, 1.f / 24.f);
  const float z3 = __fmul_rn(hi, z), z4 = __fmul_rn(z, z);
  const float s0 = __fmaf_rn(z3, sp, hi), c0 = __fmaf_rn(z4, cp, w);
  const float sr = __fadd_rn(hi, __fmaf_rn(z3, sp, __fmul_rn(lo, c0)));
  const float cr = __fadd_rn(w, __fadd_rn(we, __fmaf_rn(z4, cp, __fmaf_rn(-lo, s0, -0.5f * ze))));
  const int q = (int)__double2ll_rn(k) & 3;
  s = q & 1 ? cr : sr;
  c = q & 1 ? sr : cr;
  if (q & 2) s = -s;
  if ((q + 1) & 2) c = -c;
}
// 1 / sqrt(x), to little more than half an ulp: the approximation and one step
// of Newton's method on 1 - x y^2, formed with the product's rounding error.
// (Correctly rounded, it takes a fifth of what a head's norm does.)
__device__ __forceinline__ float inv_sqrt(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  const float t = __fmul_rn(x, y), te = __fmaf_rn(x, y, -t);
  const float e = __fmaf_rn(-te, y, __fmaf_rn(-t, y, 1.f));
  return x > 0x1p-120f && x < 0x1p120f ? __fmaf_rn(__fmul_rn(0.5f, y), e, y) : __frsqrt_rn(x);
}
__device__ __forceinline__ float sum2(f2 p) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
  return x + y;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint32_t& word(uint4& v, int i) { return reinterpret_cast<uint32_t*>(&v)[i]; }

}  // namespace

}  // namespace moe
