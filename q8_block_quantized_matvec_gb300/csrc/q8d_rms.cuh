// The factor 1 / sqrt(mean of squares + eps) of a root-mean-square norm, the
// same for every order in which the squares are added.
//
// An output in 8 or 4 bits is decided at borders between two codes, and a
// factor that is off by one unit in the last place moves one of about 10^5
// values across one.  The sum is therefore kept as an unevaluated pair of f32
// (hi, lo), each addition with its rounding error by Knuth's two-sum (Moller,
// Knuth; Dekker's pairs), what it leaves of a square by one fma: about 2^-44
// relative, so that the factor is 1 / sqrt in 64 bits rounded to f32 but
// for one row in 10^6.  That costs eight packed f32x2 instructions for two
// elements, four an element; the FP64 pipe takes half a clock of the SM for each.
#pragma once
#include "q8d_internal.cuh"

namespace q8d {

struct Pair {
  float hi, lo;
};

// p + v, the rounding error kept.
__device__ __forceinline__ void pair_add(Pair& p, float v) {
  const float t = __fadd_rn(p.hi, v);
  const float w = __fsub_rn(t, p.hi);
  const float e = __fadd_rn(__fsub_rn(p.hi, __fsub_rn(t, w)), __fsub_rn(v, w));
  p.hi = t;
  p.lo = __fadd_rn(p.lo, e);
}
__device__ __forceinline__ void pair_add(Pair& p, const Pair& o) {
  pair_add(p, o.hi);
  p.lo = __fadd_rn(p.lo, o.lo);
}
// Two sums side by side, in packed f32x2 arithmetic: p + v^2.  (v * v's own
// rounding needs no term: what t leaves of v^2 itself is one fma.)
struct Pair2 {
  uint64_t hi, lo;
};
__device__ __forceinline__ void pair2_add_square(Pair2& p, uint64_t v) {
  const uint64_t minus = 0xbf800000bf800000ull;  // -1, -1
  const uint64_t t = add2(p.hi, mul2(v, v));
  const uint64_t nw = fma2(t, minus, p.hi);  // -(t - hi)
  const uint64_t e = fma2(add2(t, nw), minus, p.hi);
  p.lo = add2(add2(p.lo, e), fma2(v, v, nw));
  p.hi = t;
}
__device__ __forceinline__ Pair pair2_join(const Pair2& p) {
  Pair a, b;
  unpack2(p.hi, a.hi, b.hi);
  unpack2(p.lo, a.lo, b.lo);
  pair_add(a, b);
  return a;
}
// p + q, the same whichever of two lanes adds: two-sum's error does not depend on
// the order, nor does the sum of the low parts.
__device__ __forceinline__ Pair pair_meet(const Pair& p, const Pair& q) {
  const float t = __fadd_rn(p.hi, q.hi);
  const float w = __fsub_rn(t, p.hi);
  const float e = __fadd_rn(__fsub_rn(p.hi, __fsub_rn(t, w)), __fsub_rn(q.hi, w));
  return {t, __fadd_rn(__fadd_rn(p.lo, q.lo), e)};
}
__device__ __forceinline__ Pair pair_shfl_xor(const Pair& p, int o, uint32_t mask) {
  return {__shfl_xor_sync(mask, p.hi, o), __shfl_xor_sync(mask, p.lo, o)};
}
// Sum over the lanes that differ in the bits below `width` (a power of two, at
// most 32); every one of them gets the same value.
__device__ __forceinline__ Pair pair_sum(Pair p, int width, uint32_t mask) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o >= width) break;
    p = pair_meet(p, pair_shfl_xor(p, o, mask));
  }
  return p;
}

// Sums outside these lose their squares' remainders below f32, or are no
// number, and above 2^100 the estimate's square loses its own: such rows are summed
// again in 64 bits.
__device__ __forceinline__ bool rms_in_range(const Pair& p, float eps) {
  return p.hi > 0x1p-80f && p.hi < 0x1p100f && eps < 0x1p100f;
}

// 1 / sqrt(ss / n + eps) rounded to f32; inv_n: 1 / n as a pair.  One Newton
// step on the hardware's estimate, its residual 1 - m y^2 in pairs.
__device__ __forceinline__ float rms_factor(const Pair& ss, const Pair& inv_n, float eps) {
  const float p = __fmul_rn(ss.hi, inv_n.hi);
  Pair m{p, __fmaf_rn(ss.hi, inv_n.hi, -p)};
  m.lo = __fmaf_rn(ss.hi, inv_n.lo, m.lo);
  m.lo = __fmaf_rn(ss.lo, inv_n.hi, m.lo);
  pair_add(m, eps);
  const float y = rsqrtf(m.hi);
  const float y2 = __fmul_rn(y, y), y2e = __fmaf_rn(y, y, -y2);
  const float q = __fmul_rn(m.hi, y2);
  float r = __fsub_rn(1.f, q);  // (exact: q is next to 1)
  r = __fsub_rn(r, __fmaf_rn(m.hi, y2, -q));
  r = __fmaf_rn(-m.hi, y2e, r);
  r = __fmaf_rn(-m.lo, y2, r);
  return __fmaf_rn(y, 0.5f * r, y);
}
// The same in 64 bits, for any sum.
__device__ __forceinline__ float rms_factor_wide(double ss, int n, float eps) {
  return (float)(1.0 / sqrt(ss / n + (double)eps));
}

inline Pair pair_inverse(int n) {
  const double v = 1.0 / n;
  Pair p;
  p.hi = (float)v;
  p.lo = (float)(v - p.hi);
  return p;
}

}  // namespace q8d
