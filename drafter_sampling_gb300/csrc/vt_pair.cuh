// Numbers held as the unevaluated sum of two fp32 values, for the few places
// where 24 bits lose what matters and the fp64 pipe (1/64 of the fp32 rate on
// sm_103a) would be too slow.
#pragma once

#include "vt_common.cuh"

namespace vt {

struct Pair {
  float h, l;  // value h + l, |l| <= half a unit of h's last place
};

// a + b = s + e exactly
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = a + b;
  const float t = s - a;
  e = (a - (s - t)) + (b - t);
}
__device__ __forceinline__ Pair pair_of(float h, float l) {
  Pair r;
  two_sum(h, l, r.h, r.l);
  return r;
}
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  Pair r;
  float e;
  two_sum(a.h, b.h, r.h, e);
  return pair_of(r.h, e + (a.l + b.l));
}
__device__ __forceinline__ Pair pair_mul(Pair a, Pair b) {
  const float p = a.h * b.h;
  return pair_of(p, fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, a.l * b.h));
}

__device__ __forceinline__ Pair pair_neg(Pair a) { return Pair{-a.h, -a.l}; }
// a quotient, or product, or sum beyond fp32 is that infinity, or NaN, in h; l is of no use then
__device__ __forceinline__ Pair pair_div(Pair a, Pair b) {
  const float q = a.h / b.h;
  const float r = fmaf(-q, b.h, a.h) + fmaf(-q, b.l, a.l);
  return pair_of(q, r / b.h);
}

// e^x to a relative error below 2^-28 for -87 <= x.h <= 88; 0 below, +infinity
// above, NaN for NaN.  Cody and Waite's reduction x = n ln 2 + r with ln 2 as
// 16 bits (whose multiples by n are exact) and a remainder, |r| <= 0.35, then the
// Taylor series with 1, r and r^2 / 2 exact and the rest (below 0.008) in fp32
// (2.6e-9 is the largest of 2e7 arguments).
static __device__ __noinline__ Pair pair_exp(Pair x) {
  const float n = rintf(x.h * VT_LOG2E);
  float r, rl;
  two_sum(fmaf(n, -0.693145751953125f, x.h), fmaf(n, -1.42860682e-6f, x.l), r, rl);
  float p = 2.4801587e-5f;                     // 1 / 8!
  p = fmaf(p, r, 1.9841270e-4f);
  p = fmaf(p, r, 1.3888889e-3f);
  p = fmaf(p, r, 8.3333333e-3f);
  p = fmaf(p, r, 4.1666667e-2f);
  p = fmaf(p, r, 1.6666667e-1f);
  const float q = r * r, ql = fmaf(r, r, -q);
  float s, e1, e2;
  two_sum(1.f, r, s, e1);
  two_sum(s, 0.5f * q, s, e2);
  const float lo = e1 + e2 + fmaf(0.5f, ql, fmaf(p, q * r, fmaf(rl, r, rl)));
  Pair y = pair_of(s, lo);
  const float f = __int_as_float((max(-126, min(127, (int)n)) + 127) << 23);
  y.h *= f;
  y.l *= f;
  // (selections, so that several of these overlap)
  const bool in = x.h >= -87.f && x.h <= 88.f;
  y.h = in ? y.h : x.h > 88.f ? INFINITY : x.h < -87.f ? 0.f : x.h;
  y.l = in ? y.l : 0.f;
  return y;
}

// ln x of 1e-37 <= x <= 1e37, to 2^-27 in absolute terms: one Newton step on the fp32 logarithm
__device__ __forceinline__ Pair pair_log(Pair x) {
  const float y = logf(x.h);
  const Pair r = pair_add(pair_mul(x, pair_exp(Pair{-y, 0.f})), Pair{-1.f, 0.f});
  return pair_of(y, r.h + r.l);
}

}  // namespace vt
