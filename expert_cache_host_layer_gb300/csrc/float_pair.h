// Numbers as the unevaluated sum of two floats, the second at most half an ulp
// of the first, and e^x, 1 / x and sigmoids of them, good to 2^-45 (against 113 bits
// the worst of 4 million sigmoids 2^-45.9, of softmax scores in rows of up to 1024
// values 2^-45.2).  (T. J. Dekker,
// "A floating-point technique for extending the available precision", 1971;
// D. E. Knuth's two-sum.)  On this GPU fp64 is slow: a warp's sigmoid takes
// 1600 cycles with its exponential and quotient, 730 with these and one fp64 sum.
// Internal to libft.
#pragma once

#include <cuda_runtime.h>

namespace ft {

struct FloatPair {
  float h, l;
};
// a + b and a * b exactly.
__device__ __forceinline__ FloatPair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ FloatPair two_product(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ FloatPair quick_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ FloatPair operator*(FloatPair a, FloatPair b) {
  const FloatPair p = two_product(a.h, b.h);
  return quick_sum(p.h, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.l, p.l)));
}
__device__ __forceinline__ FloatPair operator+(FloatPair a, FloatPair b) {
  const FloatPair s = two_sum(a.h, b.h);
  return quick_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ double wide(FloatPair a) { return (double)a.h + (double)a.l; }

// e^x for x in [-60, 0]: x = k ln 2 + r with ln 2 in three parts (k times the first is exact), |r| < 0.35, and the
// series to r^12 / 12!, of which the terms from r^7 on need no second float.
__device__ __forceinline__ FloatPair exp_pair(FloatPair x) {
  const float k = rintf(x.h * 1.44269504f);
  const FloatPair a = two_sum(x.h, -k * 0x1.62ep-1f), b = two_sum(a.h, x.l), c = two_product(k, -0x1.0bfbe8p-15f);
  const FloatPair d = two_sum(b.h, c.h);
  const FloatPair r = quick_sum(d.h, __fmaf_rn(k, -0x1.cf79acp-40f, __fadd_rn(d.l, __fadd_rn(__fadd_rn(a.l, b.l), c.l))));
  float p = 0x1.1eed8ep-29f;  // 1 / 12!
  p = __fmaf_rn(p, r.h, 0x1.ae6456p-26f);
  p = __fmaf_rn(p, r.h, 0x1.27e4fcp-22f);
  p = __fmaf_rn(p, r.h, 0x1.71de3ap-19f);
  p = __fmaf_rn(p, r.h, 0x1.a01a02p-16f);
  p = __fmaf_rn(p, r.h, 0x1.a01a02p-13f);
  const FloatPair t = two_product(r.h, p);
  // 1 / 6!, 1 / 5!, .. 1 / 0!
  constexpr float kHigh[7] = {0x1.6c16c2p-10f, 0x1.111112p-7f, 0x1.555556p-5f, 0x1.555556p-3f, 0.5f, 1.0f, 1.0f};
  constexpr float kLow[7] = {-0x1.27d27ep-35f, -0x1.dddddep-32f, -0x1.555556p-30f, -0x1.555556p-28f, 0.0f, 0.0f, 0.0f};
  FloatPair q{t.h, __fmaf_rn(r.l, p, t.l)};
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    if (i > 0) q = r * q;
    const FloatPair s = quick_sum(kHigh[i], q.h);
    q = quick_sum(s.h, __fadd_rn(s.l, __fadd_rn(kLow[i], q.l)));
  }
  const float scale = __int_as_float(((int)k + 127) << 23);
  return {q.h * scale, q.l * scale};
}
// 1 / x for x in [1, 2^60]: a quotient and two corrections by its remainder.
__device__ __forceinline__ FloatPair inverse(FloatPair x) {
  const float r = __frcp_rn(x.h);
  const FloatPair q = quick_sum(r, r * __fmaf_rn(-x.l, r, __fmaf_rn(-x.h, r, 1.0f)));
  const float e = __fmaf_rn(-x.h, q.l, __fmaf_rn(-x.l, q.h, __fmaf_rn(-x.h, q.h, 1.0f)));
  return quick_sum(q.h, __fmaf_rn(q.h, e, q.l));
}
// 1 / (1 + e^-x) for |x| <= 60.
__device__ __forceinline__ FloatPair sigmoid_pair(float x) {
  const FloatPair e = exp_pair({-fabsf(x), 0.0f}), i = inverse(FloatPair{1.0f, 0.0f} + e);
  return x < 0.0f ? e * i : i;
}

}  // namespace ft
