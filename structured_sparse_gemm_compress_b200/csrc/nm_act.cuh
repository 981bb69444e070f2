// nm_act.cuh -- activations of the fused output stages, in fp32, and the packed
// pairs of fp32 values they are computed on.
//
// The GELU is the erf form x/2 (1 + erf(x / sqrt 2)), with erf evaluated by
// Abramowitz and Stegun's formula 7.1.26 (Handbook of Mathematical Functions,
// after Hastings): for u >= 0,
//   erfc(u) = (a1 t + a2 t^2 + a3 t^3 + a4 t^4 + a5 t^5) exp(-u^2) + e(u),
//   t = 1 / (1 + p u),  |e(u)| <= 1.5e-7,
// so that, with q = erfc(|x| / sqrt 2) / 2, GELU(x) = x (1 - q) for x >= 0 and
// x q for x < 0.  The reciprocal and the power of two are the hardware's
// approximate instructions (about 1 and 2 ulp); the whole function stays within
// |y - GELU(x)| <= 4e-7 |x| + 2e-6 |GELU(x)| of the exact value (checked by a
// dense sweep against fp64 in the tests).  Pairs of values go through the
// packed fp32 pipe (add/mul/fma .f32x2: each half is its own fp32 operation,
// rounded to nearest even), which halves the instruction count of the
// arithmetic; a single value takes the same operations in the same order, so
// both give identical results.
#pragma once
#include <cstdint>

#include "nm_device.cuh"

namespace nm {

namespace gelu_as {
constexpr float kP = 0.2316418883f;     // p / sqrt 2, p = 0.3275911
constexpr float kB1 = 0.127414796f;     // a_i / 2
constexpr float kB2 = -0.142248368f;
constexpr float kB3 = 0.7107068705f;
constexpr float kB4 = -0.7265760135f;
constexpr float kB5 = 0.5307027145f;
constexpr float kE = -0.7213475204f;    // -log2(e) / 2: exp(-x^2 / 2) = 2^(kE x^2)
}  // namespace gelu_as

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 values in one 64-bit register pair, and the packed operations on them.
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void upk2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

__device__ __forceinline__ float gelu1(float x) {
  using namespace gelu_as;
  const float ax = fabsf(x);
  const float t = rcp_approx(__fmaf_rn(ax, kP, 1.0f));
  float h = __fmaf_rn(t, kB5, kB4);
  h = __fmaf_rn(t, h, kB3);
  h = __fmaf_rn(t, h, kB2);
  h = __fmaf_rn(t, h, kB1);
  h = __fmul_rn(t, h);
  const float e = ex2_approx(__fmul_rn(x, __fmul_rn(x, kE)));
  const float q = __fmul_rn(h, e);
  return __fmul_rn(x, x >= 0.0f ? __fsub_rn(1.0f, q) : q);
}

// gelu1 of both halves of a pair.
__device__ __forceinline__ void gelu2(float& x0, float& x1) {
  using namespace gelu_as;
  const uint64_t x = pk2(x0, x1);
  const uint64_t d = fma2(pk2(fabsf(x0), fabsf(x1)), pk2(kP, kP), pk2(1.0f, 1.0f));
  float d0, d1;
  upk2(d, d0, d1);
  const uint64_t t = pk2(rcp_approx(d0), rcp_approx(d1));
  uint64_t h = fma2(t, pk2(kB5, kB5), pk2(kB4, kB4));
  h = fma2(t, h, pk2(kB3, kB3));
  h = fma2(t, h, pk2(kB2, kB2));
  h = fma2(t, h, pk2(kB1, kB1));
  h = mul2(t, h);
  float w0, w1;
  upk2(mul2(x, mul2(x, pk2(kE, kE))), w0, w1);
  float q0, q1;
  upk2(mul2(h, pk2(ex2_approx(w0), ex2_approx(w1))), q0, q1);
  float r0, r1;  // 1 - q (x >= 0) or q (x < 0)
  upk2(add2(pk2(1.0f, 1.0f), pk2(-q0, -q1)), r0, r1);
  upk2(mul2(x, pk2(x0 >= 0.0f ? r0 : q0, x1 >= 0.0f ? r1 : q1)), x0, x1);
}

// SiLU(x) = x / (1 + exp(-x)) with the approximate power of two and reciprocal:
// exp(-x) to 2 ulp plus the rounding of x log2(e) (1.2e-7 |x| relative), the
// reciprocal to 1 ulp; a power that overflows gives 0, one that vanishes gives x.
constexpr float kLog2e = 1.4426950409f;
__device__ __forceinline__ float sigmoid1(float x) { return rcp_approx(__fadd_rn(1.0f, ex2_approx(__fmul_rn(x, -kLog2e)))); }
// max(x, 0) that lets a NaN through.
__device__ __forceinline__ float relu1(float x) { return x < 0.0f ? 0.0f : x; }

// max(x, y), NaN if either is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// The GELU of the gated and the microscaled products: with Q(a) = Phi(-a), the upper
// tail of the normal distribution, GELU(x) = max(x, 0) - |x| Q(|x|).  log2 Q is nearly
// a parabola, so Q is one power of two of a polynomial: degree 6, fitted on [0, 5.5]
// for the least largest error relative to the bound above (which weighs an error of
// log2 Q by Q; linear program in a Chebyshev basis).  |Q - 2^r| <= 2.3e-7 there, and
// beyond r falls on like log2 Q (-51 at 8, -78 at 10, where |x| is cut off: +infinity
// gives itself, -infinity and all below -10 give -10 2^-78 = -3.3e-23).  6.5 instructions a value, one of them in the special
// function unit, where gelu2 takes 11.5 and two; same error bound (the fit takes 0.2 of
// it), other last bits: the older output stages keep gelu2.  4-bit product 12608 x
// 1024 -> 4096 with bias: 46.4 us against 52.5 with formula 7.1.26 in 9 instructions;
// gated 12608 x 768 -> 2 x 2048: 28.3 against 32.4.
namespace gelu_tail {
constexpr float kCut = 10.0f;
constexpr float kC0 = -0.9999994261f, kC1 = -1.151132361f, kC2 = -0.4589999361f, kC3 = -0.05308722621f,
                kC4 = 0.007860025568f, kC5 = -0.0006988590001f, kC6 = 2.468365636e-05f;
}  // namespace gelu_tail
__device__ __forceinline__ void gelu2_tail(float& x0, float& x1) {
  using namespace gelu_tail;
  const uint64_t na = pk2(max_nan(-fabsf(x0), -kCut), max_nan(-fabsf(x1), -kCut));  // -min(|x|, cut)
  uint64_t r = fma2(na, pk2(kC6, kC6), pk2(-kC5, -kC5));  // odd powers change sign with the argument
  r = fma2(na, r, pk2(kC4, kC4));
  r = fma2(na, r, pk2(-kC3, -kC3));
  r = fma2(na, r, pk2(kC2, kC2));
  r = fma2(na, r, pk2(-kC1, -kC1));
  r = fma2(na, r, pk2(kC0, kC0));
  float r0, r1;
  upk2(r, r0, r1);
  upk2(fma2(na, pk2(ex2_approx(r0), ex2_approx(r1)), pk2(max_nan(x0, 0.0f), max_nan(x1, 0.0f))), x0, x1);
}

// SiLU of a pair.
__device__ __forceinline__ void silu2(float& x0, float& x1) {
  const uint64_t x = pk2(x0, x1);
  float w0, w1;
  upk2(mul2(x, pk2(-kLog2e, -kLog2e)), w0, w1);
  float d0, d1;
  upk2(add2(pk2(ex2_approx(w0), ex2_approx(w1)), pk2(1.0f, 1.0f)), d0, d1);
  upk2(mul2(x, pk2(rcp_approx(d0), rcp_approx(d1))), x0, x1);
}

// act(x) of N values, one uniform branch around each activation's loop.
template <int N>
__device__ __forceinline__ void act_run(float* x, int act) {
  static_assert(N % 2 == 0, "values go in pairs");
  if (act == ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; i += 2) gelu2_tail(x[i], x[i + 1]);
  } else if (act == ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; i += 2) silu2(x[i], x[i + 1]);
  } else if (act == ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = relu1(x[i]);
  }
}

// a = act(x) and d = act'(x) (relu: 0 at 0).  GELU: with Phi the normal
// distribution function (formula 7.1.26 as above) and phi its density,
// a = x Phi(x), d = Phi(x) + x phi(x); both share the power of two.
constexpr float kInvSqrt2Pi = 0.3989422804f;
__device__ __forceinline__ void act_slope(float x, int act, float& a, float& d) {
  if (act == ACT_GELU) {
    using namespace gelu_as;
    const float t = rcp_approx(__fmaf_rn(fabsf(x), kP, 1.0f));
    float h = __fmaf_rn(t, kB5, kB4);
    h = __fmaf_rn(t, h, kB3);
    h = __fmaf_rn(t, h, kB2);
    h = __fmaf_rn(t, h, kB1);
    h = __fmul_rn(t, h);
    const float e = ex2_approx(__fmul_rn(x, __fmul_rn(x, kE)));
    const float q = __fmul_rn(h, e);
    const float cdf = x >= 0.0f ? __fsub_rn(1.0f, q) : q;
    a = __fmul_rn(x, cdf);
    d = __fmaf_rn(x, __fmul_rn(kInvSqrt2Pi, e), cdf);
  } else if (act == ACT_SILU) {
    const float s = sigmoid1(x);
    a = __fmul_rn(x, s);
    d = __fmul_rn(s, __fmaf_rn(x, __fsub_rn(1.0f, s), 1.0f));
  } else if (act == ACT_RELU) {
    a = relu1(x);
    d = x > 0.0f ? 1.0f : 0.0f;
  } else {
    a = x;
    d = 1.0f;
  }
}

}  // namespace nm
