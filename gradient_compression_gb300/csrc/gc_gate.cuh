// The sigmoids of the gated activations (sm_103a).
#pragma once

#include "gc_act.cuh"

namespace gc {

// sigmoid(p(g)) and p'(g): the activation is g * sigmoid(p(g)), its
// derivative s + g s (1 - s) p'(g).  The tanh form of GELU is of this kind
// since (1 + tanh z) / 2 = sigmoid(2 z).  The exponential turns an error of
// u |p| in p into a relative error of the result, |p| up to 87: the rounding
// errors of g^2 and of the last product are carried along in `low` and
// applied as exp(-(p + low)) = exp(-p) (1 - low).
constexpr float GELU_C = 1.5957691216057308f, GELU_CA = 0.0713548162726009f;  // 2 sqrt(2/pi), times 0.044715
// Beyond +-30 GELU's sigmoid is 0 or 1 in fp32; the clamp keeps g^3 and p'
// finite there, so that 0 * p' stays 0 (and lets a NaN through).
constexpr float GELU_FAR = 30.0f;

// For fp32 results: correctly rounded division and CUDA's expf.  Below -80,
// where 1 + exp(-p) is exp(-p) and soon overflows, the sigmoid is exp(p).
template <int KIND>
__device__ __forceinline__ float gate_sigmoid(float g, float* dp) {
  float p = g, low = 0.0f;
  *dp = 1.0f;
  if (KIND == GC_GATE_GELU_TANH) {
    const float t = fabsf(g) > GELU_FAR ? copysignf(GELU_FAR, g) : g;
    const float t2 = __fmul_rn(t, t), w = __fmaf_rn(GELU_CA, t2, GELU_C);
    p = __fmul_rn(w, t);
    low = __fmaf_rn(GELU_CA * __fmaf_rn(t, t, -t2), t, __fmaf_rn(w, t, -p));
    *dp = __fmaf_rn(2.0f * GELU_CA, t2, w);
  }
  const bool far = p < -80.0f;
  float e = expf(far ? p : -p);
  if (KIND == GC_GATE_GELU_TANH) e = __fmaf_rn(e, far ? low : -low, e);
  return far ? e : __fdiv_rn(1.0f, __fadd_rn(1.0f, e));
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// For 16-bit results, two at a time: the hardware's exponential and
// reciprocal, a few 2^-23 off (and |p| 2^-23 from SiLU's argument), are at most 2^-8
// of the result's own rounding and a third of the instructions.
// SiLU: with h = 2^(-g log2(e) / 2) the sigmoid is 1 / (1 + h^2), taken as
// 2^-64 / (2^-64 + (2^-32 h)^2): neither the sum overflows nor the reciprocal
// vanishes before the sigmoid is below all of fp32 (1 + e^-g itself is past
// the reciprocal's 2^126 from g = -87.3 on, where the product is still 1e-36).
// GELU: with h = 2^(-z/2), z = |p| log2(e), and f = h^2 the sigmoid is
// 1 / (1 + f) on the right and f / (1 + f) on the left, where nothing
// overflows and f reaches below 2^-126 (the exponential itself does not).
template <int KIND>
__device__ __forceinline__ F2 gate_sigmoid2(const float* g, F2* dp) {
  constexpr float LOG2E = 1.4426950408889634f;
  float x[2], r[2];
  if (KIND == GC_GATE_SILU) {
    constexpr float SMALL = 5.421010862427522e-20f, ROOT = 2.3283064365386963e-10f;  // 2^-64, 2^-32
    put2(x, mul2(get2(g), f2(-0.5f * LOG2E)));
    const F2 h = mul2(f2(ex2_ftz(x[0]), ex2_ftz(x[1])), f2(ROOT));
    put2(r, fma2(h, h, f2(SMALL)));
    *dp = f2(1.0f);
    return mul2(f2(rcp_ftz(r[0]), rcp_ftz(r[1])), f2(SMALL));
  }
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(x[0]) : "f"(fabsf(g[0])), "f"(GELU_FAR));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(x[1]) : "f"(fabsf(g[1])), "f"(GELU_FAR));
  const F2 t = get2(x), minus_t = mul2(t, f2(-1.0f)), minus_t2 = mul2(t, minus_t);
  const F2 w = fma2(minus_t2, f2(-0.5f * LOG2E * GELU_CA), f2(0.5f * LOG2E * GELU_C)), minus_z = mul2(w, minus_t);
  const F2 low = fma2(mul2(t, f2(0.5f * LOG2E * GELU_CA)), fma2(t, t, minus_t2), fma2(w, t, minus_z));
  *dp = fma2(minus_t2, f2(-3.0f * GELU_CA), f2(GELU_C));
  put2(x, minus_z);
  F2 h = f2(ex2_ftz(x[0]), ex2_ftz(x[1]));
  h = fma2(h, mul2(low, f2(-0.693147180559945f)), h);
  const F2 f = mul2(h, h);
  put2(x, fma2(h, h, f2(1.0f)));
  const F2 right = f2(rcp_ftz(x[0]), rcp_ftz(x[1]));
  put2(r, right), put2(x, mul2(f, right));
  return f2(g[0] < 0.0f ? x[0] : r[0], g[1] < 0.0f ? x[1] : r[1]);
}

}  // namespace gc
