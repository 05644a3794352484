// The linear layer's activations and their slopes in f32.
//
// gelu(z) = z Phi(z).  With u = |z|, Phi(-u) = exp(-u^2 / 2) M(u), where
// M(u) = exp(u^2 / 2) Phi(-u) (Mills' ratio over sqrt(2 pi)) falls smoothly
// from 1/2: a polynomial in t = 1 / (1 + 0.35 u) holds it to 3.2e-8 relative
// over [0, 14.6] (fitted here by reweighted least squares at Chebyshev nodes;
// 3.5e-7 with f32 roundings).  So the negative tail keeps its relative
// accuracy, which 1 + erf does not, at one ex2 and one reciprocal.
#pragma once

#include <stdint.h>

namespace psk {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_SILU = 3 };

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp(-u^2 / 2): the square and its product with log2(e) / 2 in two parts, so
// that the exponent's rounding (6e-6 at u = 13 otherwise) does not show.
__device__ __forceinline__ float half_gauss(float u) {
  const float H = -0.72134752044448170368f, HL = -9.62981494545545e-09f;   // -log2(e) / 2 in two floats
  const float s = u * u, sl = fmaf(u, u, -s);
  const float a = s * H;
  const float al = fmaf(s, H, -a) + fmaf(sl, H, s * HL);
  const float e = ex2_approx(a);
  return fmaf(e, al * 0.69314718f, e);
}

__device__ __forceinline__ float mills(float u) {
  const float t = rcp_approx(fmaf(0.35f, u, 1.0f));
  float p = -0.02915963903069496f;
  p = fmaf(p, t, 0.1440395712852478f);
  p = fmaf(p, t, -0.2558571696281433f);
  p = fmaf(p, t, 0.15934081375598907f);
  p = fmaf(p, t, -0.023227162659168243f);
  p = fmaf(p, t, 0.10555890202522278f);
  p = fmaf(p, t, 0.11981963366270065f);
  p = fmaf(p, t, 0.1398637443780899f);
  p = fmaf(p, t, 0.1396212875843048f);
  return p * t;
}

// 1 / (1 + exp(-z)); exp(-z) beyond f32's range gives 0.
__device__ __forceinline__ float sigmoid(float z) {
  const float a = z * -1.44269504088896f;
  const float al = fmaf(z, -1.44269504088896f, -a) + z * -1.9259629911e-8f;
  const float e = ex2_approx(a);
  const float d = 1.0f + fmaf(e, al * 0.69314718f, e);
  return e > 3.0e38f ? 0.0f : __frcp_rn(d);
}

// At an infinite z the limit: z where the function follows it, else 0.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
  if constexpr (ACT == ACT_GELU) {
    const float u = fabsf(z);
    const float q = half_gauss(u) * mills(u);
    const float v = z < 0.0f ? z * q : fmaf(-z, q, z);
    return u > 14.5f ? (z < 0.0f ? -0.0f : z) : v;
  }
  if constexpr (ACT == ACT_SILU) {
    const float v = z * sigmoid(z);
    return z < -120.0f ? -0.0f : z > 120.0f ? z : v;
  }
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if constexpr (ACT == ACT_GELU) {
    const float u = fabsf(z);
    const float g = half_gauss(u);
    const float q = g * mills(u);
    const float s = fmaf(z * 0.39894228040143f, g, z < 0.0f ? q : 1.0f - q);
    return u > 14.5f ? (z < 0.0f ? -0.0f : 1.0f) : s;
  }
  if constexpr (ACT == ACT_SILU) {
    const float s = sigmoid(z), o = sigmoid(-z);       // o = 1 - s without cancellation
    const float v = s * fmaf(z, o, 1.0f);
    return z < -120.0f ? -0.0f : z > 120.0f ? 1.0f : v;
  }
  return 1.0f;
}

}  // namespace psk
