// The linear layer's activations and their slopes in f32, two values at a
// time (packed f32 arithmetic: one issue slot for both).
//
// gelu(z) = z Phi(z).  With u = |z|, Phi(-u) = exp(-u^2 / 2) M(u), where
// M(u) = exp(u^2 / 2) Phi(-u) (Mills' ratio over sqrt(2 pi)) falls smoothly
// from 1/2, and gelu(z) = max(z, 0) - u Phi(-u): the negative tail keeps its
// relative accuracy, which 1 + erf does not, at one ex2 and one reciprocal.
// M is a polynomial in t = 1 / (1 + k u) fitted over [0, 14.6] by reweighted
// least squares at Chebyshev nodes: nine terms and k = 0.35 hold it to 3.2e-8
// relative (FINE; 3.5e-7 with f32 roundings), six and k = 0.3 to 9e-6, enough
// for results stored in bf16 (half a step: 2e-3).  FINE also carries the
// rounding of the exponent.
//
// u is held at 14.5, where Phi(-u) is below f32's range, and z at -120 where a
// sigmoid is: at an infinite z an activation is its limit.  NaN stays NaN.
#pragma once

#include <stdint.h>

namespace psk {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_SILU = 3 };

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 pair_of(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 ex2_pair(float2 x) { return make_float2(ex2_approx(x.x), ex2_approx(x.y)); }
__device__ __forceinline__ float2 rcp_pair(float2 x) { return make_float2(rcp_approx(x.x), rcp_approx(x.y)); }
__device__ __forceinline__ float2 neg_pair(float2 x) { return make_float2(-x.x, -x.y); }

// exp(-u^2 / 2).
template <bool FINE>
__device__ __forceinline__ float2 half_gauss(float2 u) {
  const float2 H = pair_of(-0.72134751081466675f);               // -log2(e) / 2
  const float2 s = __fmul2_rn(u, u);
  const float2 a = __fmul2_rn(s, H);
  float2 e = ex2_pair(a);
  if constexpr (FINE) {
    const float2 sl = __ffma2_rn(u, u, neg_pair(s));
    float2 al = __ffma2_rn(s, H, neg_pair(a));
    al = __ffma2_rn(sl, H, __ffma2_rn(s, pair_of(-9.62981494545545e-09f), al));
    e = __ffma2_rn(e, __fmul2_rn(al, pair_of(0.69314718f)), e);
  }
  return e;
}

// M(u).
template <bool FINE>
__device__ __forceinline__ float2 mills(float2 u) {
  const float2 t = rcp_pair(__ffma2_rn(pair_of(FINE ? 0.35f : 0.3f), u, pair_of(1.0f)));
  constexpr int N = FINE ? 9 : 6;
  const float c[9] = {FINE ? 0.1396212875843048f : 0.1200542002916336f, FINE ? 0.1398637443780899f : 0.11395768821239471f,
                      FINE ? 0.11981963366270065f : 0.14333337545394897f,
                      FINE ? 0.10555890202522278f : -0.015335111878812313f,
                      FINE ? -0.023227162659168243f : 0.21461747586727142f,
                      FINE ? 0.15934081375598907f : -0.0766231119632721f, -0.2558571696281433f, 0.1440395712852478f,
                      -0.02915963903069496f};
  float2 p = pair_of(c[N - 1]);
#pragma unroll
  for (int i = N - 2; i >= 0; --i) p = __ffma2_rn(p, t, pair_of(c[i]));
  return __fmul2_rn(p, t);
}

// 1 / (1 + exp(-z)) for z above -120 (0 where exp(-z) leaves f32's range).
template <bool FINE>
__device__ __forceinline__ float2 sigmoid(float2 z) {
  const float2 L = pair_of(-1.44269502162933349609f);
  const float2 a = __fmul2_rn(z, L);
  float2 e = ex2_pair(a);
  if constexpr (FINE) {
    const float2 al = __ffma2_rn(z, pair_of(-1.92596298909109e-8f), __ffma2_rn(z, L, neg_pair(a)));
    const float2 f = __ffma2_rn(e, __fmul2_rn(al, pair_of(0.69314718f)), e);
    e.x = a.x > 126.0f ? e.x : f.x, e.y = a.y > 126.0f ? e.y : f.y;       // an infinite e has no correction
  }
  return rcp_pair(__fadd2_rn(pair_of(1.0f), e));
}

// silu far below zero, z exp(z) with the exponential in two halves: as one it
// would leave ex2's range (2^-126) where the product is still in f32's.
__device__ __forceinline__ float silu_far(float z) {
  z = max_nan(z, -120.0f);
  const float a = z * 0.72134751081466675f;                               // log2(e) / 2
  const float al = fmaf(z, 9.62981494545545e-9f, fmaf(z, 0.72134751081466675f, -a));
  float h = ex2_approx(a);
  h = fmaf(h, al * 0.69314718f, h);
  return z * h * h;
}
constexpr float SILU_FAR = -64.0f;         // from here on 1 / (1 + exp(-z)) is exp(z) (act_all looks for such z)

template <int ACT, bool FINE>
__device__ __forceinline__ float2 act_value(float2 z) {
  if constexpr (ACT == ACT_RELU) return make_float2(max_nan(z.x, 0.0f), max_nan(z.y, 0.0f));
  if constexpr (ACT == ACT_GELU) {
    const float2 u = make_float2(min_nan(fabsf(z.x), 14.5f), min_nan(fabsf(z.y), 14.5f));
    const float2 q = __fmul2_rn(half_gauss<FINE>(u), mills<FINE>(u));
    return __ffma2_rn(neg_pair(u), q, make_float2(fmaxf(z.x, 0.0f), fmaxf(z.y, 0.0f)));
  }
  if constexpr (ACT == ACT_SILU) {
    const float2 t = make_float2(max_nan(z.x, -120.0f), max_nan(z.y, -120.0f));
    const float2 c = make_float2(fminf(t.x, 120.0f), fminf(t.y, 120.0f));
    return __fmul2_rn(t, sigmoid<FINE>(c));
  }
  return z;
}

// gelu'(z) = Phi(z) + z phi(z) = 1/2 + sign(z) (1/2 - Phi(-u) + u phi(u)),
// silu'(z) = 1/2 + sign(z) (1/2 - o + u (1 - o) o) with o the sigmoid of -u:
// odd about 1/2, to f32's absolute accuracy (both stay below 1.13).
template <int ACT>
__device__ __forceinline__ float2 act_slope(float2 z) {
  if constexpr (ACT == ACT_RELU)
    return make_float2(z.x > 0.0f ? 1.0f : z.x != z.x ? z.x : 0.0f, z.y > 0.0f ? 1.0f : z.y != z.y ? z.y : 0.0f);
  if constexpr (ACT == ACT_GELU || ACT == ACT_SILU) {
    constexpr float TOP = ACT == ACT_GELU ? 14.5f : 120.0f;
    const float2 u = make_float2(min_nan(fabsf(z.x), TOP), min_nan(fabsf(z.y), TOP));
    float2 h;
    if constexpr (ACT == ACT_GELU) {
      const float2 g = half_gauss<false>(u);
      h = __ffma2_rn(neg_pair(g), mills<true>(u), pair_of(0.5f));
      h = __ffma2_rn(__fmul2_rn(u, pair_of(0.39894228040143f)), g, h);
    } else {
      const float2 o = sigmoid<true>(neg_pair(u));
      h = __fadd2_rn(pair_of(0.5f), neg_pair(o));
      h = __ffma2_rn(__fmul2_rn(u, o), __fadd2_rn(pair_of(1.0f), neg_pair(o)), h);
    }
    const uint32_t sx = __float_as_uint(z.x) & 0x80000000u, sy = __float_as_uint(z.y) & 0x80000000u;
    return __fadd2_rn(pair_of(0.5f), make_float2(__uint_as_float(__float_as_uint(h.x) ^ sx),
                                                 __uint_as_float(__float_as_uint(h.y) ^ sy)));
  }
  return pair_of(1.0f);
}

}  // namespace psk
