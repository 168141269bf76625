// The gated block's formula and its derivative (device side), shared by the
// kernels that end in it.
//
//   h  = act(gc) * v,            gc = min(g, limit), v = clamp(u, -limit, limit) + shift
//   dg = dh * v * act'(gc) * [g <= limit],   du = dh * act(gc) * [|u| <= limit]
//
// SiLU and the tanh form of GELU are both x * s with s = 1 / (1 + e^-z): z =
// alpha x, or z = 2 sqrt(2/pi) (x + 0.044715 x^3) since (1 + tanh(z/2)) / 2 =
// s(z); the derivative is s + x s (1 - s) z'.  e^-z and the reciprocal are the
// hardware's (V_EXP_F32, V_RCP_F32, 1 ulp each): with the roundings of z log2 e
// the error of s is at most (6 + 2 |z|) 2^-24 relative, (6 + 4 |z|) 2^-24 for the
// tanh form's cubic.  e^-z overflows to Inf for z < -88, where s becomes 0 and
// x s a signed zero.
//
// GELU's normal distribution function is 1 - q(x) for x > 0 and q(-x) below, with
// q(y) e^(y^2/2) = t P(t), t = 1 / (1 + 0.305 y): the left side falls smoothly from
// 1/2 as 1 / y, and P, of degree 7, is its minimax fit in relative error over y in
// [0, 14] (1.6 2^-24; e^(-y^2/2) is zero beyond), found by exchange in float64.
// With its float32 evaluation and the rounding of y^2 / 2 the error of q is at most
// (11 + 1.25 y^2) 2^-24 relative, in the tail too (a form of bounded absolute error,
// 1.5e-7, was off by 1e-2 at y = 8).  The exponential is also the density of the
// derivative, so GELU costs one exponential and one reciprocal like the others.
#pragma once

#include "mx_device.h"

namespace mx {

struct GateP {
  int act;
  float alpha, limit, shift;     // limit +inf: no clamp
  float alpha_log2e;             // alpha log2 e, rounded once
};

inline GateP gate_params(int act, float alpha, float limit, float shift) {
  return GateP{act, alpha, limit, shift, (float)((double)alpha * 1.4426950408889634)};
}

// 1 / (1 + 2^-y)
__device__ __forceinline__ float gate_sigmoid2(float y) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-y));
}

// act(x) for the mx_act value ACT, and with GRAD its derivative in d.
template <int ACT, bool GRAD>
__device__ __forceinline__ float gate_act(const GateP& p, float x, float& d) {
  if constexpr (ACT == 1) {                              // GELU
    // y^2 is capped where the exponential is already zero, so that an infinite
    // square never meets it
    const float e = __builtin_amdgcn_exp2f(__builtin_fminf(x * x, 512.0f) * -0.72134752044448170f);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(x), 0.305f, 1.0f));
    float q = __builtin_fmaf(t, 0.036699187f, -0.1529882848f);
    q = __builtin_fmaf(t, q, 0.1857168376f);
    q = __builtin_fmaf(t, q, -0.0379767753f);
    q = __builtin_fmaf(t, q, 0.1210216507f);
    q = __builtin_fmaf(t, q, 0.103420876f);
    q = __builtin_fmaf(t, q, 0.1224668175f);
    q = __builtin_fmaf(t, q, 0.121639736f);
    q = q * t * e;
    const float cdf = x > 0.0f ? 1.0f - q : q;
    if (GRAD) d = __builtin_fmaf(x * 0.39894228040143268f, e, cdf);
    return x * cdf;
  } else {
    float s, dz;
    if constexpr (ACT == 2) {                            // GELU, tanh form
      // s is exactly 0 or 1 well inside |x| = 16, so the polynomial may stop
      // there; NaN stays in the factor x
      const float c = __builtin_amdgcn_fmed3f(x, -16.0f, 16.0f), c2 = c * c;
      s = gate_sigmoid2(c * __builtin_fmaf(0.10294324f, c2, 2.30220818f));   // z log2 e
      dz = __builtin_fmaf(0.21406498f, c2, 1.59576912f);
    } else {                                             // SiLU
      s = gate_sigmoid2(p.alpha_log2e * x);
      dz = p.alpha;
    }
    const float a = x * s;
    if (GRAD) d = __builtin_fmaf(a, (1.0f - s) * dz, s);
    return a;
  }
}

// Clamps that keep NaN (V_MINIMUM3_F32, V_MAXIMUM3_F32).
__device__ __forceinline__ float gate_low(float x, float lim) { return __builtin_elementwise_minimum(x, lim); }
__device__ __forceinline__ float gate_clamp(float x, float lim) {
  return __builtin_elementwise_minimum(__builtin_elementwise_maximum(x, -lim), lim);
}

template <int ACT>
__device__ __forceinline__ float gate_forward(const GateP& p, float g, float u) {
  float d;
  return gate_act<ACT, false>(p, gate_low(g, p.limit), d) * (gate_clamp(u, p.limit) + p.shift);
}

// NaN in either projection makes both gradients NaN, past a clamp too: the zero
// there is z, NaN where u is (a limit that is passed is finite, and with it the
// clamped u), and du's takes the factor that is NaN where g is.
template <int ACT>
__device__ __forceinline__ void gate_backward(const GateP& p, float g, float u, float dh, float& dg, float& du) {
  float d;
  const float a = gate_act<ACT, true>(p, gate_low(g, p.limit), d), c = gate_clamp(u, p.limit);
  const float z = c - c;
  dg = g > p.limit ? z : dh * (c + p.shift) * d;
  du = __builtin_fabsf(u) <= p.limit ? dh * a : z * a;
}

}  // namespace mx
