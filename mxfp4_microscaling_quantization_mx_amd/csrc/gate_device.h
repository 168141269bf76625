// The gated block's formula and its derivative (device side), shared by the
// kernels that end in it.
//
//   h  = act(gc) * v,            gc = min(g, limit), v = clamp(u, -limit, limit) + shift
//   dg = dh * v * act'(gc) * [g <= limit],   du = dh * act(gc) * [|u| <= limit]
//
// SiLU and the tanh form of GELU are both x * s with s = 1 / (1 + e^-z): z =
// alpha x, or z = 2 sqrt(2/pi) (x + 0.044715 x^3) since (1 + tanh(z/2)) / 2 =
// s(z); the derivative is s + x s (1 - s) z'.  e^-z and the reciprocal are the
// hardware's (V_EXP_F32, V_RCP_F32, 1 ulp each): with the rounding of z log2 e
// the error of s is about (2 + |z|) 2^-24 relative.  e^-z overflows to Inf for
// z < -88, where s becomes 0 and x s a signed zero.
//
// GELU's normal distribution function is 1 - q(x) for x > 0 and q(-x) below,
// q(y) = (a1 t + ... + a5 t^5) e^(-y^2/2) / 2, t = 1 / (1 + p y / sqrt 2):
// Abramowitz and Stegun, "Handbook of Mathematical Functions", 7.1.26, with
// |error| <= 0.75e-7.  Its exponential is also the density of the derivative,
// so GELU costs one exponential and one reciprocal like the others.
#pragma once

#include "mx_device.h"

namespace mx {

struct GateP {
  int act;
  float alpha, limit, shift;     // limit +inf: no clamp
};

__device__ __forceinline__ float gate_sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

// act(x) for the mx_act value ACT, and with GRAD its derivative in d.
template <int ACT, bool GRAD>
__device__ __forceinline__ float gate_act(const GateP& p, float x, float& d) {
  if constexpr (ACT == 1) {                              // GELU
    // y^2 is capped where the exponential is already zero, so that an infinite
    // square never meets it
    const float e = __builtin_amdgcn_exp2f(__builtin_fminf(x * x, 512.0f) * -0.72134752044448170f);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(x), 0.23164188775f, 1.0f));
    float q = __builtin_fmaf(t, 0.5307027145f, -0.7265760135f);
    q = __builtin_fmaf(t, q, 0.7107068705f);
    q = __builtin_fmaf(t, q, -0.1422483680f);
    q = __builtin_fmaf(t, q, 0.1274147960f);
    q = q * t * e;
    const float cdf = x > 0.0f ? 1.0f - q : q;
    if (GRAD) d = __builtin_fmaf(x * 0.39894228040143268f, e, cdf);
    return x * cdf;
  } else {
    float z, dz;
    if constexpr (ACT == 2) {                            // GELU, tanh form
      // s is exactly 0 or 1 well inside |x| = 16, so the polynomial may stop
      // there; NaN stays in the factor x
      const float c = __builtin_amdgcn_fmed3f(x, -16.0f, 16.0f), c2 = c * c;
      z = 1.59576912160573071f * __builtin_fmaf(0.044715f * c2, c, c);
      dz = 1.59576912160573071f * __builtin_fmaf(0.134145f, c2, 1.0f);
    } else {                                             // SiLU
      z = p.alpha * x;
      dz = p.alpha;
    }
    const float s = gate_sigmoid(z);
    if (GRAD) d = __builtin_fmaf(x, s * (1.0f - s) * dz, s);
    return x * s;
  }
}

// (the comparisons keep NaN)
template <int ACT>
__device__ __forceinline__ float gate_forward(const GateP& p, float g, float u) {
  const float gc = g > p.limit ? p.limit : g;
  const float uc = u > p.limit ? p.limit : u < -p.limit ? -p.limit : u;
  float d;
  return gate_act<ACT, false>(p, gc, d) * (uc + p.shift);
}

template <int ACT>
__device__ __forceinline__ void gate_backward(const GateP& p, float g, float u, float dh, float& dg, float& du) {
  const float gc = g > p.limit ? p.limit : g;
  const bool hi = u > p.limit, lo = u < -p.limit;
  const float uc = hi ? p.limit : lo ? -p.limit : u;
  float d;
  const float a = gate_act<ACT, true>(p, gc, d);
  dg = g > p.limit ? 0.0f : dh * (uc + p.shift) * d;
  du = hi || lo ? 0.0f : dh * a;
}

// The same with the activation chosen at run time.
__device__ __forceinline__ float gate_forward_any(const GateP& p, float g, float u) {
  return p.act == 0 ? gate_forward<0>(p, g, u) : p.act == 1 ? gate_forward<1>(p, g, u) : gate_forward<2>(p, g, u);
}
__device__ __forceinline__ void gate_backward_any(const GateP& p, float g, float u, float dh, float& dg, float& du) {
  if (p.act == 0) gate_backward<0>(p, g, u, dh, dg, du);
  else if (p.act == 1) gate_backward<1>(p, g, u, dh, dg, du);
  else gate_backward<2>(p, g, u, dh, dg, du);
}

}  // namespace mx
