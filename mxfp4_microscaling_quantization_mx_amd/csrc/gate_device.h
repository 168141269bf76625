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
#pragma once

#include "mx_device.h"

namespace mx {

struct GateP {
  int act, halves;
  float alpha, limit, shift;     // limit +inf: no clamp
};

__device__ __forceinline__ float gate_sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

// act(x), and with GRAD its derivative in d.
template <bool GRAD>
__device__ __forceinline__ float gate_act(const GateP& p, float x, float& d) {
  if (p.act == 1) {                                      // GELU
    const float cdf = __builtin_fmaf(0.5f, erff(x * 0.70710678118654752f), 0.5f);
    if (GRAD) {
      // x^2 is capped where the density is already zero, so that an infinite
      // square never meets it
      const float t = __builtin_fminf(x * x, 256.0f);
      d = __builtin_fmaf(x * 0.39894228040143268f, __builtin_amdgcn_exp2f(t * -0.72134752044448170f), cdf);
    }
    return x * cdf;
  }
  float z, dz;
  if (p.act == 2) {                                      // GELU, tanh form
    // s is exactly 0 or 1 well inside |x| = 16, so the polynomial may stop
    // there; NaN stays in the factor x
    const float c = __builtin_amdgcn_fmed3f(x, -16.0f, 16.0f), c2 = c * c;
    z = 1.59576912160573071f * __builtin_fmaf(0.044715f * c2, c, c);
    dz = 1.59576912160573071f * __builtin_fmaf(0.134145f, c2, 1.0f);
  } else {                                               // SiLU
    z = p.alpha * x;
    dz = p.alpha;
  }
  const float s = gate_sigmoid(z);
  if (GRAD) d = __builtin_fmaf(x, s * (1.0f - s) * dz, s);
  return x * s;
}

// (the comparisons keep NaN)
__device__ __forceinline__ float gate_forward(const GateP& p, float g, float u) {
  const float gc = g > p.limit ? p.limit : g;
  const float uc = u > p.limit ? p.limit : u < -p.limit ? -p.limit : u;
  float d;
  return gate_act<false>(p, gc, d) * (uc + p.shift);
}

__device__ __forceinline__ void gate_backward(const GateP& p, float g, float u, float dh, float& dg, float& du) {
  const float gc = g > p.limit ? p.limit : g;
  const bool hi = u > p.limit, lo = u < -p.limit;
  const float uc = hi ? p.limit : lo ? -p.limit : u;
  float d;
  const float a = gate_act<true>(p, gc, d);
  dg = g > p.limit ? 0.0f : dh * (uc + p.shift) * d;
  du = hi || lo ? 0.0f : dh * a;
}

}  // namespace mx
