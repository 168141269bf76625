// Layer norm and its backward pass for gfx950.
//
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   y  = xh * w + b,   xh = (x - mean) * rstd
//   dx = rstd * (gy - sum(gy) / C - xh * sum(gy xh) / C),  gy = dy * w
//   dw = sum over rows of dy * xh,  db = sum over rows of dy
//
// Statistics and formulas are float32; the variance is taken from the centred
// values (a difference of sums would cancel where |mean| >> the spread).
//
// A workgroup takes one row and reads it once per sum (the later reads come
// from cache), so any width works.  The weight's gradient sums over rows:
// each workgroup of a grid over (columns, row groups) adds every G-th row of
// its columns in registers and stores one partial row [2][C] of dw and db; a
// second launch adds the G partials in order.  No atomics: the same bits on
// every run.
#include "mx_device.h"
#include "mx_launch.h"

namespace mx {

namespace {

template <bool BF16>
__device__ __forceinline__ float ld1(const void* p, int64_t i) {
  if (BF16) return bf16lo(static_cast<const uint16_t*>(p)[i]);
  return static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void st1(void* p, int64_t i, float v) {
  if (BF16) static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16_rne(v);
  else static_cast<float*>(p)[i] = v;
}
__device__ __forceinline__ float ldw(const void* p, bool bf16, int64_t i) {
  return bf16 ? ld1<true>(p, i) : ld1<false>(p, i);
}

// Sum of v over the 64 lanes, in every lane: neighbours and quads by DPP, the
// 16-lane rows by mirrors, then the gfx950 row and half-wave swaps.
__device__ __forceinline__ float wave_sum(float v) {
#define MX_DPP_ADD(CTRL) \
  v = v + __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true))
  MX_DPP_ADD(0xB1);    // lane ^ 1
  MX_DPP_ADD(0x4E);    // lane ^ 2
  MX_DPP_ADD(0x141);   // the other quad of 8 lanes (half-row mirror)
  MX_DPP_ADD(0x140);   // the other half of 16 lanes (row mirror)
#undef MX_DPP_ADD
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const uint32_t t = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(t, t, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Sum of v over the WAVES waves of the workgroup, in every thread.
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if (WAVES == 1) return v;
  __syncthreads();                              // red may still be read by the previous sum
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int i = 1; i < WAVES; ++i) s = s + red[i];
  return s;
}

constexpr int LW = 4;                           // waves per row of the any-width kernels

// Workgroups of a kernel that takes one row per workgroup and pass.
unsigned row_grid(int64_t R) { return (unsigned)(R < (1 << 20) ? R : (1 << 20)); }

template <bool BF16>
__global__ __launch_bounds__(64 * LW) void k_norm_any(NormArgs a) {
  __shared__ float red[LW];
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + r * a.ldx * (BF16 ? 2 : 4);
    char* y = static_cast<char*>(a.y) + r * a.ldy * (BF16 ? 2 : 4);
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < a.C; c += 64 * LW) s = s + ld1<BF16>(x, c);
    const float mean = block_sum<LW>(s, red) / (float)a.C;
    float q = 0.0f;
    for (int64_t c = threadIdx.x; c < a.C; c += 64 * LW) {
      const float d = ld1<BF16>(x, c) - mean;
      q = __builtin_fmaf(d, d, q);
    }
    const float rstd = 1.0f / __builtin_sqrtf(block_sum<LW>(q, red) / (float)a.C + a.eps);
    // (y may be x: every element is read and written by the same thread)
    for (int64_t c = threadIdx.x; c < a.C; c += 64 * LW) {
      const float xh = (ld1<BF16>(x, c) - mean) * rstd;
      const float w = a.weight ? ldw(a.weight, a.w_bf16, c) : 1.0f;
      const float b = a.bias ? ldw(a.bias, a.w_bf16, c) : 0.0f;
      st1<BF16>(y, c, __builtin_fmaf(xh, w, b));
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

template <bool BF16>
__global__ __launch_bounds__(64 * LW) void k_norm_dx_any(NormBwdArgs a) {
  __shared__ float red[LW];
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const int es = BF16 ? 2 : 4;
    const char* x = static_cast<const char*>(a.x) + r * a.ldx * es;
    const char* dy = static_cast<const char*>(a.dy) + r * a.lddy * es;
    char* dx = static_cast<char*>(a.dx) + r * a.lddx * es;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < a.C; c += 64 * LW) {
      const float xh = (ld1<BF16>(x, c) - mean) * rstd;
      const float gy = ld1<BF16>(dy, c) * (a.weight ? ldw(a.weight, a.w_bf16, c) : 1.0f);
      s1 = s1 + gy;
      s2 = __builtin_fmaf(gy, xh, s2);
    }
    s1 = block_sum<LW>(s1, red) / (float)a.C;
    s2 = block_sum<LW>(s2, red) / (float)a.C;
    // (dx may be dy or x: every element is read and written by the same thread)
    for (int64_t c = threadIdx.x; c < a.C; c += 64 * LW) {
      const float xh = (ld1<BF16>(x, c) - mean) * rstd;
      const float gy = ld1<BF16>(dy, c) * (a.weight ? ldw(a.weight, a.w_bf16, c) : 1.0f);
      st1<BF16>(dx, c, rstd * ((gy - s1) - xh * s2));
    }
  }
}

// Partial sums of dw and db: thread = column, rows blockIdx.y, + G, + 2G, ...
template <bool BF16>
__global__ __launch_bounds__(256) void k_norm_dw_any(NormBwdArgs a, int G) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.C) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t r = blockIdx.y; r < a.R; r += G) {
    const float xh = (ld1<BF16>(a.x, r * a.ldx + c) - a.mean[r]) * a.rstd[r];
    const float dy = ld1<BF16>(a.dy, r * a.lddy + c);
    dw = __builtin_fmaf(dy, xh, dw);
    db = db + dy;
  }
  float* p = a.workspace + (int64_t)blockIdx.y * 2 * a.C;
  p[c] = dw;
  p[a.C + c] = db;
}

// dw and db from the G partial rows: 64 columns per workgroup, 16 waves each
// adding every 16th partial, their sums added in wave order.
__global__ __launch_bounds__(1024) void k_norm_dw_sum(const float* __restrict__ part, int G, int64_t C,
                                                      void* dweight, void* dbias, int w_bf16) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  void* const out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  float s = 0.0f;
  if (c < C)
    for (int g = w; g < G; g += 16) s = s + part[((int64_t)g * 2 + blockIdx.y) * C + c];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s = s + red[i][lane];
    if (w_bf16) st1<true>(out, c, s);
    else st1<false>(out, c, s);
  }
}

// Partial rows of dw and db: enough row groups to fill the chip, fewer where a
// partial row is itself long.
int64_t norm_groups(int64_t R, int64_t C) {
  const int64_t most = C <= 24576 ? 512 : 64;
  return R < most ? R : most;
}

}  // namespace

size_t norm_backward_workspace(int64_t R, int64_t C) {
  return (size_t)norm_groups(R, C) * 2 * (size_t)C * sizeof(float);
}

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t st) {
  if (a.R == 0 || a.C == 0) return hipSuccess;
  if (a.bf16) hipLaunchKernelGGL((k_norm_any<true>), dim3(row_grid(a.R)), dim3(64 * LW), 0, st, a);
  else hipLaunchKernelGGL((k_norm_any<false>), dim3(row_grid(a.R)), dim3(64 * LW), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(const NormBwdArgs& a, hipStream_t st) {
  if (a.C == 0) return hipSuccess;
  // the weight's gradients first: dx may be written over dy or x
  if (a.dweight || a.dbias) {
    const int G = (int)norm_groups(a.R, a.C);
    if (G > 0) {
      const dim3 grid((unsigned)((a.C + 255) / 256), (unsigned)G);
      if (a.bf16) hipLaunchKernelGGL((k_norm_dw_any<true>), grid, dim3(256), 0, st, a, G);
      else hipLaunchKernelGGL((k_norm_dw_any<false>), grid, dim3(256), 0, st, a, G);
    }
    hipLaunchKernelGGL(k_norm_dw_sum, dim3((unsigned)((a.C + 63) / 64), 2), dim3(1024), 0, st, a.workspace, G, a.C,
                       a.dweight, a.dbias, (int)a.w_bf16);
  }
  if (a.dx && a.R > 0) {
    if (a.bf16) hipLaunchKernelGGL((k_norm_dx_any<true>), dim3(row_grid(a.R)), dim3(64 * LW), 0, st, a);
    else hipLaunchKernelGGL((k_norm_dx_any<false>), dim3(row_grid(a.R)), dim3(64 * LW), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace mx
