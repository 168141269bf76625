// Layer norm and its backward pass for gfx950.
//
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   y  = xh * w + b,   xh = (x - mean) * rstd
//   dx = rstd * (gy - sum(gy) / C - xh * sum(gy xh) / C),  gy = dy * w
//   dw = sum over rows of dy * xh,  db = sum over rows of dy
//
// Statistics and formulas are float32, but for a row's mean, which is summed in
// double and subtracted in two float32 parts (Mean); the variance is taken from
// the centred values (a difference of sums would cancel where |mean| >> the
// spread).
//
// Both directions are bound by HBM bandwidth (bf16: 4 bytes per element
// forward, 6 backward; a device copy reaches 5.1 TB/s), so a row is read once
// and held in registers:
//  * k_norm: 1 to 8 waves per row, as few as leave a lane about 24 elements:
//    VEC consecutive ones (16 bytes where the rows allow it, else single
//    elements) of every NV-th piece of the row.  Workgroups of 8 waves walk
//    the rows; each lane keeps its weights in registers and requests a row
//    while the one before is worked on.  16384 x 2880 bf16: 38 us, 5.0 TB/s
//    (44 us with one row per wave, whose weights came through L2 each time);
//    the double sum is hidden behind the loads (37.7 with a float32 one).
//  * k_norm_backward: the same, one workgroup per CU (two lost 10 % to the
//    doubled partial rows), each lane also keeping its sums of dw and db; the
//    workgroup's row groups are added through LDS at the end and stored as one
//    partial row [2][C].  16384 x 2880 bf16: 51 us, 5.6 TB/s (72 us with one
//    wave per row, the weights read again and no row ahead), 57 with the sum of
//    the partial rows.  Rows that no 16-byte piece fits are read element by
//    element, as many loads in bf16 as in float32 and slower ones: 4099 x 1111
//    with a weight 17.9 us in float32 (3.1 TB/s; 15.4 without), 33.6 in bf16
//    (0.8); forward 9.5 and 12.8.
//  * k_norm_any, k_norm_dx_any, k_norm_dw_any: rows too long for registers,
//    read once per sum (the later reads come from cache), the weight's
//    gradient by columns.
// k_norm_dw_sum then adds the partial rows in order.  No atomics: the same
// bits on every run.
#include "mx_device.h"
#include "mx_launch.h"

#include <initializer_list>

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
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ float wave_sum(float v) {
#define MX_DPP_ADD(CTRL) v = v + __uint_as_float(dpp<CTRL>(__float_as_uint(v)))
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
__device__ __forceinline__ double from_words(uint32_t lo, uint32_t hi) {
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
#define MX_WORDS(V) const uint64_t q = __builtin_bit_cast(uint64_t, V); const uint32_t lo = (uint32_t)q, hi = (uint32_t)(q >> 32)
#define MX_DPP_ADD(CTRL) { MX_WORDS(v); v = v + from_words(dpp<CTRL>(lo), dpp<CTRL>(hi)); }
  MX_DPP_ADD(0xB1) MX_DPP_ADD(0x4E) MX_DPP_ADD(0x141) MX_DPP_ADD(0x140)
#undef MX_DPP_ADD
  {
    MX_WORDS(v);
    const auto a = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
    v = from_words(a[0], b[0]) + from_words(a[1], b[1]);
  }
  MX_WORDS(v);
#undef MX_WORDS
  const auto a = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
  return from_words(a[0], b[0]) + from_words(a[1], b[1]);
}

// Sum of v over the WAVES waves of the workgroup, in every thread.
template <int WAVES, class T>
__device__ __forceinline__ T block_sum(T v, T* red) {
  v = wave_sum(v);
  if (WAVES == 1) return v;
  __syncthreads();                              // red may still be read by the previous sum
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  T s = red[0];
#pragma unroll
  for (int i = 1; i < WAVES; ++i) s = s + red[i];
  return s;
}

// A row's mean from its sum, as a float32 and what that leaves: subtracting both
// keeps a centred value's error at its own roundings, where a float32 mean's 2^-24
// |mean| would be in every value of the row and stay (a row of one value must
// centre to zero).  The quotient is corrected to the last bit, so such a row's
// mean is its value.
struct Mean {
  float hi, lo;
  __device__ __forceinline__ float centre(float x) const { return (x - hi) - lo; }
};
__device__ __forceinline__ Mean row_mean(double sum, double C, double inv) {
  double m = sum * inv;
  m = __builtin_fma(__builtin_fma(-m, C, sum), inv, m);
  const float hi = (float)m;
  return {hi, (float)(m - (double)hi)};
}

constexpr int LW = 4;                           // waves per row of the any-width kernels

// Workgroups of a kernel that takes one row per workgroup and pass.
unsigned row_grid(int64_t R) { return (unsigned)(R < (1 << 20) ? R : (1 << 20)); }

template <bool BF16>
__global__ __launch_bounds__(64 * LW) void k_norm_any(NormArgs a) {
  __shared__ double redm[LW];
  __shared__ float red[LW];
  const double inv = 1.0 / (double)a.C;
  for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + r * a.ldx * (BF16 ? 2 : 4);
    char* y = static_cast<char*>(a.y) + r * a.ldy * (BF16 ? 2 : 4);
    double s = 0.0;
    for (int64_t c = threadIdx.x; c < a.C; c += 64 * LW) s = s + (double)ld1<BF16>(x, c);
    const Mean mean = row_mean(block_sum<LW>(s, redm), (double)a.C, inv);
    float q = 0.0f;
    for (int64_t c = threadIdx.x; c < a.C; c += 64 * LW) {
      const float d = mean.centre(ld1<BF16>(x, c));
      q = __builtin_fmaf(d, d, q);
    }
    const float rstd = 1.0f / __builtin_sqrtf(block_sum<LW>(q, red) / (float)a.C + a.eps);
    // (y may be x: every element is read and written by the same thread)
    for (int64_t c = threadIdx.x; c < a.C; c += 64 * LW) {
      const float xh = mean.centre(ld1<BF16>(x, c)) * rstd;
      const float w = a.weight ? ldw(a.weight, a.w_bf16, c) : 1.0f;
      const float b = a.bias ? ldw(a.bias, a.w_bf16, c) : 0.0f;
      st1<BF16>(y, c, __builtin_fmaf(xh, w, b));
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean.hi;
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

// ------------------------------------------------------------ rows in registers
// VEC consecutive elements at element i of a row (16 bytes, or one element).
// The row pointer is wave-uniform and i 32 bits, so one scalar base and one
// lane offset address the whole row.
template <bool BF16, int VEC>
struct Vec;
template <>
struct Vec<true, 8> {
  uint4 w;
  __device__ void load(const void* p, uint32_t i) {
    w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  }
  __device__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ float get(int k) const {
    const uint32_t v = (&w.x)[k >> 1];
    return (k & 1) ? bf16hi(v) : bf16lo(v);
  }
  static __device__ void store(void* p, uint32_t i, const float* f) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = (uint32_t)__builtin_bit_cast(unsigned short, (__bf16)f[2 * k]) |
             ((uint32_t)__builtin_bit_cast(unsigned short, (__bf16)f[2 * k + 1]) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(o[0], o[1], o[2], o[3]);
  }
};
template <>
struct Vec<false, 4> {
  float4 w;
  __device__ void load(const void* p, uint32_t i) { w = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i); }
  __device__ void zero() { w = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ float get(int k) const { return (&w.x)[k]; }
  static __device__ void store(void* p, uint32_t i, const float* f) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <bool BF16>
struct Vec<BF16, 1> {
  float w;
  __device__ void load(const void* p, uint32_t i) {
    w = BF16 ? bf16lo(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
  }
  __device__ void zero() { w = 0.0f; }
  __device__ float get(int) const { return w; }
  static __device__ void store(void* p, uint32_t i, const float* f) { st1<BF16>(p, i, f[0]); }
};

// VEC weight (or bias) entries at column c, or `none` without one.
template <int VEC>
__device__ __forceinline__ void load_param(const void* p, bool bf16, uint32_t c, float none, float f[VEC]) {
  if (!p) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[k] = none;
  } else if constexpr (VEC == 1) {
    f[0] = ldw(p, bf16, c);
  } else if (bf16) {
    uint32_t w[VEC / 2];
    if constexpr (VEC == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + c);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + c);
      w[0] = v.x, w[1] = v.y;
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[k] = (k & 1) ? bf16hi(w[k >> 1]) : bf16lo(w[k >> 1]);
  } else {
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) {
      const float4 v = reinterpret_cast<const float4*>(static_cast<const float*>(p) + c)[q];
      f[4 * q] = v.x, f[4 * q + 1] = v.y, f[4 * q + 2] = v.z, f[4 * q + 3] = v.w;
    }
  }
}

constexpr int BW = 8;                           // waves of a workgroup

// Two sums over a row group of WPR waves; red[2] alternates between the rows
// of a workgroup's walk, so one barrier per row is enough (a wave can write
// buffer i again only after the barrier of the row between, which every
// reader of buffer i has passed on its way to).
template <int WPR>
__device__ __forceinline__ void group_sum2(float& p, float& q, float2 (*red)[BW], int turn) {
  p = wave_sum(p);
  q = wave_sum(q);
  if (WPR == 1) return;
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) red[turn][w] = make_float2(p, q);
  __syncthreads();
  const int w0 = w / WPR * WPR;
  p = red[turn][w0].x;
  q = red[turn][w0].y;
#pragma unroll
  for (int i = 1; i < WPR; ++i) {
    p = p + red[turn][w0 + i].x;
    q = q + red[turn][w0 + i].y;
  }
}

template <int WPR, class T>
__device__ __forceinline__ T group_sum(T p, T (*red)[BW], int turn) {
  p = wave_sum(p);
  if (WPR == 1) return p;
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) red[turn][w] = p;
  __syncthreads();
  const int w0 = w / WPR * WPR;
  p = red[turn][w0];
#pragma unroll
  for (int i = 1; i < WPR; ++i) p = p + red[turn][w0 + i];
  return p;
}

// Each wave holds its columns of weight and bias, and requests a row while the
// row before it is worked on.
template <bool BF16, int VEC, int NV, int WPR>
__global__ __launch_bounds__(64 * BW) void k_norm(NormArgs a) {
  constexpr int RPB = BW / WPR, RL = 64 * WPR;  // row groups, lanes per row
  constexpr int ES = BF16 ? 2 : 4;
  __shared__ double redm[2][BW];                // mean and variance, each alternating
  __shared__ float redv[2][BW];
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x / RL);
  const uint32_t t = threadIdx.x % RL, C = (uint32_t)a.C;
  const double inv = 1.0 / (double)a.C;
  float w[NV * VEC], b[NV * VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const uint32_t c = (v * RL + t) * VEC;
    load_param<VEC>(c < C ? a.weight : nullptr, a.w_bf16, c, 1.0f, w + v * VEC);
    load_param<VEC>(c < C ? a.bias : nullptr, a.w_bf16, c, 0.0f, b + v * VEC);
  }
  Vec<BF16, VEC> next[NV];
  auto load = [&](int64_t r) {
    const char* const xr = static_cast<const char*>(a.x) + (r < a.R ? r : 0) * a.ldx * ES;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint32_t c = (v * RL + t) * VEC;
      if (r < a.R && c < C) next[v].load(xr, c);
      else next[v].zero();
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t base = (int64_t)blockIdx.x * RPB;
  load(base + sub);
  // every wave of the workgroup makes the same number of passes (they share
  // the barriers)
  for (int turn = 0; base < a.R; base += step, turn ^= 1) {
    const int64_t r = base + sub;
    float x[NV * VEC];
    double s = 0.0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        x[v * VEC + k] = next[v].get(k);
        s = s + (double)x[v * VEC + k];
      }
    if (base + step < a.R) load(r + step);
    const Mean mean = row_mean(group_sum<WPR>(s, redm, turn), (double)a.C, inv);
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const bool live = (v * RL + t) * VEC < C;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        x[v * VEC + k] = live ? mean.centre(x[v * VEC + k]) : 0.0f;
        q = __builtin_fmaf(x[v * VEC + k], x[v * VEC + k], q);
      }
    }
    const float rstd = 1.0f / __builtin_sqrtf(group_sum<WPR>(q, redv, turn) / (float)a.C + a.eps);
    if (r >= a.R) continue;
    char* const yr = static_cast<char*>(a.y) + r * a.ldy * ES;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint32_t c = (v * RL + t) * VEC;
      if (c < C) {
        float y[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          y[k] = __builtin_fmaf(x[v * VEC + k] * rstd, w[v * VEC + k], b[v * VEC + k]);
        Vec<BF16, VEC>::store(yr, c, y);
      }
    }
    if (t == 0) {
      if (a.mean) a.mean[r] = mean.hi;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

// Each wave holds its columns of the weight and its sums of dw and db over all
// its rows, and requests a row's x and dy while the row before it is worked on.
template <bool BF16, int VEC, int NV, int WPR>
__global__ __launch_bounds__(64 * BW) void k_norm_backward(NormBwdArgs a) {
  constexpr int RPB = BW / WPR, RL = 64 * WPR;  // row groups, lanes per row
  constexpr int ES = BF16 ? 2 : 4;
  constexpr int S = NV < 8 / VEC ? NV : 8 / VEC > 0 ? 8 / VEC : 1;   // pieces per LDS exchange at the end
  __shared__ float2 red[2][BW];
  __shared__ float part[2][RPB][RL * VEC * S];
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x / RL);
  const uint32_t t = threadIdx.x % RL, C = (uint32_t)a.C;
  const float inv = 1.0f / (float)a.C;
  float w[NV * VEC], dw[NV * VEC], db[NV * VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const uint32_t c = (v * RL + t) * VEC;
    load_param<VEC>(c < C ? a.weight : nullptr, a.w_bf16, c, 1.0f, w + v * VEC);
  }
#pragma unroll
  for (int k = 0; k < NV * VEC; ++k) dw[k] = db[k] = 0.0f;
  struct Row {
    Vec<BF16, VEC> x[NV], g[NV];
    float mean, rstd;
  };
  // a row group past the last row reads zeros, with mean = rstd = 0
  auto load = [&](Row& o, int64_t r) {
    const bool row = r < a.R;
    const int64_t at = row ? r : 0;
    o.mean = row ? a.mean[at] : 0.0f;
    o.rstd = row ? a.rstd[at] : 0.0f;
    const char* const xr = static_cast<const char*>(a.x) + at * a.ldx * ES;
    const char* const gr = static_cast<const char*>(a.dy) + at * a.lddy * ES;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint32_t c = (v * RL + t) * VEC;
      if (row && c < C) {
        o.x[v].load(xr, c);
        o.g[v].load(gr, c);
      } else {
        o.x[v].zero();
        o.g[v].zero();
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t base = (int64_t)blockIdx.x * RPB;
  Row next;
  load(next, base + sub);
  // every wave of the workgroup makes the same number of passes (they share
  // the barriers)
  for (int turn = 0; base < a.R; base += step, turn ^= 1) {
    const Row cur = next;
    const int64_t r = base + sub;
    if (base + step < a.R) load(next, r + step);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      // a row and a column past the end have dy = 0 and xh = 0 (0 - mean would
      // be, times rstd, an infinity where both are large)
      const float mean = (v * RL + t) * VEC < C ? cur.mean : 0.0f;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const int e = v * VEC + k;
        const float dy = cur.g[v].get(k), xh = (cur.x[v].get(k) - mean) * cur.rstd, gy = dy * w[e];
        s1 = s1 + gy;
        s2 = __builtin_fmaf(gy, xh, s2);
        dw[e] = __builtin_fmaf(dy, xh, dw[e]);
        db[e] = db[e] + dy;
      }
    }
    group_sum2<WPR>(s1, s2, red, turn);
    if (a.dx && r < a.R) {
      s1 = s1 * inv;
      s2 = s2 * inv;
      char* const dr = static_cast<char*>(a.dx) + r * a.lddx * ES;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const uint32_t c = (v * RL + t) * VEC;
        if (c < C) {
          float o[VEC];
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            const float xh = (cur.x[v].get(k) - cur.mean) * cur.rstd;
            o[k] = cur.rstd * ((cur.g[v].get(k) * w[v * VEC + k] - s1) - xh * s2);
          }
          Vec<BF16, VEC>::store(dr, c, o);
        }
      }
    }
  }
  if (!a.workspace) return;
  // the row groups' sums, S pieces at a time, added in group order; a launch
  // of one workgroup writes the results themselves
  const bool last = gridDim.x == 1;
  float* const out = a.workspace + (int64_t)blockIdx.x * 2 * a.C;
#pragma unroll
  for (int v0 = 0; v0 < NV; v0 += S) {
#pragma unroll
    for (int v = v0; v < v0 + S && v < NV; ++v)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        part[0][sub][((v - v0) * RL + t) * VEC + k] = dw[v * VEC + k];
        part[1][sub][((v - v0) * RL + t) * VEC + k] = db[v * VEC + k];
      }
    __syncthreads();
    constexpr int LEN = RL * VEC * S;
    for (int i = threadIdx.x; i < 2 * LEN; i += 64 * BW) {
      const int which = i / LEN, j = i - which * LEN, c = v0 * RL * VEC + j;
      if (c >= a.C || j >= (NV - v0) * RL * VEC) continue;
      float s = part[which][0][j];
#pragma unroll
      for (int q = 1; q < RPB; ++q) s = s + part[which][q][j];
      if (!last) {
        out[(int64_t)which * a.C + c] = s;
      } else if (void* const d = which ? a.dbias : a.dweight) {
        if (a.w_bf16) st1<true>(d, c, s);
        else st1<false>(d, c, s);
      }
    }
    __syncthreads();
  }
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
  if (c < C) {
    const float* const p = part + (int64_t)blockIdx.y * C + c;
    int g = w;
    for (; g + 7 * 16 < G; g += 8 * 16) {       // eight loads in flight
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = p[(int64_t)(g + 16 * k) * 2 * C];
#pragma unroll
      for (int k = 0; k < 8; ++k) s = s + v[k];
    }
    for (; g < G; g += 16) s = s + p[(int64_t)g * 2 * C];
  }
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s = s + red[i][lane];
    if (w_bf16) st1<true>(out, c, s);
    else st1<false>(out, c, s);
  }
}

// Workgroups of k_norm per CU: 16384 x 2880 bf16 41.6 us with 1, 37.7 with 2,
// 41.2 with 3; single elements per lane need more waves (4099 x 1111 bf16 on
// inputs in the caches 13.5 us with 2, 9.8 with 3, 9.2 with 4, 10.7 with 8).
template <int VEC>
constexpr int64_t norm_per_cu() { return VEC == 1 ? 4 : 2; }
// Most partial rows of dw and db: workgroups of k_norm_backward (one for each of
// the 256 CUs) and row groups of k_norm_dw_any.  A constant, so that the order of
// the sums does not follow the card.
constexpr int64_t MOST_GROUPS = 256;
int64_t norm_groups(int64_t R) { return R < MOST_GROUPS ? R : MOST_GROUPS; }

// Whether rows of C elements at these strides and addresses can be read 16
// bytes at a time, weights included.
bool norm_vec(int64_t C, bool bf16, std::initializer_list<int64_t> ld, std::initializer_list<const void*> p) {
  const int64_t vec = bf16 ? 8 : 4;
  bool ok = C % vec == 0;
  for (int64_t l : ld) ok = ok && l % vec == 0;
  for (const void* q : p) ok = ok && (uintptr_t)q % 16 == 0;
  return ok;
}

template <bool BF16, int VEC, int NV, int WPR>
int64_t start_norm(const NormArgs& a, hipStream_t st) {
  constexpr int RPB = BW / WPR;
  const int64_t want = (a.R + RPB - 1) / RPB, most = norm_per_cu<VEC>() * (int64_t)cu_count();
  hipLaunchKernelGGL((k_norm<BF16, VEC, NV, WPR>), dim3((unsigned)(want < most ? want : most)), dim3(64 * BW), 0, st,
                     a);
  return 1;
}

template <bool BF16, int VEC, int NV, int WPR>
int64_t start_norm_backward(const NormBwdArgs& a, hipStream_t st) {
  constexpr int RPB = BW / WPR;
  const int64_t G = norm_groups((a.R + RPB - 1) / RPB);
  hipLaunchKernelGGL((k_norm_backward<BF16, VEC, NV, WPR>), dim3((unsigned)G), dim3(64 * BW), 0, st, a);
  return G;
}

// Launch with the first of the compiled (pieces per lane, waves per row) that
// holds a row of C elements; 0 if the row is longer than all of them, else the
// launch's partial rows (backward).
#define MX_NV(K_, NV_, WPR_) \
  if (a.C <= (int64_t)(NV_) * VEC * 64 * (WPR_)) return K_<BF16, VEC, NV_, WPR_>(a, st);

template <bool BF16, int VEC>
int64_t try_norm(const NormArgs& a, hipStream_t st) {
  if constexpr (VEC == 8) {
    MX_NV(start_norm, 1, 1) MX_NV(start_norm, 2, 1) MX_NV(start_norm, 3, 1) MX_NV(start_norm, 2, 2)
    MX_NV(start_norm, 3, 2) MX_NV(start_norm, 2, 4) MX_NV(start_norm, 3, 4) MX_NV(start_norm, 2, 8)
    MX_NV(start_norm, 3, 8) MX_NV(start_norm, 4, 8) MX_NV(start_norm, 5, 8)
  } else if constexpr (VEC == 4) {
    MX_NV(start_norm, 1, 1) MX_NV(start_norm, 2, 1) MX_NV(start_norm, 4, 1) MX_NV(start_norm, 6, 1)
    MX_NV(start_norm, 4, 2) MX_NV(start_norm, 6, 2) MX_NV(start_norm, 4, 4) MX_NV(start_norm, 6, 4)
    MX_NV(start_norm, 4, 8) MX_NV(start_norm, 6, 8) MX_NV(start_norm, 8, 8)
  } else {
    MX_NV(start_norm, 2, 1) MX_NV(start_norm, 4, 1) MX_NV(start_norm, 8, 1) MX_NV(start_norm, 6, 2)
    MX_NV(start_norm, 9, 2) MX_NV(start_norm, 6, 4) MX_NV(start_norm, 9, 4) MX_NV(start_norm, 6, 8)
    MX_NV(start_norm, 9, 8) MX_NV(start_norm, 12, 8) MX_NV(start_norm, 18, 8) MX_NV(start_norm, 24, 8)
  }
  return 0;
}

template <bool BF16, int VEC>
int64_t try_norm_backward(const NormBwdArgs& a, hipStream_t st) {
  if constexpr (VEC == 8) {
    MX_NV(start_norm_backward, 1, 1) MX_NV(start_norm_backward, 2, 1) MX_NV(start_norm_backward, 3, 1)
    MX_NV(start_norm_backward, 2, 2) MX_NV(start_norm_backward, 3, 2) MX_NV(start_norm_backward, 2, 4)
    MX_NV(start_norm_backward, 3, 4) MX_NV(start_norm_backward, 2, 8) MX_NV(start_norm_backward, 3, 8)
    MX_NV(start_norm_backward, 4, 8)
  } else if constexpr (VEC == 4) {
    MX_NV(start_norm_backward, 1, 1) MX_NV(start_norm_backward, 2, 1) MX_NV(start_norm_backward, 4, 1)
    MX_NV(start_norm_backward, 3, 2) MX_NV(start_norm_backward, 4, 2) MX_NV(start_norm_backward, 3, 4)
    MX_NV(start_norm_backward, 4, 4) MX_NV(start_norm_backward, 3, 8) MX_NV(start_norm_backward, 4, 8)
    MX_NV(start_norm_backward, 6, 8)
  } else {
    MX_NV(start_norm_backward, 2, 1) MX_NV(start_norm_backward, 4, 1) MX_NV(start_norm_backward, 8, 1)
    MX_NV(start_norm_backward, 12, 1) MX_NV(start_norm_backward, 9, 2) MX_NV(start_norm_backward, 12, 2)
    MX_NV(start_norm_backward, 9, 4) MX_NV(start_norm_backward, 12, 4) MX_NV(start_norm_backward, 9, 8)
    MX_NV(start_norm_backward, 12, 8) MX_NV(start_norm_backward, 18, 8)
  }
  return 0;
}
#undef MX_NV

}  // namespace

size_t norm_backward_workspace(int64_t R, int64_t C) {
  return (size_t)norm_groups(R) * 2 * (size_t)C * sizeof(float);
}

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t st) {
  if (a.R == 0 || a.C == 0) return hipSuccess;
  const bool vec = norm_vec(a.C, a.bf16, {a.ldx, a.ldy}, {a.x, a.y, a.weight, a.bias});
  const int64_t held = a.bf16 ? (vec ? try_norm<true, 8>(a, st) : try_norm<true, 1>(a, st))
                           : (vec ? try_norm<false, 4>(a, st) : try_norm<false, 1>(a, st));
  if (!held) {
    if (a.bf16) hipLaunchKernelGGL((k_norm_any<true>), dim3(row_grid(a.R)), dim3(64 * LW), 0, st, a);
    else hipLaunchKernelGGL((k_norm_any<false>), dim3(row_grid(a.R)), dim3(64 * LW), 0, st, a);
  }
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(const NormBwdArgs& args, hipStream_t st) {
  NormBwdArgs a = args;
  if (a.C == 0) return hipSuccess;
  const bool sums = a.dweight || a.dbias;
  if (!sums) a.workspace = nullptr;
  int64_t G = 0;
  if (a.R > 0 && (sums || a.dx)) {
    const bool vec = norm_vec(a.C, a.bf16, {a.ldx, a.lddy, a.dx ? a.lddx : 0}, {a.x, a.dy, a.dx, a.weight});
    G = a.bf16 ? (vec ? try_norm_backward<true, 8>(a, st) : try_norm_backward<true, 1>(a, st))
               : (vec ? try_norm_backward<false, 4>(a, st) : try_norm_backward<false, 1>(a, st));
    if (G == 1) return hipGetLastError();             // (its one workgroup wrote them)
    if (G == 0) {
      // the weight's gradients first: dx may be written over dy or x
      if (sums) {
        G = norm_groups(a.R);
        const dim3 grid((unsigned)((a.C + 255) / 256), (unsigned)G);
        if (a.bf16) hipLaunchKernelGGL((k_norm_dw_any<true>), grid, dim3(256), 0, st, a, (int)G);
        else hipLaunchKernelGGL((k_norm_dw_any<false>), grid, dim3(256), 0, st, a, (int)G);
      }
      if (a.dx) {
        if (a.bf16) hipLaunchKernelGGL((k_norm_dx_any<true>), dim3(row_grid(a.R)), dim3(64 * LW), 0, st, a);
        else hipLaunchKernelGGL((k_norm_dx_any<false>), dim3(row_grid(a.R)), dim3(64 * LW), 0, st, a);
      }
    }
  }
  if (sums)
    hipLaunchKernelGGL(k_norm_dw_sum, dim3((unsigned)((a.C + 63) / 64), 2), dim3(1024), 0, st, a.workspace, (int)G,
                       a.C, a.dweight, a.dbias, (int)a.w_bf16);
  return hipGetLastError();
}

}  // namespace mx
