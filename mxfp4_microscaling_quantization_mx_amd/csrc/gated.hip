// The gated feed-forward block on MX operands for gfx950: both projections,
// the activation and the product in one kernel, and the backward pass that
// recomputes the projections (formulas in gate_device.h).
//
// k_gated_direct takes any shape, element types, scale layout and alignment.
// A workgroup of 8 waves computes 32 rows by 16 hidden columns: its B tile is
// the 32 weight rows of those columns' gates (first 16) and ups (last 16), so
// one V_MFMA_SCALE_F32_32X32X64_F8F6F4 per 64-deep step gives both
// projections.  The waves take consecutive parts of the K range, each lane
// loading its operand block straight from global memory, and add their
// partial tiles through LDS in wave order; then one thread per output applies
// the formula.
#include "gate_device.h"
#include "mx_device.h"
#include "mx_launch.h"

namespace mx {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// MFMA operand-format field of mx_elem F.
template <int F>
constexpr int mfma_fmt() {
  if constexpr (F == 0) return 4;
  else return ElemT<F>::MFMA;
}

// The expert and rows of row tile `slot` (TM rows each, numbered in expert
// order) from the device offsets, clamped to [0, cap]; every wave works it out
// by itself.  False past the last tile.
template <int TM>
__device__ __forceinline__ bool find_slot(const int32_t* __restrict__ off, int E, int64_t cap, int64_t slot, int& ex,
                                          int64_t& row0, int& rows) {
  const int lane = threadIdx.x & 63;
  int64_t carry = 0;
  for (int base = 0; base < E; base += 64) {
    const int e = base + lane;
    int64_t l0 = 0, h0 = 0;
    if (e < E) {
      l0 = off[e];
      h0 = off[e + 1];
      l0 = l0 < 0 ? 0 : (l0 > cap ? cap : l0);
      h0 = h0 < l0 ? l0 : (h0 > cap ? cap : h0);
    }
    const int tiles = (int)((h0 - l0 + TM - 1) / TM);
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl += v;
    }
    const int64_t s = slot - carry;
    const unsigned long long m = __ballot(s >= incl - tiles && s < incl);
    if (m) {
      const int src = __ffsll((long long)m) - 1;
      const int pre = __shfl(incl - tiles, src, 64);
      const int lo = __shfl((int)l0, src, 64), hi = __shfl((int)h0, src, 64);
      ex = __builtin_amdgcn_readfirstlane(base + src);
      const int r = __builtin_amdgcn_readfirstlane(lo + (int)(s - pre) * TM);
      const int n = __builtin_amdgcn_readfirstlane(hi) - r;
      row0 = r;
      rows = n < TM ? n : TM;
      return true;
    }
    carry += __shfl(incl, 63, 64);
  }
  return false;
}

// This lane's operand registers and scale byte of 64-deep step ks (K-blocks
// 2 ks and 2 ks + 1, the second of which may lie past K: zero codes at scale
// 1).  FP4 and FP6 lanes take K-block 2 ks + hi whole, FP8 lanes the 16-byte
// halves [16 hi, +16) of both blocks.
template <int F>
__device__ __forceinline__ v8i load_step(const uint8_t* __restrict__ row, const uint8_t* __restrict__ srow, int ks,
                                         int nkb, int hi, int& sc) {
  const int kb = 2 * ks + hi;
  const bool whole = 2 * ks + 1 < nkb;
  const bool live = kb < nkb;
  sc = live ? (int)srow[live ? kb : 0] : 127;
  v8i v;
  if constexpr (elem_bits<F>() == 8) {
    const uint4 x = *reinterpret_cast<const uint4*>(row + 64 * (int64_t)ks + 16 * hi);
    uint4 y = make_uint4(0, 0, 0, 0);
    if (whole) y = *reinterpret_cast<const uint4*>(row + 64 * (int64_t)ks + 32 + 16 * hi);
    v = v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
  } else if constexpr (elem_bits<F>() == 6) {
    uint2 x = make_uint2(0, 0), y = x, z = x;
    if (live) {
      const uint2* p = reinterpret_cast<const uint2*>(row + 24 * (int64_t)kb);
      x = p[0];
      y = p[1];
      z = p[2];
    }
    v = v8i{(int)x.x, (int)x.y, (int)y.x, (int)y.y, (int)z.x, (int)z.y, 0, 0};
  } else {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (live) x = *reinterpret_cast<const uint4*>(row + 16 * (int64_t)kb);
    v = v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
  }
  return v;
}

__device__ __forceinline__ float load_out(const void* p, bool bf16, int64_t i) {
  return bf16 ? bf16lo(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_out(void* p, bool bf16, int64_t i, float v) {
  if (bf16) static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16_rne(v);
  else static_cast<float*>(p)[i] = v;
}

constexpr int DW = 8;               // waves of k_gated_direct, splitting K

template <int FA, int FB>
__global__ __launch_bounds__(64 * DW) void k_gated_direct(GatedArgs a, int64_t tiles, int64_t tiles_n) {
  __shared__ float red[DW][32][33];
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t slot = t / tiles_n;
    int ex = 0, rows;
    int64_t row0;
    if (a.offsets) {
      if (!find_slot<32>(a.offsets, a.E, a.M, slot, ex, row0, rows)) return;   // past the last tile
    } else {
      row0 = slot * 32;
      rows = (int)(a.M - row0 < 32 ? a.M - row0 : 32);
    }
    const int64_t n0 = (t - slot * tiles_n) * 16;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int l32 = lane & 31, hi = lane >> 5;
    // rows and columns past the end read the last one; their results are dropped
    const int64_t ra = row0 + (l32 < rows ? l32 : rows - 1);
    const int64_t n = n0 + (l32 & 15) < a.N ? n0 + (l32 & 15) : a.N - 1;
    const int64_t rb = a.halves ? (int64_t)(l32 >> 4) * a.N + n : 2 * n + (l32 >> 4);
    const uint8_t* pa = a.A.codes + ra * a.A.ld_codes;
    const uint8_t* sa = a.A.scales + (a.a_2d ? ra >> 5 : ra) * a.A.ld_scales;
    const uint8_t* pb = a.B.codes + ex * a.stride_codes + rb * a.B.ld_codes;
    const uint8_t* sb = a.B.scales + ex * a.stride_scales + (a.b_2d ? rb >> 5 : rb) * a.B.ld_scales;
    const int nkb = (int)(a.K / 32), steps = (nkb + 1) / 2, per = (steps + DW - 1) / DW;
    const int k0 = w * per, k1 = k0 + per < steps ? k0 + per : steps;
    v16f acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
    for (int ks = k0; ks < k1; ++ks) {
      int xa, xb;
      const v8i va = load_step<FA>(pa, sa, ks, nkb, hi, xa);
      const v8i vb = load_step<FB>(pb, sb, ks, nkb, hi, xb);
      acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va, vb, acc, mfma_fmt<FA>(), mfma_fmt<FB>(), 0, xa, 0, xb);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) red[w][8 * (r >> 2) + 4 * hi + (r & 3)][l32] = acc[r];
    __syncthreads();
    const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
    if (row < rows && n0 + col < a.N) {
    float g = red[0][row][col], u = red[0][row][col + 16];
#pragma unroll
    for (int i = 1; i < DW; ++i) {
      g = g + red[i][row][col];
      u = u + red[i][row][col + 16];
    }
    const GateP p{a.act, a.alpha, a.limit, a.up_shift};
    const int64_t orow = row0 + row, c = n0 + col;
    if (!a.dH) {
      store_out(a.out, a.out_bf16, orow * a.ldo + c, gate_forward_any(p, g, u));
    } else {
      float dg, du;
      gate_backward_any(p, g, u, load_out(a.dH, a.dh_bf16, orow * a.lddh + c), dg, du);
      store_out(a.out, a.out_bf16, orow * a.ldo + (a.halves ? c : 2 * c), dg);
      store_out(a.out, a.out_bf16, orow * a.ldo + (a.halves ? a.N + c : 2 * c + 1), du);
    }
    }
    __syncthreads();                  // red is free again
  }
}

// Row tiles of TM rows a grouped launch must offer: every expert with rows
// adds at most one partial tile.
int64_t slot_bound(const GatedArgs& a, int TM) {
  if (!a.offsets) return (a.M + TM - 1) / TM;
  return a.M / TM + (a.E < a.M ? a.E : a.M);
}

template <int FA, int FB>
hipError_t launch_direct(const GatedArgs& a, hipStream_t st) {
  const int64_t tiles_n = (a.N + 15) / 16, tiles = tiles_n * slot_bound(a, 32);
  const unsigned grid = (unsigned)(tiles < (1 << 20) ? tiles : (1 << 20));
  hipLaunchKernelGGL((k_gated_direct<FA, FB>), dim3(grid), dim3(64 * DW), 0, st, a, tiles, tiles_n);
  return hipGetLastError();
}

template <int FA>
hipError_t launch_direct_b(const GatedArgs& a, hipStream_t st) {
  switch (a.b_elem) {
    case 1: return launch_direct<FA, 1>(a, st);
    case 2: return launch_direct<FA, 2>(a, st);
    case 3: return launch_direct<FA, 3>(a, st);
    case 4: return launch_direct<FA, 4>(a, st);
    default: return launch_direct<FA, 0>(a, st);
  }
}

}  // namespace

hipError_t launch_gated(const GatedArgs& a, hipStream_t st) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  if (a.M >= 256 && a.N >= 128 && gated256_layout_ok(a)) return launch_gated256(a, st);
  if (a.M >= 256 && a.N >= 128 && gated_f8_layout_ok(a)) return launch_gated_f8(a, st);
  switch (a.a_elem) {
    case 1: return launch_direct_b<1>(a, st);
    case 2: return launch_direct_b<2>(a, st);
    case 3: return launch_direct_b<3>(a, st);
    case 4: return launch_direct_b<4>(a, st);
    default: return launch_direct_b<0>(a, st);
  }
}

}  // namespace mx
