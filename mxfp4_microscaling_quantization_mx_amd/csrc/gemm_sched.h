// Tile schedules of the persistent 256x256 GEMM kernels (dense, and grouped by
// expert), shared by the plain products and the gated block.
// Include after gemm_tile256.h has defined namespace t256 (MX_T256_SWAP 0).
#pragma once

#include "mx_device.h"
#include "mx_launch.h"

namespace mx {
namespace {

// Persistent kernels: one workgroup per CU (G workgroups).  Workgroup b runs
// on XCD b % 8, so XCD x holds the step_x workgroups b = x, x+8, ...  The
// tiles, in the grouped order below, are cut into 8 contiguous ranges sized
// in proportion to step_x, one per XCD, and the XCD's workgroups take its
// range round-robin: the tiles one XCD works on at a time are consecutive,
// and each operand panel is fetched into one XCD's L2 rather than into all.
struct XcdShare {
  int first, n, step, k;                   // tiles first + k + j*step < first + n
  __device__ XcdShare(int b, int G, int T) {
    const int x = b % 8;
    step = G / 8 + (x < G % 8 ? 1 : 0);
    k = b / 8;
    // workgroups on the XCDs before x and up to x
    const int64_t w0 = (int64_t)x * (G / 8) + (x < G % 8 ? x : G % 8);
    const int64_t w1 = w0 + step;
    first = (int)(w0 * T / G);
    n = (int)(w1 * T / G) - first;
  }
  __device__ int count() const { return k < n ? (n - k + step - 1) / step : 0; }
  __device__ int tile(int j) const { return first + k + j * step; }
};

// Tile order (t256c::group_order): groups of GM M-tiles, each walked N-tile
// by N-tile (GM = 8 for the dense GEMM; 2 for the grouped one, whose row tiles
// belong to different experts' weights, measured ~3 % faster there).
using t256c::group_order;

constexpr int GW = t256::WAVES;

// BM: which rows of B a tile's LDS rows hold (t256c::B_*); a gated tile covers
// 128 hidden columns, and N counts those.
template <int BM>
constexpr int tile_cols() { return BM == t256c::B_ROWS ? t256::TN : t256::TN / 2; }

template <int BM = t256c::B_ROWS>
struct DenseSchedT {
  static constexpr bool UNITS = false;
  static constexpr int BMAP = BM;
  const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
  int M, N, tiles_m, tiles_n;
  XcdShare share;
  __device__ int count() const { return share.count(); }
  __device__ t256::TileInfo tile(int j) const {
    int tm, tn;
    group_order<8>(share.tile(j), tiles_m, tiles_n, tm, tn);
    t256::TileInfo ti;
    ti.a_codes = a_codes;
    ti.a_scales = a_scales;
    ti.b_codes = b_codes;
    ti.b_scales = b_scales;
    ti.m0 = tm * t256::TM;
    ti.n0 = tn * tile_cols<BM>();
    ti.M = M;
    ti.N = N;
    ti.c_row0 = ti.m0;
    return ti;
  }
};
using DenseSched = DenseSchedT<>;

// Grouped (MoE) GEMM.  A row tile ("slot") never straddles two experts: the
// slots of expert e are the ceil(rows_e / 256) tiles of its rows, numbered in
// expert order.  Each workgroup first builds, in LDS, the clamped row range of
// every expert and the exclusive prefix count of slots, from the device
// offsets (so the schedule needs no host synchronization); a tile's expert is
// then found by one wave-wide comparison against that prefix.
constexpr int GG_EMAX = 960;                // experts the LDS table holds (it fits beside the ring)

__device__ __forceinline__ int lds_i32(const int* p) {
  int v;
  const uint32_t a = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
  // an asm read that waits only for itself (not for loads in flight to LDS)
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(a) : "memory");
  return v;
}

// Per-launch parameters of the grouped GEMM, kept in LDS and read back per
// tile (holding them in scalar registers across the pipeline would spill).
struct alignas(16) GroupedParams {
  const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
  int64_t stride_codes, stride_scales;      // between experts of B
  int lda, ldsa, N, tiles_n, E, total_slots, pad0, pad1;
};
static_assert(sizeof(GroupedParams) == 80, "five 16-byte LDS reads");

// Read a wave-uniform GroupedParams from LDS with one wait.
__device__ __forceinline__ GroupedParams load_params(const GroupedParams* p) {
  typedef int v4i_ __attribute__((ext_vector_type(4)));
  v4i_ q[5];
  const uint32_t a = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
  asm volatile(
      "ds_read_b128 %0, %5\n\t"
      "ds_read_b128 %1, %5 offset:16\n\t"
      "ds_read_b128 %2, %5 offset:32\n\t"
      "ds_read_b128 %3, %5 offset:48\n\t"
      "ds_read_b128 %4, %5 offset:64\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(q[0]), "=&v"(q[1]), "=&v"(q[2]), "=&v"(q[3]), "=&v"(q[4])
      : "v"(a)
      : "memory");
  int w[20];
#pragma unroll
  for (int i = 0; i < 5; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) w[4 * i + k] = __builtin_amdgcn_readfirstlane(q[i][k]);
  return __builtin_bit_cast(GroupedParams, w);
}

// Two LDS words at per-lane addresses, one wait.
__device__ __forceinline__ void lds_i32x2(const int* p0, const int* p1, int& v0, int& v1) {
  const uint32_t a0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p0;
  const uint32_t a1 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p1;
  asm volatile("ds_read_b32 %0, %2\n\tds_read_b32 %1, %3\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(v0), "=&v"(v1)
               : "v"(a0), "v"(a1)
               : "memory");
}

template <int BM = t256c::B_ROWS>
struct GroupedSchedT {
  static constexpr bool UNITS = false;
  static constexpr int BMAP = BM;
  const GroupedParams* prm;                 // LDS
  const int* tab;                           // LDS: pre [E+1] exclusive prefix of slots, lo [E], hi [E]
  XcdShare share;
  __device__ int count() const { return share.count(); }
  __device__ t256::TileInfo tile(int j) const {
    const GroupedParams P = load_params(prm);
    int slot, tn;
    group_order<2>(share.tile(j), P.total_slots, P.tiles_n, slot, tn);
    const int* pre = tab;
    const int* lo = tab + GG_EMAX + 1;
    const int* hi = lo + GG_EMAX;
    const int lane = threadIdx.x & 63;
    int ex = P.E - 1;
    for (int base = 0; base < P.E; base += 64) {
      const int e = base + lane < P.E ? base + lane : P.E - 1;
      int p0, p1;
      lds_i32x2(pre + e, pre + e + 1, p0, p1);
      const unsigned long long m = __ballot(base + lane < P.E && slot >= p0 && slot < p1);
      if (m) {
        ex = base + __ffsll((long long)m) - 1;
        break;
      }
    }
    ex = __builtin_amdgcn_readfirstlane(ex);
    int l0, p0, h0;
    lds_i32x2(lo + ex, pre + ex, l0, p0);
    h0 = lds_i32(hi + ex);
    const int row0 = __builtin_amdgcn_readfirstlane(l0 + (slot - p0) * t256::TM);
    const int end = __builtin_amdgcn_readfirstlane(h0);
    const int rows = end - row0 < t256::TM ? end - row0 : t256::TM;
    t256::TileInfo ti;
    ti.a_codes = P.a_codes + (int64_t)row0 * P.lda;
    ti.a_scales = P.a_scales + (int64_t)row0 * P.ldsa;
    ti.b_codes = P.b_codes + (int64_t)ex * P.stride_codes;
    ti.b_scales = P.b_scales + (int64_t)ex * P.stride_scales;
    ti.m0 = 0;
    ti.n0 = tn * tile_cols<BM>();
    ti.M = rows;
    ti.N = P.N;
    ti.c_row0 = row0;
    return ti;
  }
};
using GroupedSched = GroupedSchedT<>;

// Fill the LDS expert table: pre [E+1] exclusive prefix of row tiles,
// lo [E] and hi [E] the clamped row range of each expert (wave 0 computes it;
// ends with a workgroup barrier).
__device__ __forceinline__ void build_expert_table(const int32_t* __restrict__ offsets, int E, int64_t M_cap,
                                                   int* tab) {
  int* pre = tab;
  int* lo = tab + GG_EMAX + 1;
  int* hi = lo + GG_EMAX;
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int base = 0; base < E; base += 64) {
      const int e = base + lane;
      int64_t l0 = 0, h0 = 0;
      if (e < E) {
        l0 = offsets[e];
        h0 = offsets[e + 1];
        l0 = l0 < 0 ? 0 : (l0 > M_cap ? M_cap : l0);
        h0 = h0 < l0 ? l0 : (h0 > M_cap ? M_cap : h0);
      }
      const int tiles = (int)((h0 - l0 + t256::TM - 1) / t256::TM);
      int incl = tiles;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(incl, d, 64);
        if (lane >= d) incl += v;
      }
      if (e < E) {
        pre[e] = carry + incl - tiles;
        lo[e] = (int)l0;
        hi[e] = (int)h0;
      }
      carry += __shfl(incl, 63, 64);
    }
    if (lane == 0) pre[E] = carry;
  }
  __syncthreads();
}

}  // namespace
}  // namespace mx
