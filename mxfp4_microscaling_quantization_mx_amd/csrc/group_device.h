// Row tiles of rows grouped by expert, found from the device offsets.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

// Rows of expert e, clamped to [0, cap] and never negative in number.
__device__ __forceinline__ void expert_rows(const int32_t* __restrict__ off, int e, int64_t cap, int64_t& lo,
                                            int64_t& hi) {
  lo = off[e];
  hi = off[e + 1];
  lo = lo < 0 ? 0 : (lo > cap ? cap : lo);
  hi = hi < lo ? lo : (hi > cap ? cap : hi);
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
    if (e < E) {                      // (expert_rows, written out: called, it cost k_gated_tile 1 %)
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

// Row tiles of TM rows of the experts before e (every wave by itself).
template <int TM>
__device__ __forceinline__ int64_t slots_before(const int32_t* __restrict__ off, int e, int64_t cap) {
  const int lane = threadIdx.x & 63;
  int64_t n = 0;
  for (int i = lane; i < e; i += 64) {
    int64_t lo, hi;
    expert_rows(off, i, cap, lo, hi);
    n += (hi - lo + TM - 1) / TM;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d, 64);
  return n;
}

}  // namespace mx
