// Pieces of a row of bf16 or float32 elements, 16 bytes per lane.  A row may
// start at any element: gfx950 loads and stores 16 bytes at any element-aligned
// address, only slower where a piece crosses a cache line.
#pragma once

#include "mx_device.h"

namespace mx {

typedef uint32_t row_words __attribute__((ext_vector_type(4)));
// (the compiler may assume no more than a bf16 element's alignment)
typedef row_words loose_words __attribute__((aligned(2)));

template <bool BF16>
struct RowPiece {
  static constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES;
  typedef row_words words;

  float v[VEC];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 0.0f;
  }
  __device__ __forceinline__ void unpack(const words w) {
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[2 * i] = bf16lo(w[i]), v[2 * i + 1] = bf16hi(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ words pack() const {
    words w;
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i]) |
               ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i + 1]) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
    }
    return w;
  }

  // n elements at p (n < VEC: the row's last ones, one at a time, the rest 0).
  static __device__ __forceinline__ words load(const void* p, int n) {
    if (n >= VEC) return *static_cast<const loose_words*>(p);
    words w = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < VEC - 1; ++i)
      if (i < n) {
        if constexpr (BF16) w[i / 2] |= (uint32_t) static_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
        else w[i] = static_cast<const uint32_t*>(p)[i];
      }
    return w;
  }
  static __device__ __forceinline__ void store(void* p, const words w, int n) {
    if (n >= VEC) {
      *static_cast<loose_words*>(p) = w;
      return;
    }
#pragma unroll
    for (int i = 0; i < VEC - 1; ++i)
      if (i < n) {
        if constexpr (BF16) static_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        else static_cast<uint32_t*>(p)[i] = w[i];
      }
  }
};

}  // namespace mx
