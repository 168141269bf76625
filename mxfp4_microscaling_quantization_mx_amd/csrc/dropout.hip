// Dropout from Philox4x32-10 draws for gfx950: the mask is recomputed wherever
// it is needed and never stored.
//
// One Philox call gives eight 16-bit draws, so a lane takes the eight
// consecutive elements 8q .. 8q+7 of the row-major [R, C] order and makes the
// call of its q.  An element is dropped iff its draw is below T (a drop
// probability of exactly T / 65536) and kept values are multiplied by
// 65536 / (65536 - T), rounded to float32 once on the host.
//
// Bound by HBM bandwidth: 16384 x 2880 bf16 with a residual 49 us, 5.8 TB/s (a
// device copy 5.1); one element at a time 162.  A call's ten rounds are 20
// 64-bit multiplies per eight elements, hidden behind the loads.  1023 x 1111
// float32 6.0-6.5 us, the cost of a launch.  Rows that no 16-byte piece fits go
// element by element: 4099 x 1111 bf16 with a residual 8.6 us contiguous (one long
// row), 23 with a padded row stride.
#include "mx_device.h"
#include "mx_launch.h"

namespace mx {

namespace {

// The elements of call q one at a time, at any strides and alignments.
template <bool BF16>
__device__ __forceinline__ void dropout_elements(const DropoutArgs& a, uint64_t q, uint64_t n, float scale) {
  uint32_t w[4];
  sr_words(q, a.seed, a.offset, w);
  uint64_t e = 8 * q;
  int64_t r = (int64_t)(e / (uint64_t)a.C), c = (int64_t)(e - (uint64_t)r * (uint64_t)a.C);
#pragma unroll
  for (int i = 0; i < 8; ++i, ++e) {
    if (e >= n) break;
    const uint32_t draw = (w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
    const int64_t ix = r * a.ldx + c, ir = r * a.ldr + c, iy = r * a.ldy + c;
    float v = 0.0f;
    if (draw >= a.threshold)
      v = scale * (BF16 ? bf16lo(static_cast<const uint16_t*>(a.x)[ix]) : static_cast<const float*>(a.x)[ix]);
    if (a.residual)
      v = v + (BF16 ? bf16lo(static_cast<const uint16_t*>(a.residual)[ir]) : static_cast<const float*>(a.residual)[ir]);
    if (BF16) static_cast<uint16_t*>(a.y)[iy] = (uint16_t)f32_to_bf16_rne(v);
    else static_cast<float*>(a.y)[iy] = v;
    if (++c == a.C) {
      c = 0;
      ++r;
    }
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_dropout(DropoutArgs a, uint64_t n, float scale) {
  const uint64_t ncalls = (n + 7) / 8;
  for (uint64_t q = (uint64_t)blockIdx.x * 256 + threadIdx.x; q < ncalls; q += (uint64_t)gridDim.x * 256)
    dropout_elements<BF16>(a, q, n, scale);
}

// Eight elements at index i of a buffer, 16 bytes at a time.
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, uint64_t i, float x[8]) {
  if (BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = (k & 1) ? bf16hi(v[k >> 1]) : bf16lo(v[k >> 1]);
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void* p, uint64_t i, const float x[8]) {
  if (BF16) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = (uint32_t)__builtin_bit_cast(unsigned short, (__bf16)x[2 * k]) |
             ((uint32_t)__builtin_bit_cast(unsigned short, (__bf16)x[2 * k + 1]) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(x[0], x[1], x[2], x[3]);
    q[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// The same where the eight elements of a call are consecutive and 16-byte
// aligned in every buffer: rows of whole calls (ROWS, cpr = C / 8 per row), or
// buffers without gaps between rows, taken as one row of n elements whose
// last call may be short.
template <bool BF16, bool RES, bool ROWS>
__global__ __launch_bounds__(256) void k_dropout8(DropoutArgs a, uint64_t n, uint32_t cpr, float scale) {
  const uint64_t ncalls = (n + 7) / 8;
  for (uint64_t q = (uint64_t)blockIdx.x * 256 + threadIdx.x; q < ncalls; q += (uint64_t)gridDim.x * 256) {
    uint64_t ix = 8 * q, ir = ix, iy = ix;
    if (!ROWS && ix + 8 > n) {
      dropout_elements<BF16>(a, q, n, scale);
      return;
    }
    if (ROWS) {
      const uint64_t r = q >> 32 ? q / cpr : (uint32_t)q / cpr, c = 8 * (q - r * cpr);
      ix = r * (uint64_t)a.ldx + c;
      ir = r * (uint64_t)a.ldr + c;
      iy = r * (uint64_t)a.ldy + c;
    }
    float x[8], y[8];
    load8<BF16>(a.x, ix, x);
    if (RES) load8<BF16>(a.residual, ir, y);
    uint32_t w[4];
    sr_words(q, a.seed, a.offset, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t draw = (k & 1) ? w[k >> 1] >> 16 : w[k >> 1] & 0xFFFFu;
      const float v = draw >= a.threshold ? scale * x[k] : 0.0f;
      y[k] = RES ? v + y[k] : v;
    }
    store8<BF16>(a.y, iy, y);
  }
}

}  // namespace

// Workgroups of 256 calls.
static unsigned call_grid(uint64_t calls) {
  const uint64_t want = (calls + 255) / 256;
  return (unsigned)(want < (1u << 20) ? want : (1u << 20));
}

template <bool BF16>
static hipError_t launch_dropout_type(const DropoutArgs& a, hipStream_t st) {
  const uint64_t n = (uint64_t)a.R * (uint64_t)a.C, ncalls = (n + 7) / 8;
  // T = 65536 drops everything (no draw reaches it); the scale is then unused
  const float scale = a.threshold < 65536u ? (float)(65536.0 / (65536.0 - (double)a.threshold)) : 0.0f;
  const bool res = a.residual != nullptr;
  const bool aligned = ((uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)a.residual) % 16 == 0;
  const bool flat = a.R == 1 || (a.ldx == a.C && a.ldy == a.C && (!res || a.ldr == a.C));
  const int64_t v = BF16 ? 8 : 4;
  const bool rows = a.C % 8 == 0 && a.C / 8 <= 0xFFFFFFFFll && a.ldx % v == 0 && a.ldy % v == 0 &&
                    (!res || a.ldr % v == 0);
  const dim3 grid = dim3(call_grid(ncalls));
  if (aligned && (flat || rows)) {
    const uint32_t cpr = flat ? 1u : (uint32_t)(a.C / 8);
#define MX_D8(RES_, ROWS_) \
  hipLaunchKernelGGL((k_dropout8<BF16, RES_, ROWS_>), grid, dim3(256), 0, st, a, n, cpr, scale)
    if (flat) { if (res) MX_D8(true, false); else MX_D8(false, false); }
    else { if (res) MX_D8(true, true); else MX_D8(false, true); }
#undef MX_D8
  } else {
    hipLaunchKernelGGL((k_dropout<BF16>), grid, dim3(256), 0, st, a, n, scale);
  }
  return hipGetLastError();
}

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t st) {
  if (a.R == 0 || a.C == 0) return hipSuccess;
  return a.bf16 ? launch_dropout_type<true>(a, st) : launch_dropout_type<false>(a, st);
}

}  // namespace mx
