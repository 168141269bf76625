// Dropout from Philox4x32-10 draws for gfx950: the mask is recomputed wherever
// it is needed and never stored.
//
// One Philox call gives eight 16-bit draws, so a lane takes the eight
// consecutive elements 8q .. 8q+7 of the row-major [R, C] order and makes the
// call of its q.  An element is dropped iff its draw is below T (a drop
// probability of exactly T / 65536) and kept values are multiplied by
// 65536 / (65536 - T), rounded to float32 once on the host.
#include "mx_device.h"
#include "mx_launch.h"

namespace mx {

namespace {

template <bool BF16>
__global__ __launch_bounds__(256) void k_dropout(DropoutArgs a, uint64_t ncalls, float scale) {
  const uint64_t n = (uint64_t)a.R * (uint64_t)a.C;
  for (uint64_t q = (uint64_t)blockIdx.x * 256 + threadIdx.x; q < ncalls; q += (uint64_t)gridDim.x * 256) {
    uint32_t w[4];
    sr_words(q, a.seed, a.offset, w);
    uint64_t e = 8 * q;
    int64_t r = (int64_t)(e / (uint64_t)a.C), c = (int64_t)(e - (uint64_t)r * (uint64_t)a.C);
    for (int i = 0; i < 8 && e < n; ++i, ++e) {
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
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t st) {
  if (a.R == 0 || a.C == 0) return hipSuccess;
  const uint64_t n = (uint64_t)a.R * (uint64_t)a.C, ncalls = (n + 7) / 8;
  const uint64_t want = (ncalls + 255) / 256;
  const unsigned grid = (unsigned)(want < (1u << 20) ? want : (1u << 20));
  // T = 65536 drops everything (no draw reaches it); the scale is then unused
  const float scale = a.threshold < 65536u ? (float)(65536.0 / (65536.0 - (double)a.threshold)) : 0.0f;
  if (a.bf16) hipLaunchKernelGGL((k_dropout<true>), dim3(grid), dim3(256), 0, st, a, ncalls, scale);
  else hipLaunchKernelGGL((k_dropout<false>), dim3(grid), dim3(256), 0, st, a, ncalls, scale);
  return hipGetLastError();
}

}  // namespace mx
