// The linear layer on the 256x256 MXFP4 pipeline: bias and residual (the kernels with an
// activation are in linear256_act.hip, compiled beside this file).
#include "linear256.h"

namespace mx {

// The pipeline fetches scale rows 16 bytes at a time and addresses an operand,
// and a tile's rows of the buffers, with 32-bit offsets.  The kernels with an activation
// take 1-D scales of A only: one more layout would double them for a case (2-D scales
// are for weights) that the 128-row tiles serve.
bool linear256_layout_ok(const LinearArgs& a) {
  const int64_t lim = 1ll << 31;
  const bool words = a.A.ld_scales % 16 == 0 && a.B.ld_scales % 16 == 0 && a.stride_scales % 16 == 0 &&
                     (uintptr_t)a.A.scales % 16 == 0 && (uintptr_t)a.B.scales % 16 == 0;
  const int64_t arows = a.offsets ? 256 : a.M;
  const bool small = arows * a.A.ld_codes < lim && a.N * a.B.ld_codes < lim && arows * a.A.ld_scales < lim &&
                     a.N * a.B.ld_scales < lim && 256 * a.ldo * 4 < lim && 256 * a.lddh * 4 < lim &&
                     a.K < (1ll << 30);
  const int64_t slots = a.offsets ? (a.M + 255) / 256 + a.E : (a.M + 255) / 256;
  return a.a_elem == 0 && a.b_elem == 0 && !(a.a_2d && a.act != 3) && words && small && (!a.offsets || a.E <= GG_EMAX) &&
         slots * ((a.N + 255) / 256) < lim;
}

hipError_t launch_linear256(const LinearArgs& a, hipStream_t st) {
  if (a.act != 3) return launch_linear256_act(a, st);
  constexpr int OUT = t256::OUT_LINEAR + 3;
  if (a.a_2d) return a.b_2d ? launch_out<true, true, OUT>(a, st) : launch_out<true, false, OUT>(a, st);
  return a.b_2d ? launch_out<false, true, OUT>(a, st) : launch_out<false, false, OUT>(a, st);
}

}  // namespace mx
