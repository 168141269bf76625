// The linear layer with its epilogue on the MXFP8 / MXFP6 pipeline, forward with FP8 A
// (FP6 A and the backward pass are in files of their own, compiled beside this one).
#include "linear_f8.h"

namespace mx {

// Scale rows are fetched a 32-bit word at a time; 256 rows of the operands and of
// the buffers are addressed with 32-bit offsets.
bool linear_f8_layout_ok(const LinearArgs& a) {
  const int64_t lim = 1ll << 31;
  const bool words = a.A.ld_scales % 4 == 0 && a.B.ld_scales % 4 == 0 && a.stride_scales % 4 == 0 &&
                     (uintptr_t)a.A.scales % 4 == 0 && (uintptr_t)a.B.scales % 4 == 0;
  const bool small = 256 * a.A.ld_codes < lim && 256 * a.B.ld_codes < lim && 256 * a.A.ld_scales < lim &&
                     256 * a.B.ld_scales < lim && 256 * a.ldo * 4 < lim && 256 * a.lddh * 4 < lim &&
                     a.K < (1ll << 30);
  const int64_t slots = a.offsets ? (a.M + 255) / 256 + a.E : (a.M + 255) / 256;
  return a.a_elem >= 1 && a.b_elem >= 1 && words && small && (!a.offsets || a.E <= GG_EMAX) &&
         slots * ((a.N + 255) / 256) < lim;
}

hipError_t launch_linear_f8(const LinearArgs& a, hipStream_t st) {
  if (a.backward) return launch_linear_f8_backward(a, st);
  switch (a.a_elem) {
    case 1: return launch_f8_b<1, 4>(a, st);
    case 2: return launch_f8_b<2, 4>(a, st);
    default: return launch_linear_f8_fp6(a, st);
  }
}

}  // namespace mx
