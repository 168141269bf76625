// The linear layer with its epilogue on the MXFP8 / MXFP6 pipeline, forward (the
// backward kernels are in linear_f8_backward.hip, compiled beside it).
#include "linear_f8.h"

namespace mx {

// Scale rows are fetched a 32-bit word at a time; 256 rows of the operands and of
// the buffers are addressed with 32-bit offsets.
bool linear_f8_layout_ok(const GatedArgs& a) {
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

hipError_t launch_linear_f8(const GatedArgs& a, hipStream_t st) {
  return a.backward ? launch_linear_f8_backward(a, st) : launch_f8_a<false>(a, st);
}

}  // namespace mx
