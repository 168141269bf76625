// The linear layer's backward pass on the MXFP8 / MXFP6 pipeline, FP6 A.
#include "linear_f8.h"

namespace mx {

hipError_t launch_linear_f8_backward_fp6(const LinearArgs& a, hipStream_t st) {
  return a.a_elem == 3 ? launch_f8_b<3, 5>(a, st) : launch_f8_b<4, 5>(a, st);
}

}  // namespace mx
