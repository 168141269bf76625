// The linear layer's backward pass on the MXFP8 / MXFP6 pipeline, FP8 A.
#include "linear_f8.h"

namespace mx {

hipError_t launch_linear_f8_backward(const LinearArgs& a, hipStream_t st) {
  switch (a.a_elem) {
    case 1: return launch_f8_b<1, 5>(a, st);
    case 2: return launch_f8_b<2, 5>(a, st);
    default: return launch_linear_f8_backward_fp6(a, st);
  }
}

}  // namespace mx
