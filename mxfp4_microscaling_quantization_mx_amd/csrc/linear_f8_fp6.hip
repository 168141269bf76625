// The linear layer on the MXFP8 / MXFP6 pipeline, forward with FP6 A.
#include "linear_f8.h"

namespace mx {

hipError_t launch_linear_f8_fp6(const LinearArgs& a, hipStream_t st) {
  return a.a_elem == 3 ? launch_f8_b<3, 4>(a, st) : launch_f8_b<4, 4>(a, st);
}

}  // namespace mx
