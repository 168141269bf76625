// The linear layer's backward pass on the MXFP8 / MXFP6 pipeline.
#include "linear_f8.h"

namespace mx {

hipError_t launch_linear_f8_backward(const GatedArgs& a, hipStream_t st) { return launch_f8_a<true>(a, st); }

}  // namespace mx
