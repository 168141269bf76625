// The linear layer with an activation on the 256x256 MXFP4 pipeline, forward and backward.
#include "linear256.h"

namespace mx {
namespace {

template <int ACT>
hipError_t launch_act(const LinearArgs& a, hipStream_t st) {
  constexpr int F = t256::OUT_LINEAR + ACT, B = t256::OUT_LINEAR_BWD + ACT;
  if (a.backward) return a.b_2d ? launch_out<false, true, B>(a, st) : launch_out<false, false, B>(a, st);
  return a.b_2d ? launch_out<false, true, F>(a, st) : launch_out<false, false, F>(a, st);
}

}  // namespace

hipError_t launch_linear256_act(const LinearArgs& a, hipStream_t st) {
  switch (a.act) {
    case 0: return launch_act<0>(a, st);
    case 1: return launch_act<1>(a, st);
    default: return launch_act<2>(a, st);
  }
}

}  // namespace mx
