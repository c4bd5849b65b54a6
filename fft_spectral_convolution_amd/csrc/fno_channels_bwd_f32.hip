// Backward pass of channel products of float32 fields with a float32 grad_out.
#include "fno_channels_bwd.hpp"

namespace fno {

hipError_t launch_backward_f32(const BackwardArgs& a, bool last, bool out_last, hipStream_t s) {
    return launch_backward<float, float>(a, last, out_last, s);
}

}  // namespace fno
