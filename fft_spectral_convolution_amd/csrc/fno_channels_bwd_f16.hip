// Backward pass of channel products of float16 fields with a float16 grad_out.
#include "fno_channels_bwd.hpp"

namespace fno {

hipError_t launch_backward_f16(const BackwardArgs& a, bool last, bool out_last, hipStream_t s) {
    return launch_backward<f16, f16>(a, last, out_last, s);
}

}  // namespace fno
