// Channel products of float16 fields.
#include "fno_channels_kernel.hpp"

namespace fno {

hipError_t launch_product_f16(const ProductArgs& a, bool last, bool out_last, int out_type, hipStream_t s) {
    if (out_type == kTypeF32) return launch_layouts<f16, float>(a, last, out_last, s);
    return launch_layouts<f16, f16>(a, last, out_last, s);
}

}  // namespace fno
