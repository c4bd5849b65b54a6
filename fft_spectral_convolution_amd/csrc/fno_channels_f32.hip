// Channel products of float32 fields.
#include "fno_channels_kernel.hpp"

namespace fno {

hipError_t launch_product_f32(const ProductArgs& a, bool last, bool out_last, int out_type, hipStream_t s) {
    if (out_type == kTypeBf16) return launch_layouts<float, bf16>(a, last, out_last, s);
    if (out_type == kTypeF16) return launch_layouts<float, f16>(a, last, out_last, s);
    return launch_layouts<float, float>(a, last, out_last, s);
}

}  // namespace fno
