// Channel products of bfloat16 fields.
#include "fno_channels_kernel.hpp"

namespace fno {

hipError_t launch_product_bf16(const ProductArgs& a, bool last, bool out_last, int out_type, hipStream_t s) {
    if (out_type == kTypeF32) return launch_layouts<bf16, float>(a, last, out_last, s);
    return launch_layouts<bf16, bf16>(a, last, out_last, s);
}

}  // namespace fno
