// Channel products: which kernels a call runs, and the gradient of the weight.
#include <algorithm>
#include <string_view>

#include "fno_channels.hpp"

namespace fno {
namespace {

// grad_w and, behind it, grad_b: sums over the splits, 64 values a workgroup at a time, each
// wave a quarter of the splits.
__global__ __launch_bounds__(256) void k_weight_sum(const float* __restrict__ part, float* __restrict__ grad_w,
                                                    float* __restrict__ grad_b, int64_t weights, int couts,
                                                    int splits) {
    __shared__ double join[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t all = weights + couts;
    for (int64_t first = (int64_t)blockIdx.x * 64; first < all; first += (int64_t)gridDim.x * 64) {
        const int64_t k = first + lane;
        double s = 0.0;
        if (k < all) {
            int i = wave;
            for (; i + 28 < splits; i += 32) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = part[(i + 4 * u) * all + k];
#pragma unroll
                for (int u = 0; u < 8; ++u) s += (double)v[u];
            }
            for (; i < splits; i += 4) s += (double)part[i * all + k];
        }
        join[wave][lane] = s;
        __syncthreads();
        if (wave == 0 && k < all) {
            const float v = (float)((join[0][lane] + join[1][lane]) + (join[2][lane] + join[3][lane]));
            if (k < weights) {
                if (grad_w) grad_w[k] = v;
            } else if (grad_b) {
                grad_b[k - weights] = v;
            }
        }
        __syncthreads();
    }
}

// Workgroups of it: a grid's threads are counted in 32 bits, the weights are up to 2^32.
unsigned sum_groups(const ChannelProduct& c) {
    return (unsigned)std::min<int64_t>(((int64_t)c.Cin * c.Cout + c.Cout + 63) / 64, 1 << 20);
}

// Shares of the positions: up to two workgroups a CU, each of a tile of 32 a wave or more.
int weight_splits(const ChannelProduct& c) {
    const int64_t tiles = c.B * ((c.P + 31) / 32);
    const int64_t parts = (int64_t)((c.Cin + 63) / 64) * ((c.Cout + 63) / 64);
    return (int)std::max<int64_t>(1, std::min<int64_t>(tiles / 4, 512 / parts));
}

hipError_t launch_product(const ProductArgs& a, int x_type, bool last, bool out_last, int out_type, hipStream_t s) {
    if (x_type == kTypeBf16) return launch_product_bf16(a, last, out_last, out_type, s);
    if (x_type == kTypeF16) return launch_product_f16(a, last, out_last, out_type, s);
    return launch_product_f32(a, last, out_last, out_type, s);
}

size_t round_up(size_t v) { return (v + 255) / 256 * 256; }

// Whether g = grad_out act'(z) is a field of its own.
bool keeps_g(const ChannelProduct& c) { return c.act != kActNone; }

bool fits(const ChannelProduct& c) { return backward_fits(c.Cin, c.Cout, c.x_type); }

// Workgroups of the one-kernel backward pass: one a CU, two where the registers that 32 channels take leave room.
int backward_groups(const ChannelProduct& c) {
    const int64_t tiles = c.x_last && c.out_last ? (c.B * c.P + 31) / 32 : c.B * ((c.P + 31) / 32);
    return (int)std::min<int64_t>((tiles + 3) / 4, std::max(c.Cin, c.Cout) <= 32 ? 512 : 256);
}

hipError_t launch_backward(const BackwardArgs& a, const ChannelProduct& c, hipStream_t s) {
    if (c.x_type == kTypeF32) return launch_backward_f32(a, c.x_last, c.out_last, s);
    if (c.x_type == kTypeBf16)
        return c.out_type == kTypeF32 ? launch_backward_bf16_f32(a, c.x_last, c.out_last, s)
                                      : launch_backward_bf16(a, c.x_last, c.out_last, s);
    return c.out_type == kTypeF32 ? launch_backward_f16_f32(a, c.x_last, c.out_last, s)
                                  : launch_backward_f16(a, c.x_last, c.out_last, s);
}

}  // namespace

size_t channel_workspace(const ChannelProduct& c, bool backward) {
    if (!backward) return 0;
    const size_t g = keeps_g(c) && !fits(c) ? round_up((size_t)(c.B * c.P * c.Cout) * sizeof(float)) : 0;
    const int splits = fits(c) ? backward_groups(c) : weight_splits(c);
    return g + round_up((size_t)splits * ((size_t)c.Cin + 1) * c.Cout * sizeof(float));
}

int channel_kernels(const ChannelProduct& c, const ChannelArgs& a, bool backward, const char** names) {
    if (!backward) {
        names[0] = "channels";
        return 1;
    }
    int n = 0;
    const bool sums = a.grad_w || a.grad_b;
    if (fits(c)) {
        names[n++] = "channels_bwd";
    } else {
        if (keeps_g(c)) names[n++] = "channels_slope";
        if (a.grad_x) names[n++] = "channels_grad_x";
        if (sums) names[n++] = "channels_grad_w";
    }
    if (sums) names[n++] = "channels_grad_sum";
    return n;
}

hipError_t launch_channels(const ChannelProduct& c, const ChannelArgs& a, bool backward, int kernel, hipStream_t s) {
    const char* names[4] = {};
    channel_kernels(c, a, backward, names);
    const bool slope = names[kernel] == std::string_view("channels_slope");
    ProductArgs q{};
    q.B = c.B;
    q.P = c.P;
    q.Cin = c.Cin;
    q.Cout = c.Cout;
    q.x = a.x;
    q.w = a.w;
    q.w_type = c.x_type;
    q.bias = a.bias;
    q.branch = a.branch;
    q.branch_after = c.branch_after;
    q.act = c.act;
    if (!backward) {
        q.out = a.out;
        return launch_product(q, c.x_type, c.x_last, c.out_last, c.out_type, s);
    }
    float* g = static_cast<float*>(a.ws);
    const bool own_g = keeps_g(c) && !fits(c);
    float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) +
                                           (own_g ? round_up((size_t)(c.B * c.P * c.Cout) * sizeof(float)) : 0));
    const int splits = fits(c) ? backward_groups(c) : weight_splits(c);
    if (names[kernel] == std::string_view("channels_bwd")) {
        BackwardArgs b{};
        b.x = a.x;
        b.w = a.w;
        b.bias = a.bias;
        b.branch = c.branch_after || c.act == kActNone ? nullptr : a.branch;
        b.grad = a.out;
        b.grad_x = a.grad_x;
        b.grad_branch = a.grad_branch;
        b.part = a.grad_w || a.grad_b ? part : nullptr;
        b.B = c.B;
        b.P = c.P;
        b.Cin = c.Cin;
        b.Cout = c.Cout;
        b.act = c.act;
        b.groups = splits;
        return launch_backward(b, c, s);
    }
    if (slope) {
        if (c.branch_after) q.branch = nullptr;
        q.slope = true;
        q.grad = a.out;
        q.g = g;
        q.out = a.grad_branch;
        return launch_product(q, c.x_type, c.x_last, c.out_last, c.out_type, s);
    }
    const void* gp = own_g ? static_cast<const void*>(g) : a.out;
    const int g_type = own_g ? kTypeF32 : c.out_type;
    if (names[kernel] == std::string_view("channels_grad_x")) {
        q.x = gp;
        q.bias = nullptr;
        q.branch = nullptr;
        q.act = kActNone;
        q.transposed = true;
        q.Cin = c.Cout;
        q.Cout = c.Cin;
        q.out = a.grad_x;
        return launch_product(q, g_type, c.out_last, c.x_last, c.x_type, s);
    }
    if (names[kernel] == std::string_view("channels_grad_w")) {
        WeightGradArgs w{};
        w.x = a.x;
        w.g = gp;
        w.part = part;
        w.B = c.B;
        w.P = c.P;
        w.Cin = c.Cin;
        w.Cout = c.Cout;
        w.splits = splits;
        return launch_channel_weight_grad(w, c.x_type, g_type, c.x_last, c.out_last, s);
    }
    const int64_t weights = (int64_t)c.Cin * c.Cout;
    return launch_kernel(k_weight_sum, dim3(sum_groups(c)), dim3(256), 0, s,
                         static_cast<const float*>(part), a.grad_w, a.grad_b, weights, c.Cout, splits);
}

}  // namespace fno
