// Channel products: which kernels a call runs, and the joining of the sums of the parameters' gradients.
#include <algorithm>

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

// Tiles of 32 positions that a backward pass takes: where both sides are channels last, all positions are one run.
int64_t tiles_of(const ChannelProduct& c) {
    return c.x_last && c.out_last ? (c.B * c.P + 31) / 32 : c.B * ((c.P + 31) / 32);
}

// Shares of the positions: up to two workgroups a CU, each of a tile a wave or more.
int weight_splits(const ChannelProduct& c) {
    const int64_t tiles = tiles_of(c);
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
    return (int)std::min<int64_t>((tiles_of(c) + 3) / 4, std::max(c.Cin, c.Cout) <= 32 ? 512 : 256);
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

namespace {

// The kernels of a call.
enum Step { kForward, kSlope, kGradX, kGradW, kOnePass, kSum };

int steps_of(const ChannelProduct& c, const ChannelArgs& a, bool backward, Step* steps) {
    if (!backward) {
        steps[0] = kForward;
        return 1;
    }
    int n = 0;
    const bool sums = a.grad_w || a.grad_b;
    if (fits(c)) {
        steps[n++] = kOnePass;
    } else {
        if (keeps_g(c)) steps[n++] = kSlope;
        if (a.grad_x) steps[n++] = kGradX;
        if (sums) steps[n++] = kGradW;
    }
    if (sums) steps[n++] = kSum;
    return n;
}

// Types of what a product reads and writes, and its channels: of the step kForward, kSlope or kGradX.
struct Sides {
    int x_type, out_type;
    bool last, out_last;
};
Sides sides_of(const ChannelProduct& c, Step step) {
    if (step == kGradX) return {keeps_g(c) ? kTypeF32 : c.out_type, c.x_type, c.out_last, c.x_last};
    return {c.x_type, c.out_type, c.x_last, c.out_last};
}
ProductArgs product_of(const ChannelProduct& c, Step step) {
    ProductArgs q{};
    q.B = c.B;
    q.P = c.P;
    q.Cin = step == kGradX ? c.Cout : c.Cin;
    q.Cout = step == kGradX ? c.Cin : c.Cout;
    q.w_type = c.x_type;
    return q;
}

// A kernel's name, with the form it takes: output channels a wave, and whether the weight
// takes a workgroup of eight waves (wide) or does not fit LDS at all (staged).
#define FNO_FORMS(name) \
    {name "_32", name "_32_wide", name "_32_staged", name "_64", name "_64_wide", name "_64_staged", \
     name "_128", name "_128_wide", name "_128_staged"}
const char* name_of(const ChannelProduct& c, Step step) {
    static const char* const forms[3][9] = {FNO_FORMS("channels"), FNO_FORMS("channels_slope"),
                                            FNO_FORMS("channels_grad_x")};
    switch (step) {
        case kGradW: return "channels_grad_w";
        case kOnePass: return "channels_bwd";
        case kSum: return "channels_grad_sum";
        default: break;
    }
    const Sides t = sides_of(c, step);
    const ProductPlan p = plan_product(product_of(c, step), t.x_type, t.out_type, t.last && t.out_last);
    return forms[step][(p.mt == 4 ? 6 : p.mt == 2 ? 3 : 0) + (p.chunk < p.nks ? 2 : p.waves == 8 ? 1 : 0)];
}
#undef FNO_FORMS

}  // namespace

int channel_kernels(const ChannelProduct& c, const ChannelArgs& a, bool backward, const char** names) {
    Step steps[4];
    const int n = steps_of(c, a, backward, steps);
    for (int k = 0; k < n; ++k) names[k] = name_of(c, steps[k]);
    return n;
}

hipError_t launch_channels(const ChannelProduct& c, const ChannelArgs& a, bool backward, int kernel, hipStream_t s) {
    Step steps[4];
    steps_of(c, a, backward, steps);
    const Step step = steps[kernel];
    const Sides t = sides_of(c, step);
    ProductArgs q = product_of(c, step);
    q.x = a.x;
    q.w = a.w;
    q.bias = a.bias;
    q.branch = a.branch;
    q.branch_after = c.branch_after;
    q.act = c.act;
    if (step == kForward) {
        q.out = a.out;
        return launch_product(q, t.x_type, t.last, t.out_last, t.out_type, s);
    }
    float* g = static_cast<float*>(a.ws);
    const bool own_g = keeps_g(c) && !fits(c);
    float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) +
                                           (own_g ? round_up((size_t)(c.B * c.P * c.Cout) * sizeof(float)) : 0));
    const int splits = fits(c) ? backward_groups(c) : weight_splits(c);
    if (step == kOnePass) {
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
    if (step == kSlope) {
        if (c.branch_after) q.branch = nullptr;
        q.slope = true;
        q.grad = a.out;
        q.g = g;
        q.out = a.grad_branch;
        return launch_product(q, t.x_type, t.last, t.out_last, t.out_type, s);
    }
    const void* gp = own_g ? static_cast<const void*>(g) : a.out;
    const int g_type = own_g ? kTypeF32 : c.out_type;
    if (step == kGradX) {
        q.x = gp;
        q.bias = nullptr;
        q.branch = nullptr;
        q.act = kActNone;
        q.transposed = true;
        q.out = a.grad_x;
        return launch_product(q, t.x_type, t.last, t.out_last, t.out_type, s);
    }
    if (step == kGradW) {
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
