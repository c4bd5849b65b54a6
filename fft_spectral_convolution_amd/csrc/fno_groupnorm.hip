// Group norm with an activation, and its backward pass.
//
// With n = P D values in a group (D = C / groups channels of all P positions):
//   mean = sum x / n,  var = sum (x - mean)^2 / n,  rstd = (var + eps)^-1/2
//   xh = (x - mean) rstd,  z = xh w_c + b_c,  out = act(z)
// and, for grad_out = dL/dout, g = grad_out act'(z):
//   grad_b_c = sum_{b,p} g,  grad_w_c = sum_{b,p} g xh
//   s1 = sum_group g w_c / n,  s2 = sum_group g w_c xh / n
//   grad_x = rstd (g w_c - s1 - xh s2)
// (the last from differentiating mean and rstd, which both depend on x).
#include "fno_fields.hpp"

namespace fno {
namespace {

constexpr int kThreads = 256;

struct View {
    int64_t B, C, P, G;
    bool last;
    __device__ __forceinline__ int64_t at(int64_t b, int64_t c, int64_t p) const {
        return last ? (b * P + p) * C + c : (b * C + c) * P + p;
    }
};

// One workgroup per (item, group): mean first, then the squares about it.
template <typename TX>
__global__ __launch_bounds__(kThreads) void k_gn_stats(const TX* __restrict__ x, float* __restrict__ stats, View v,
                                                       float eps) {
    __shared__ float red[16];
    const int64_t b = blockIdx.x / v.G, g = blockIdx.x % v.G, D = v.C / v.G, n = D * v.P;
    float sum = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const int64_t d = v.last ? i % D : i / v.P, p = v.last ? i / D : i % v.P;
        sum += (float)x[v.at(b, g * D + d, p)];
    }
    const float mean = block_sum(sum, red) / (float)n;
    float sq = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const int64_t d = v.last ? i % D : i / v.P, p = v.last ? i / D : i % v.P;
        const float t = (float)x[v.at(b, g * D + d, p)] - mean;
        sq = fmaf(t, t, sq);
    }
    sq = block_sum(sq, red);
    if (threadIdx.x == 0) {
        stats[2 * blockIdx.x] = mean;
        stats[2 * blockIdx.x + 1] = rsqrtf(sq / (float)n + eps);
    }
}

template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void k_gn_apply(const TX* __restrict__ x, const float* __restrict__ w,
                                                       const float* __restrict__ bias,
                                                       const float* __restrict__ stats, TY* __restrict__ out, View v,
                                                       bool out_last) {
    const int64_t total = v.B * v.C * v.P;
    View o = v;
    o.last = out_last;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t b = i / (v.C * v.P), r = i % (v.C * v.P);
        const int64_t c = out_last ? r % v.C : r / v.P, p = out_last ? r / v.C : r % v.P;
        const float* st = stats + 2 * (b * v.G + c / (v.C / v.G));
        const float xh = ((float)x[v.at(b, c, p)] - st[0]) * st[1];
        out[i] = (TY)act_value<ACT>(fmaf(xh, w ? w[c] : 1.0f, bias ? bias[c] : 0.0f));
    }
}

// One workgroup per (item, channel): part[b][c] = (sum g, sum g xh).
template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void k_gn_bwd_sums(const TX* __restrict__ x, const TY* __restrict__ dy,
                                                          const float* __restrict__ w,
                                                          const float* __restrict__ bias,
                                                          const float* __restrict__ stats, float2* __restrict__ part,
                                                          View v, bool out_last) {
    __shared__ float red[16];
    const int64_t b = blockIdx.x / v.C, c = blockIdx.x % v.C;
    const float* st = stats + 2 * (b * v.G + c / (v.C / v.G));
    const float wc = w ? w[c] : 1.0f, bc = bias ? bias[c] : 0.0f;
    View o = v;
    o.last = out_last;
    float sg = 0.0f, sgx = 0.0f;
    for (int64_t p = threadIdx.x; p < v.P; p += kThreads) {
        const float xh = ((float)x[v.at(b, c, p)] - st[0]) * st[1];
        const float g = (float)dy[o.at(b, c, p)] * act_slope<ACT>(fmaf(xh, wc, bc));
        sg += g;
        sgx = fmaf(g, xh, sgx);
    }
    sg = block_sum(sg, red);
    sgx = block_sum(sgx, red);
    if (threadIdx.x == 0) part[blockIdx.x] = make_float2(sg, sgx);
}

// Items B G: gsum[b][g] = (s1, s2).  Items B G + c: grad_weight, grad_bias.
__global__ __launch_bounds__(kThreads) void k_gn_bwd_reduce(const float2* __restrict__ part,
                                                            const float* __restrict__ w, float2* __restrict__ gsum,
                                                            float* __restrict__ gw, float* __restrict__ gb, View v) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i < v.B * v.G) {
        const int64_t b = i / v.G, g = i % v.G, D = v.C / v.G;
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = g * D; c < (g + 1) * D; ++c) {
            const float2 q = part[b * v.C + c];
            const float wc = w ? w[c] : 1.0f;
            s1 = fmaf(wc, q.x, s1);
            s2 = fmaf(wc, q.y, s2);
        }
        const float inv = 1.0f / ((float)D * (float)v.P);
        gsum[i] = make_float2(s1 * inv, s2 * inv);
    } else if (i < v.B * v.G + v.C) {
        const int64_t c = i - v.B * v.G;
        float sg = 0.0f, sgx = 0.0f;
        for (int64_t b = 0; b < v.B; ++b) {
            const float2 q = part[b * v.C + c];
            sg += q.x;
            sgx += q.y;
        }
        if (gw) gw[c] = sgx;
        if (gb) gb[c] = sg;
    }
}

template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void k_gn_bwd_apply(const TX* __restrict__ x, const TY* __restrict__ dy,
                                                           const float* __restrict__ w,
                                                           const float* __restrict__ bias,
                                                           const float* __restrict__ stats,
                                                           const float2* __restrict__ gsum, TX* __restrict__ gx,
                                                           View v, bool out_last) {
    const int64_t total = v.B * v.C * v.P;
    View o = v;
    o.last = out_last;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t b = i / (v.C * v.P), r = i % (v.C * v.P);
        const int64_t c = v.last ? r % v.C : r / v.P, p = v.last ? r / v.C : r % v.P;
        const int64_t gi = b * v.G + c / (v.C / v.G);
        const float rstd = stats[2 * gi + 1], wc = w ? w[c] : 1.0f;
        const float xh = ((float)x[i] - stats[2 * gi]) * rstd;
        const float g = (float)dy[o.at(b, c, p)] * act_slope<ACT>(fmaf(xh, wc, bias ? bias[c] : 0.0f));
        const float2 s = gsum[gi];
        gx[i] = (TX)(rstd * (fmaf(g, wc, -s.x) - xh * s.y));
    }
}

template <typename F>
hipError_t with_types(const GroupNorm& g, F&& f) {
    switch (g.x_type * 4 + g.out_type) {
        case kTypeF32 * 4 + kTypeF32: return f(float{}, float{});
        case kTypeBf16 * 4 + kTypeBf16: return f(bf16{}, bf16{});
        case kTypeBf16 * 4 + kTypeF32: return f(bf16{}, float{});
        case kTypeF16 * 4 + kTypeF16: return f(f16{}, f16{});
        default: return f(f16{}, float{});
    }
}
template <typename F>
hipError_t with_act(int act, F&& f) {
    switch (act) {
        case kActGelu: return f(std::integral_constant<int, kActGelu>{});
        case kActSilu: return f(std::integral_constant<int, kActSilu>{});
        default: return f(std::integral_constant<int, kActNone>{});
    }
}

}  // namespace

int group_norm_kernels(const GroupNorm&, bool backward, bool need_x, const char** names) {
    names[0] = backward ? "gn_bwd_sums" : "gn_stats";
    names[1] = backward ? "gn_bwd_reduce" : "gn_apply";
    names[2] = "gn_bwd_apply";
    return backward && need_x ? 3 : 2;
}

size_t group_norm_workspace(const GroupNorm& g) { return sizeof(float2) * (size_t)(g.B * g.C + g.B * g.groups); }

hipError_t launch_group_norm(const GroupNorm& g, const GroupNormArgs& a, bool backward, int kernel, hipStream_t s) {
    const View v{g.B, g.C, g.P, g.groups, g.x_last};
    const unsigned flat = (unsigned)std::min<int64_t>((g.B * g.C * g.P + kThreads - 1) / kThreads, 8192);
    float2* part = static_cast<float2*>(a.ws);
    float2* gsum = part + g.B * g.C;
    return with_types(g, [&](auto tx, auto ty) {
        using TX = decltype(tx);
        using TY = decltype(ty);
        const TX* x = static_cast<const TX*>(a.x);
        TY* o = static_cast<TY*>(a.out);
        return with_act(g.act, [&](auto act) {
            constexpr int ACT = decltype(act)::value;
            if (!backward && kernel == 0)
                return launch_kernel(k_gn_stats<TX>, dim3((unsigned)(g.B * g.groups)), dim3(kThreads), 0, s, x,
                                     a.stats, v, g.eps);
            if (!backward)
                return launch_kernel(k_gn_apply<ACT, TX, TY>, dim3(flat), dim3(kThreads), 0, s, x, a.weight, a.bias,
                                     (const float*)a.stats, o, v, g.out_last);
            if (kernel == 0)
                return launch_kernel(k_gn_bwd_sums<ACT, TX, TY>, dim3((unsigned)(g.B * g.C)), dim3(kThreads), 0, s, x,
                                     (const TY*)o, a.weight, a.bias, (const float*)a.stats, part, v, g.out_last);
            if (kernel == 1)
                return launch_kernel(k_gn_bwd_reduce,
                                     dim3((unsigned)((g.B * g.groups + g.C + kThreads - 1) / kThreads)),
                                     dim3(kThreads), 0, s, (const float2*)part, a.weight, gsum, a.grad_weight,
                                     a.grad_bias, v);
            return launch_kernel(k_gn_bwd_apply<ACT, TX, TY>, dim3(flat), dim3(kThreads), 0, s, x, (const TY*)o,
                                 a.weight, a.bias, (const float*)a.stats, (const float2*)gsum,
                                 static_cast<TX*>(a.grad_x), v, g.out_last);
        });
    });
}

}  // namespace fno
