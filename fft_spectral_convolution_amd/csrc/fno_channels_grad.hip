// Gradient of the weight of channel products with more channels than one kernel
// takes (fno_channels_bwd.hpp): grad_W[o][i] = sum over positions g[o] x[i].
//
// A workgroup takes 64 x 64 channels and a share of the positions, its waves 32
// positions at a time: both operands are turned by products with the identity
// and stay in registers, as in the one-kernel pass.  A field is read once for every 64
// channels of the other, mostly from the caches.  256 -> 256 bfloat16, 65536
// positions: the four kernels of the backward pass 158 to 165 us (283 with operands
// loaded value by value), against 100 MB, 20 us: this one 69, forming z and g 56, grad_x 40, the joining 5.
#include "fno_channels.hpp"

namespace fno {
namespace {

// (Two waves a SIMD where the registers of 16-bit fields' parts leave room.)
template <typename T, typename TG, bool LAST, bool G_LAST>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void k_weight_grad(WeightGradArgs a) {
    typedef Scheme<T> S;
    __shared__ float join[4096];
    __shared__ float sums[64];
    __shared__ uint32_t marked[128], spoilt;         // rows o, columns i; whether any
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // shares of the same positions are neighbours
    const int parts_in = (a.Cin + 63) / 64, parts = parts_in * ((a.Cout + 63) / 64);
    const int share = blockIdx.x / parts, part = blockIdx.x % parts;
    const int i0 = part % parts_in * 64, o0 = part / parts_in * 64;

    if (threadIdx.x < 128) marked[threadIdx.x] = 0;
    spoilt = 1;
    __syncthreads();
    bf16x8 one[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) one[s][i] = (lane & 31) == 16 * h + 8 * s + i ? 1.0f : 0.0f;
    f32x16 dw[2][2];
    float db[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int r = 0; r < 16; ++r) dw[u][v][r] = 0.0f;

    Values<T> x[2];
    Values<TG> g[2];
    auto tile_at = [&](int64_t t) __attribute__((always_inline)) {
        Tile q;
        q.item = a.merged ? 0 : t / a.tiles_item;
        q.p0 = (a.merged ? t : t % a.tiles_item) * 32;
        q.pn = 1;
        q.pj = 0;
        q.full = q.p0 + 32 <= a.P;
        return q;
    };
    auto fetch = [&](int64_t t) __attribute__((always_inline)) {
        const Tile q = tile_at(t);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (i0 + 32 * u < a.Cin) Places<T, LAST, 1>(q, a.Cin, a.P, a.B, i0 + 32 * u).fetch(a.x, 0, x[u]);
            if (o0 + 32 * u < a.Cout) Places<TG, G_LAST, 1>(q, a.Cout, a.P, a.B, o0 + 32 * u).fetch(a.g, 0, g[u]);
        }
    };
    const int64_t stride = (int64_t)a.splits * 4;
    int64_t t = (int64_t)share * 4 + wave;
    if (t < a.tiles) fetch(t);
    for (; t < a.tiles; t += stride) {
        Frag<bf16x8, S::x> xs[2][2], xt[2][2];
        Frag<bf16x8, 3> gs[2][2], gt[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            x[u].keep(a.Cin, i0 + 32 * u);
            g[u].keep(a.Cout, o0 + 32 * u);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                xs[u][s] = step_of<S::x>(x[u].v, s);
                gs[u][s] = step_of<3>(g[u].v, s);
            }
        }
        if (t + stride < a.tiles) fetch(t + stride);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            turned(xs[u], one, xt[u]);
            db[u] += turned(gs[u], one, gt[u]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int s = 0; s < 2; ++s) dw[u][v] = mfma_upto<S::gw>(gt[u][s], xt[v][s], dw[u][v]);
    }
    float* const to = a.part + (int64_t)share * (a.Cin + 1) * a.Cout;
    if (__builtin_expect(!__builtin_amdgcn_readfirstlane(__syncthreads_or(any_not_finite<2, 2>(dw, db))), 1)) {
        join_sums<2, 2>(dw, db, join, sums, nullptr, nullptr, nullptr, to, o0, i0, a.Cout, a.Cin);
        return;
    }
    // the sums again, 32 x 32 channels at a time, with what is not finite set apart
#pragma unroll 1
    for (int block = 0; block < 4; ++block) {
        const int u = block >> 1, v = block & 1;
        if (o0 + 32 * u >= a.Cout || i0 + 32 * v >= a.Cin) continue;
        f32x16 sum[1][1];
        float sum_b[1] = {0.0f};
#pragma unroll
        for (int r = 0; r < 16; ++r) sum[0][0][r] = 0.0f;
#pragma unroll 1
        for (t = (int64_t)share * 4 + wave; t < a.tiles; t += stride) {
            const Tile q = tile_at(t);
            Values<TG> gv;
            Values<T> xv;
            Places<TG, G_LAST, 1>(q, a.Cout, a.P, a.B, o0 + 32 * u).fetch(a.g, 0, gv);
            Places<T, LAST, 1>(q, a.Cin, a.P, a.B, i0 + 32 * v).fetch(a.x, 0, xv);
            gv.keep(a.Cout, o0 + 32 * u);
            xv.keep(a.Cin, i0 + 32 * v);
            Frag<bf16x8, 3> gs[2], gt[2];
            Frag<bf16x8, S::x> xs[2], xt[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                gs[s] = step_of<3>(gv.v, s);
                xs[s] = step_of<S::x>(xv.v, s);
            }
            set_apart(gs, marked + 32 * u);
            sum_b[0] += turned(gs, one, gt);
            set_apart(xs, marked + 64 + 32 * v);
            turned(xs, one, xt);
#pragma unroll
            for (int s = 0; s < 2; ++s) sum[0][0] = mfma_upto<S::gw>(gt[s], xt[s], sum[0][0]);
        }
        join_sums<1, 1>(sum, sum_b, join, sums, &spoilt, marked + 32 * u, marked + 64 + 32 * v, to, o0 + 32 * u,
                        i0 + 32 * v, a.Cout, a.Cin);
    }
}

template <typename T, typename TG>
hipError_t launch(const WeightGradArgs& a, bool last, bool g_last, hipStream_t s) {
    const dim3 grid((unsigned)(a.splits * (int64_t)((a.Cin + 63) / 64) * ((a.Cout + 63) / 64))), block(256);
    if (last && g_last) return launch_kernel(k_weight_grad<T, TG, true, true>, grid, block, 0, s, a);
    if (last) return launch_kernel(k_weight_grad<T, TG, true, false>, grid, block, 0, s, a);
    if (g_last) return launch_kernel(k_weight_grad<T, TG, false, true>, grid, block, 0, s, a);
    return launch_kernel(k_weight_grad<T, TG, false, false>, grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_channel_weight_grad(WeightGradArgs a, int x_type, int g_type, bool x_last, bool g_last,
                                      hipStream_t s) {
    a.merged = x_last && g_last;
    if (a.merged) {
        a.P *= a.B;
        a.B = 1;
    }
    a.tiles_item = (int)((a.P + 31) / 32);
    a.tiles = a.B * a.tiles_item;
    if (x_type == kTypeF32) return launch<float, float>(a, x_last, g_last, s);
    if (x_type == kTypeBf16 && g_type == kTypeF32) return launch<bf16, float>(a, x_last, g_last, s);
    if (x_type == kTypeBf16) return launch<bf16, bf16>(a, x_last, g_last, s);
    return g_type == kTypeF32 ? launch<f16, float>(a, x_last, g_last, s) : launch<f16, f16>(a, x_last, g_last, s);
}

}  // namespace fno
