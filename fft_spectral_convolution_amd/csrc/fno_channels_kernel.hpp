// Channel product of a field with its epilogue:
//   z[b,o,p] = sum_i W[o,i] x[b,i,p] + bias[o],  out = act(z + branch) or act(z) + branch.
//
// A wave takes 32 NT positions and 32 MT output channels: x goes from memory
// to registers as the operand it is (fno_channels.hpp), the weight stays in LDS
// as parts in the order of the operands, and the result leaves from registers.
//
// Included by one source file for each type of x, so that they build side by side.
#pragma once

#include <algorithm>

#include "fno_channels.hpp"

namespace fno {
namespace {

constexpr int kProductThreads = 512;

// Eight weights of output channel o from input channel i on, zero where there are none.  (All loads
// at once, those outside the weight from its start: a branch for each would wait for each.)
__device__ __forceinline__ void weights_at(const ProductArgs& a, int o, int i, float (&v)[8]) {
    with_field_type(a.w_type, [&](auto e) {
        typedef decltype(e) W;
        const W* w = static_cast<const W*>(a.w);
        const int64_t at = a.transposed ? (int64_t)i * a.Cout + o : (int64_t)o * a.Cin + i;
        const int step = a.transposed ? a.Cout : 1;
        W q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = w[o < a.Cout && i + k < a.Cin ? at + (int64_t)k * step : 0];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = o < a.Cout && i + k < a.Cin ? (float)q[k] : 0.0f;
    });
}

template <int ACT, bool FINE>
__device__ __forceinline__ void activate(float (&z)[16], bool slope) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = slope ? act_slope<ACT>(z[i]) : product_act<ACT, FINE>(z[i]);
}

// Parts of x and of the weight, and the products of them that are formed (i + j up to `most`).  A
// float32 x with a 16-bit result is the g of a 16-bit field's backward pass: the weight is of the
// result's type, held exactly by one (bfloat16) or two parts.  Two parts of g are within 2^-17 of it, and a float16
// weight's product leaves out its second part with g's, up to 2^-16: a step of the result is 2^-7 or 2^-10.
template <typename T, typename TO>
struct Parts {
    static constexpr bool g = sizeof(T) == 4 && sizeof(TO) == 2;
    static constexpr int x = g ? 2 : Operand<T>::parts, w = weight_parts(Operand<T>::type, Operand<TO>::type),
                         most = g ? 1 : Operand<T>::parts - 1;
};

// What bounds it: 64 -> 64 float32 channels first with a branch and GELU, 524288 positions,
// 80 to 89 us, 403 MB at 4.5 to 5.0 TB/s, memory (the float32 matrix instructions alone would take 27 us at
// their peak, the six part products 10); 3 -> 64 from channels last 27 us, 140 MB at 5.1
// TB/s.  64 -> 256 bfloat16 channels last with GELU 155 to 164 us, 335 MB at 2.1 TB/s, no one unit: 23
// vector instructions a value of the output take half of the time, 45% of the waves' time is waiting.  Without the
// activation (10 instructions) 114 us, with the output channels first as well, so not turned through LDS, 78 of a
// floor of 66: with two waves a SIMD neither the activation nor the turning hides behind memory.  256 -> 256 with
// SiLU and a residual, 65536 positions, 43 to 46 us, of which 12 do not grow with the positions: the staging
// of the weight and the first loads of x behind it (262144 positions: 135 us, floor 79).
// Two waves a SIMD with 64 or 32 channels of x on the way measured faster than three or four without
// (64 -> 256: 164 against 208 and 268 us; 64 -> 64: 81 against 98 and 132).
template <typename T, typename TO, bool LAST, bool OUT_LAST, int MT, int NT>
__global__ __launch_bounds__(kProductThreads, MT * NT <= 2 ? 3 : 2) void k_channels(ProductArgs a) {
    typedef Parts<T, TO> Q;
    typedef typename Operand<T>::V V;
    constexpr int parts = Q::x, wparts = Q::w, ahead = steps_ahead(Operand<T>::type);
    extern __shared__ __align__(16) unsigned char lds[];
    V* wfrag = reinterpret_cast<V*>(lds);                     // [part][mt][chunk][64]
    float* bias = reinterpret_cast<float*>(wfrag + wparts * MT * a.chunk * 64);
    const int lane = threadIdx.x & 63, h = lane >> 5;
    unsigned char* const turn = reinterpret_cast<unsigned char*>(bias + 32 * MT) + (threadIdx.x >> 6) * kTurnBytes;
    const int waves = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Neighbouring workgroups are on different XCDs: those that read the same positions for
    // other output channels are eight apart, on one XCD, and share its L2.
    const int lanes8 = a.groups % 8 == 0 ? 8 : 1;
    const int slot = blockIdx.x / lanes8, c0 = slot % a.cout_tiles * 32 * MT;
    const int64_t group = (int64_t)(slot / a.cout_tiles) * lanes8 + blockIdx.x % lanes8, groups = a.groups;

    auto stage = [&](int first) {
        const int steps = min(a.chunk, a.nks - first);
        for (int q = threadIdx.x; q < MT * steps * 64; q += blockDim.x) {
            const int l = q & 63, mt = (q >> 6) / steps, ks = (q >> 6) % steps;
            const int o = c0 + 32 * mt + row_channel(l & 31), k = 16 * (first + ks) + 8 * (l >> 5);
            float v[8];
            weights_at(a, o, k, v);
            const Frag<V, wparts> f = split<V, wparts>(v);
#pragma unroll
            for (int p = 0; p < wparts; ++p) wfrag[((p * MT + mt) * a.chunk + ks) * 64 + l] = f.part[p];
        }
    };
    auto tile_at = [&](int64_t t) {
        Tile q;
        q.item = a.merged ? 0 : t / a.tiles_item;
        q.p0 = (a.merged ? t : t % a.tiles_item) * (32 * NT);
        q.pn = a.merged ? 1 : NT;
        q.pj = a.merged ? 32 : 1;
        q.full = q.p0 + 32 * NT <= a.P;
        return q;
    };
    for (int i = threadIdx.x; i < 32 * MT; i += blockDim.x)
        bias[i] = a.bias && c0 + i < a.Cout ? a.bias[c0 + i] : 0.0f;
    const bool once = a.chunk >= a.nks;
    if (once) stage(0);
    __syncthreads();

    const int64_t stride = groups * waves;
    // every wave of a workgroup makes the same number of rounds (the barriers of staged weights)
    const int64_t rounds = (a.tiles + stride - 1) / stride;
    Raw<T, LAST, NT> raw[ahead];
    int64_t t = group * waves + wave;
    Tile tile = tile_at(min(t, a.tiles - 1));
#pragma unroll
    for (int k = 0; k < ahead; ++k)
        if (t < a.tiles && k < a.nks) load_raw(raw[k], a.x, tile, a.Cin, a.P, a.B, 16 * k);
    for (int64_t round = 0; round < rounds; ++round, t += stride) {
        const bool live = t < a.tiles;
        const Tile next = tile_at(min(t + stride, a.tiles - 1));
        f32x16 acc[MT][NT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[mt][j][r] = bias[32 * mt + 16 * h + r];
        for (int first = 0; first < a.nks; first += a.chunk) {
            if (!once) {
                __syncthreads();
                stage(first);
                __syncthreads();
            }
            if (!live) continue;
            const int steps = min(a.chunk, a.nks - first);
            for (int base = 0; base < steps; base += ahead) {
#pragma unroll
                for (int k = 0; k < ahead; ++k) {
                    const int ks = base + k;
                    if (ks >= steps) break;
                    Frag<V, parts> b[NT];
                    raw[k].keep(a.Cin, 16 * (first + ks));
#pragma unroll
                    for (int j = 0; j < NT; ++j) b[j] = operand<parts>(raw[k], j);
                    if (first + ks + ahead < a.nks) {
                        load_raw(raw[k], a.x, tile, a.Cin, a.P, a.B, 16 * (first + ks + ahead));
                    } else if (t + stride < a.tiles) {
                        load_raw(raw[k], a.x, next, a.Cin, a.P, a.B, 16 * k);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        Frag<V, wparts> w;
#pragma unroll
                        for (int p = 0; p < wparts; ++p) w.part[p] = wfrag[((p * MT + mt) * a.chunk + ks) * 64 + lane];
#pragma unroll
                        for (int j = 0; j < NT; ++j) acc[mt][j] = mfma_upto<Q::most>(w, b[j], acc[mt][j]);
                    }
                }
            }
        }
        if (!live) continue;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            int c = c0 + 32 * mt;
            if (c >= a.Cout) break;
            asm volatile("" : "+s"(c));          // (formed here, not for all parts before the first)
            const Places<TO, OUT_LAST, NT> at(tile, a.Cout, a.P, a.B, c);
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                float z[16], u[16];
                if (a.branch) at.load(a.branch, q, u);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int j = chunk_pos<OUT_LAST, NT>(q, i), r = chunk_row<OUT_LAST, NT>(q, i);
                    z[i] = acc[mt][j][r];
                }
                if (a.branch && !a.branch_after) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) z[i] += u[i];
                }
                if (a.act == kActGelu) activate<kActGelu, sizeof(TO) == 4>(z, a.slope);
                else if (a.act == kActSilu) activate<kActSilu, true>(z, a.slope);
                if (a.slope) {
                    at.load(a.grad, q, u);
#pragma unroll
                    for (int i = 0; i < 16; ++i) z[i] *= u[i];
                    Places<float, OUT_LAST, NT>(tile, a.Cout, a.P, a.B, c).store(a.g, q, z, turn);
                } else if (a.branch && a.branch_after) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) z[i] += u[i];
                }
                if (a.out) at.store(a.out, q, z, turn);
            }
        }
        tile = next;
    }
}

template <typename T, typename TO, bool LAST, bool OUT_LAST, int MT, int NT>
hipError_t launch_tiles(ProductArgs a, const ProductPlan& plan, hipStream_t s) {
    a.tiles_item = (int)((a.P + 32 * NT - 1) / (32 * NT));
    a.tiles = a.B * a.tiles_item;
    a.cout_tiles = (a.Cout + 32 * MT - 1) / (32 * MT);
    a.nks = plan.nks;
    a.chunk = plan.chunk;
    const int waves = plan.waves;
    // as many waves as the CUs hold; groups of workgroups that read the same positions are dealt out in eights
    const int64_t most_groups = 256 * (MT * NT <= 2 ? 3 : 2) * 4 / waves / std::min(a.cout_tiles, 8);
    a.groups = (int)std::max<int64_t>(1, std::min<int64_t>((a.tiles + waves - 1) / waves, most_groups));
    if (a.groups > 8) a.groups = (a.groups + 7) / 8 * 8;
    const size_t lds = (size_t)a.chunk * Parts<T, TO>::w * MT * 1024 + 32 * MT * sizeof(float) +
                       (OUT_LAST ? waves * kTurnBytes : 0);
    return launch_kernel(k_channels<T, TO, LAST, OUT_LAST, MT, NT>, dim3((unsigned)(a.groups * a.cout_tiles)),
                         dim3(64 * waves), lds, s, a);
}

template <typename T, typename TO, bool LAST, bool OUT_LAST>
hipError_t launch_couts(const ProductArgs& a, hipStream_t s) {
    constexpr bool merged = LAST && OUT_LAST;
    constexpr int NT = positions_a_wave(merged) / 32;
    const ProductPlan plan = plan_product(a, Operand<T>::type, Operand<TO>::type, merged);
    if (plan.mt == 4) return launch_tiles<T, TO, LAST, OUT_LAST, 4, NT>(a, plan, s);
    if (plan.mt == 2) return launch_tiles<T, TO, LAST, OUT_LAST, 2, NT>(a, plan, s);
    return launch_tiles<T, TO, LAST, OUT_LAST, 1, NT>(a, plan, s);
}

// all channels last: one run of positions
template <typename T, typename TO>
hipError_t launch_layouts(ProductArgs a, bool last, bool out_last, hipStream_t s) {
    a.merged = last && out_last;
    if (a.merged) {
        a.P *= a.B;
        a.B = 1;
        return launch_couts<T, TO, true, true>(a, s);
    }
    if (last) return launch_couts<T, TO, true, false>(a, s);
    return out_last ? launch_couts<T, TO, false, true>(a, s) : launch_couts<T, TO, false, false>(a, s);
}

}  // namespace
}  // namespace fno
