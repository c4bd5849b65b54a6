// Backward pass of a channel product, everything in one pass over x and grad_out:
//   z = W x + bias (+ branch),  g = grad_out act'(z),
//   grad_x = W^T g,  grad_W += g x^T,  grad_bias += g.
//
// A wave takes 32 positions at a time and all channels.  The result of a product
// (fno_channels.hpp) has positions in lanes and 16 channels in a lane's
// registers, which is an operand again: two steps of 8 of them, channel
// 16 (lane / 32) + 8 s + i in step s.  x is loaded in the same order, so z's operands,
// g's for W^T g and both transposes share it.  grad_W sums over positions, so its
// operands have channels in lanes: they are turned by products with the
// identity, exactly, part by part, without a byte of LDS; the turned
// positions come in an order that is the same for g and x.  Sums of grad_W stay in
// registers over all of a wave's tiles; then those of a workgroup's waves are
// joined in LDS and the workgroups' by k_weight_sum, in a fixed order.
//
// Channels and positions that do not exist are zeros of both operands.
//
// g of a 16-bit field is three bfloat16 parts as a float32 one's is: the parameters'
// gradients are float32 sums, in which two parts would leave up to 2^-17 of every g.  grad_x,
// rounded to 16 bits, takes two of them, of float16 without the second parts' product (2^-16).  x
// and W of float16 are two parts each, which hold them exactly.
//
// Included by one source file for each pair of types, so that they build side by side.
#pragma once

#include "fno_channels.hpp"

namespace fno {
namespace {

// 64 -> 64 float32 channels first with a branch and GELU, 524288 positions: 184 to 190 us, 671 MB at 3.5 to 3.6
// TB/s; 64 -> 128 bfloat16 channels last 159 to 161 us, 269 MB at 1.7 TB/s; 30 -> 50 float16, 8601 positions, 18
// us, two launches.  One wave a SIMD (the sums, a tile's operands and the next tile's
// fields take up to 512 registers) leaves latencies in the open: of the first case's 30 000 cycles a tile
// and SIMD, matrix instructions take 5400, vector instructions about 11 000.  Two waves with the
// same state spilled (254 us); four phases with less alive spilled as well (311 us).
template <typename T, typename TG, bool LAST, bool OUT_LAST, int MO, int MI>
__global__ __launch_bounds__(256, MO * MI == 1 ? 2 : 1) void k_channels_bwd(BackwardArgs a) {
    typedef Scheme<T> S;
    typedef Frag<bf16x8, S::x> FX;
    typedef Frag<bf16x8, 3> FG;
    extern __shared__ __align__(16) unsigned char lds[];
    bf16x8* wz = reinterpret_cast<bf16x8*>(lds);             // [part][mo][mi][step][64]: rows o, steps over i
    bf16x8* wx = wz + S::x * MO * MI * 128;                  // [part][mi][mo][step][64]: rows i, steps over o
    float* bias = reinterpret_cast<float*>(wx + S::x * MO * MI * 128);
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t* const marked = reinterpret_cast<uint32_t*>(bias + 32 * MO);        // rows o, columns i, whether any
    unsigned char* const turn =
        reinterpret_cast<unsigned char*>(marked + 32 * (MO + MI + 1)) + (threadIdx.x >> 6) * kTurnBytes;

    const T* w = static_cast<const T*>(a.w);
    for (int q = threadIdx.x; q < MO * MI * 128; q += 256) {
        const int l = q & 63, s = (q >> 6) & 1, mi = (q >> 7) % MI, mo = (q >> 7) / MI;
        const int row = row_channel(l & 31), k = 16 * (l >> 5) + 8 * s;
        // (all loads at once, those outside the weight from its start: a branch for each would wait for each)
        T p[8], r[8];
        float v[8], u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int o = 32 * mo + row, ci = 32 * mi + k + i, o2 = 32 * mo + k + i, ci2 = 32 * mi + row;
            p[i] = w[o < a.Cout && ci < a.Cin ? o * a.Cin + ci : 0];
            r[i] = w[o2 < a.Cout && ci2 < a.Cin ? o2 * a.Cin + ci2 : 0];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = 32 * mo + row < a.Cout && 32 * mi + k + i < a.Cin ? (float)p[i] : 0.0f;
            u[i] = 32 * mo + k + i < a.Cout && 32 * mi + row < a.Cin ? (float)r[i] : 0.0f;
        }
        const FX f = split<bf16x8, S::x>(v), g = split<bf16x8, S::x>(u);
#pragma unroll
        for (int p = 0; p < S::x; ++p) {
            wz[(((p * MO + mo) * MI + mi) * 2 + s) * 64 + l] = f.part[p];
            wx[(((p * MI + mi) * MO + mo) * 2 + s) * 64 + l] = g.part[p];
        }
    }
    for (int i = threadIdx.x; i < 32 * MO; i += 256) bias[i] = a.bias && i < a.Cout ? a.bias[i] : 0.0f;
    for (int i = threadIdx.x; i <= 32 * (MO + MI); i += 256) marked[i] = 0;
    __syncthreads();

    bf16x8 one[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) one[s][i] = (lane & 31) == 16 * h + 8 * s + i ? 1.0f : 0.0f;

    f32x16 dw[MO][MI];
    float db[MO];
#pragma unroll
    for (int mo = 0; mo < MO; ++mo) {
        db[mo] = 0.0f;
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int r = 0; r < 16; ++r) dw[mo][mi][r] = 0.0f;
    }
    auto tile_at = [&](int64_t t) __attribute__((always_inline)) {
        Tile q;
        q.item = a.merged ? 0 : t / a.tiles_item;
        q.p0 = (a.merged ? t : t % a.tiles_item) * 32;
        q.pn = 1;
        q.pj = 0;
        q.full = q.p0 + 32 <= a.P;
        return q;
    };
    auto fetch_x = [&](Values<T> (&raw)[MI], const Tile& t) __attribute__((always_inline)) {
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
            if (32 * mi < a.Cin) {
                Places<T, LAST, 1>(t, a.Cin, a.P, a.B, 32 * mi).fetch(a.x, 0, raw[mi]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) raw[mi].v[i] = (T)0.0f;
            }
        }
    };

    if constexpr (MI <= 2) {
        // Of each field the next tile's values are on their way from the moment that this tile's are used.
        const int64_t stride = (int64_t)a.groups * 4;
        int64_t t = (int64_t)blockIdx.x * 4 + wave;
        if (t >= a.tiles) t = a.tiles;
        Values<T> raw[MI];
        Values<TG> go[MO], br[MO];
        Tile tile = tile_at(min(t, a.tiles - 1));
        if (t < a.tiles) {
            fetch_x(raw, tile);
#pragma unroll
            for (int mo = 0; mo < MO; ++mo)
                if (32 * mo < a.Cout) {
                    const Places<TG, OUT_LAST, 1> at(tile, a.Cout, a.P, a.B, 32 * mo);
                    at.fetch(a.grad, 0, go[mo]);
                    if (a.branch) at.fetch(a.branch, 0, br[mo]);
                }
        }
        for (; t < a.tiles; t += stride) {
            const bool more = t + stride < a.tiles;
            const Tile next = tile_at(min(t + stride, a.tiles - 1));
            FX x[MI][2], xt[MI][2];
#pragma unroll
            for (int mi = 0; mi < MI; ++mi) {
                raw[mi].keep(a.Cin, 32 * mi);
#pragma unroll
                for (int s = 0; s < 2; ++s) x[mi][s] = step_of<S::x>(raw[mi].v, s);
            }
            if (more) fetch_x(raw, next);

            // z of all output channels first, so that x is no longer needed but turned; of 128, whose z would
            // take 64 registers, 32 at a time
            constexpr bool kEach = MO == 4;
            f32x16 z[kEach ? 1 : MO];
            auto form_z = [&](int mo, f32x16& q) {
#pragma unroll
                for (int r = 0; r < 16; ++r) q[r] = bias[32 * mo + 16 * h + r];
#pragma unroll
                for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        FX f;
#pragma unroll
                        for (int p = 0; p < S::x; ++p) f.part[p] = wz[(((p * MO + mo) * MI + mi) * 2 + s) * 64 + lane];
                        q = mfma_upto<S::z>(f, x[mi][s], q);
                    }
            };
            if (!kEach && a.act != kActNone) {
#pragma unroll
                for (int mo = 0; mo < MO; ++mo) form_z(mo, z[mo]);
            }
            if (a.part) {
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) turned(x[mi], one, xt[mi]);
            }
            f32x16 dx[MI];
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                for (int r = 0; r < 16; ++r) dx[mi][r] = 0.0f;
#pragma unroll
            for (int mo = 0; mo < MO; ++mo) {
                int c = 32 * mo;
                if (c >= a.Cout) break;
                asm volatile("" : "+s"(c));
                float g[16];
                go[mo].keep(a.Cout, c);
#pragma unroll
                for (int i = 0; i < 16; ++i) g[i] = (float)go[mo].v[i];
                if (a.act != kActNone) {
                    f32x16& q = z[kEach ? 0 : mo];
                    if (kEach) form_z(mo, q);
                    if (a.branch) {
                        br[mo].keep(a.Cout, c);
#pragma unroll
                        for (int i = 0; i < 16; ++i) q[i] += (float)br[mo].v[i];
                    }
                    if (a.act == kActGelu) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) g[i] *= act_slope<kActGelu>(q[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) g[i] *= act_slope<kActSilu>(q[i]);
                    }
                    if (a.grad_branch)
                        Places<TG, OUT_LAST, 1>(tile, a.Cout, a.P, a.B, c).store(a.grad_branch, 0, g, turn);
                }
                if (more) {
                    const Places<TG, OUT_LAST, 1> at(next, a.Cout, a.P, a.B, c);
                    at.fetch(a.grad, 0, go[mo]);
                    if (a.branch) at.fetch(a.branch, 0, br[mo]);
                }
                FG gs[2];
#pragma unroll
                for (int s = 0; s < 2; ++s) gs[s] = step_of<3>(g, s);
                if (a.grad_x) {
#pragma unroll
                    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            FX f;
#pragma unroll
                            for (int p = 0; p < S::x; ++p)
                                f.part[p] = wx[(((p * MI + mi) * MO + mo) * 2 + s) * 64 + lane];
                            dx[mi] = mfma_upto<S::gx>(f, gs[s], dx[mi]);
                        }
                }
                if (a.part) {
                    FG gt[2];
                    db[mo] += turned(gs, one, gt);
#pragma unroll
                    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                        for (int s = 0; s < 2; ++s) dw[mo][mi] = mfma_upto<S::gw>(gt[s], xt[mi][s], dw[mo][mi]);
                }
            }
            if (a.grad_x) {
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    int c = 32 * mi;
                    if (c >= a.Cin) break;
                    asm volatile("" : "+s"(c));
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = dx[mi][i];
                    Places<T, LAST, 1>(tile, a.Cin, a.P, a.B, c).store(a.grad_x, 0, v, turn);
                }
            }
            tile = next;
        }
    } else {
        auto fetch_g = [&](Values<TG>& go, Values<TG>& br, const Tile& t, int c) {
            if (c >= a.Cout) return;
            const Places<TG, OUT_LAST, 1> at(t, a.Cout, a.P, a.B, c);
            at.fetch(a.grad, 0, go);
            if (a.branch) at.fetch(a.branch, 0, br);
        };
        auto parts_of_x = [&](Values<T> (&raw)[MI], FX (&x)[MI][2]) {
#pragma unroll
            for (int mi = 0; mi < MI; ++mi) {
                raw[mi].keep(a.Cin, 32 * mi);
#pragma unroll
                for (int s = 0; s < 2; ++s) x[mi][s] = step_of<S::x>(raw[mi].v, s);
            }
        };
        auto form_z = [&](const FX (&x)[MI][2], f32x16 (&z)[MO]) {
            if (a.act == kActNone) return;
#pragma unroll
            for (int mo = 0; mo < MO; ++mo) {
#pragma unroll
                for (int r = 0; r < 16; ++r) z[mo][r] = bias[32 * mo + 16 * h + r];
#pragma unroll
                for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        FX f;
#pragma unroll
                        for (int p = 0; p < S::x; ++p) f.part[p] = wz[(((p * MO + mo) * MI + mi) * 2 + s) * 64 + lane];
                        z[mo] = mfma_upto<S::z>(f, x[mi][s], z[mo]);
                    }
            }
        };
        // g of the 32 output channels from c on, stored where it is asked for, and its parts
        auto form_g = [&](const Tile& tile, int c, f32x16& z, Values<TG>& go, Values<TG>& br, FG (&gs)[2]) {
            float g[16];
            go.keep(a.Cout, c);
#pragma unroll
            for (int i = 0; i < 16; ++i) g[i] = (float)go.v[i];
            if (a.act != kActNone) {
                if (a.branch) {
                    br.keep(a.Cout, c);
#pragma unroll
                    for (int i = 0; i < 16; ++i) z[i] += (float)br.v[i];
                }
                if (a.act == kActGelu) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) g[i] *= act_slope<kActGelu>(z[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) g[i] *= act_slope<kActSilu>(z[i]);
                }
                if (a.grad_branch) Places<TG, OUT_LAST, 1>(tile, a.Cout, a.P, a.B, c).store(a.grad_branch, 0, g, turn);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) gs[s] = step_of<3>(g, s);
        };
        auto add_grad_x = [&](const FG (&gs)[2], int mo, int mi, f32x16& dx) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                FX f;
#pragma unroll
                for (int p = 0; p < S::x; ++p) f.part[p] = wx[(((p * MI + mi) * MO + mo) * 2 + s) * 64 + lane];
                dx = mfma_upto<S::gx>(f, gs[s], dx);
            }
        };
        auto store_grad_x = [&](const Tile& tile, int c, const f32x16& dx) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = dx[i];
            Places<T, LAST, 1>(tile, a.Cin, a.P, a.B, c).store(a.grad_x, 0, v, turn);
        };

        const int64_t stride = (int64_t)a.groups * 4;
        int64_t t = (int64_t)blockIdx.x * 4 + wave;
        if (t >= a.tiles) t = a.tiles;
        Values<T> raw[MI];
        Values<TG> go[MO], br[MO];
        Tile tile = tile_at(min(t, a.tiles - 1));
        if (t < a.tiles) {
            fetch_x(raw, tile);
            fetch_g(go[0], br[0], tile, 0);
        }
        // 128 channels of x: all of g first, then 32 input channels at a time, so that fewer of x's values are
        // alive together.  On their way are the next tile's x and the next 32 channels' grad_out and branch.
        for (; t < a.tiles; t += stride) {
            const bool more = t + stride < a.tiles;
            const Tile next = tile_at(min(t + stride, a.tiles - 1));
            FX x[MI][2];
            f32x16 z[MO];
            parts_of_x(raw, x);
            if (more) fetch_x(raw, next);
            form_z(x, z);
            // all of g first, then 32 input channels at a time: fewer of x's values are alive together
            FG gs[MO][2];
#pragma unroll
            for (int mo = 0; mo < MO; ++mo) {
                int c = 32 * mo;
                asm volatile("" : "+s"(c));
                if (mo + 1 < MO) fetch_g(go[mo + 1], br[mo + 1], tile, c + 32);
                if (c < a.Cout) {
                    form_g(tile, c, z[mo], go[mo], br[mo], gs[mo]);
                } else {
                    const float none[16] = {};
                    gs[mo][0] = gs[mo][1] = step_of<3>(none, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            if (more) fetch_g(go[0], br[0], next, 0);
            if (a.grad_x) {
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    int c = 32 * mi;
                    if (c >= a.Cin) break;
                    asm volatile("" : "+s"(c));
                    f32x16 dx;
#pragma unroll
                    for (int r = 0; r < 16; ++r) dx[r] = 0.0f;
#pragma unroll
                    for (int mo = 0; mo < MO; ++mo) add_grad_x(gs[mo], mo, mi, dx);
                    store_grad_x(tile, c, dx);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            if (a.part) {
#pragma unroll
                for (int mo = 0; mo < MO; ++mo) {
                    FG gt[2];
                    db[mo] += turned(gs[mo], one, gt);
                    gs[mo][0] = gt[0];
                    gs[mo][1] = gt[1];
                }
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    FX xt[2];
                    turned(x[mi], one, xt);
#pragma unroll
                    for (int mo = 0; mo < MO; ++mo)
#pragma unroll
                        for (int s = 0; s < 2; ++s) dw[mo][mi] = mfma_upto<S::gw>(gs[mo][s], xt[s], dw[mo][mi]);
                }
            }
            tile = next;
        }
    }

    if (!a.part) return;
    uint32_t* const spoilt = marked + 32 * (MO + MI);
    if (__builtin_expect(any_not_finite<MO, MI>(dw, db), 0)) {
        *spoilt = 1;
        // the wave's sums again, 32 output channels at a time, with what is not finite set apart
#pragma unroll 1
        for (int mo = 0; 32 * mo < a.Cout; ++mo) {
            f32x16 sum[MI];
            float sum_b = 0.0f;
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                for (int r = 0; r < 16; ++r) sum[mi][r] = 0.0f;
#pragma unroll 1
            for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.tiles; t += (int64_t)a.groups * 4) {
                const Tile tile = tile_at(t);
                Values<T> raw[MI];
                fetch_x(raw, tile);
                FX x[MI][2];
                f32x16 z;
#pragma unroll
                for (int r = 0; r < 16; ++r) z[r] = bias[32 * mo + 16 * h + r];
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    raw[mi].keep(a.Cin, 32 * mi);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        x[mi][s] = step_of<S::x>(raw[mi].v, s);
                        FX f;
#pragma unroll
                        for (int p = 0; p < S::x; ++p)
                            f.part[p] = wz[(((p * MO + mo) * MI + mi) * 2 + s) * 64 + lane];
                        z = mfma_upto<S::z>(f, x[mi][s], z);
                    }
                }
                const Places<TG, OUT_LAST, 1> at(tile, a.Cout, a.P, a.B, 32 * mo);
                Values<TG> go, br;
                at.fetch(a.grad, 0, go);
                go.keep(a.Cout, 32 * mo);
                if (a.branch) {
                    at.fetch(a.branch, 0, br);
                    br.keep(a.Cout, 32 * mo);
#pragma unroll
                    for (int i = 0; i < 16; ++i) z[i] += (float)br.v[i];
                }
                float g[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    g[i] = (float)go.v[i];
                    if (a.act == kActGelu) g[i] *= act_slope<kActGelu>(z[i]);
                    if (a.act == kActSilu) g[i] *= act_slope<kActSilu>(z[i]);
                }
                FG gs[2], gt[2];
#pragma unroll
                for (int s = 0; s < 2; ++s) gs[s] = step_of<3>(g, s);
                set_apart(gs, marked + 32 * mo);
                sum_b += turned(gs, one, gt);
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    FX xt[2];
                    set_apart(x[mi], marked + 32 * (MO + mi));
                    turned(x[mi], one, xt);
#pragma unroll
                    for (int s = 0; s < 2; ++s) sum[mi] = mfma_upto<S::gw>(gt[s], xt[s], sum[mi]);
                }
            }
#pragma unroll
            for (int m = 0; m < MO; ++m) {
                if (m != mo) continue;
                db[m] = sum_b;
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) dw[m][mi] = sum[mi];
            }
        }
    }
    // (the weights in LDS are no longer needed)
    join_sums<MO, MI>(dw, db, reinterpret_cast<float*>(lds), bias, spoilt, marked, marked + 32 * MO,
                      a.part + (int64_t)blockIdx.x * (a.Cin + 1) * a.Cout, 0, 0, a.Cout, a.Cin);
}

template <typename T, typename TG, bool LAST, bool OUT_LAST, int MO, int MI>
hipError_t launch_backward_tiles(BackwardArgs a, hipStream_t s) {
    const size_t lds = (size_t)2 * Scheme<T>::x * MO * MI * 2048 + 32 * (2 * MO + MI + 1) * sizeof(float) +
                       (LAST || OUT_LAST ? 4 * kTurnBytes : 0);
    return launch_kernel(k_channels_bwd<T, TG, LAST, OUT_LAST, MO, MI>, dim3((unsigned)a.groups), dim3(256), lds, s, a);
}

template <typename T, typename TG, bool LAST, bool OUT_LAST>
hipError_t launch_backward_couts(const BackwardArgs& a, hipStream_t s) {
    if (a.Cin <= 32 && a.Cout <= 32) return launch_backward_tiles<T, TG, LAST, OUT_LAST, 1, 1>(a, s);
    if (a.Cin <= 64 && a.Cout <= 64) return launch_backward_tiles<T, TG, LAST, OUT_LAST, 2, 2>(a, s);
    if constexpr (sizeof(T) == 2) {
        if (a.Cin <= 64) return launch_backward_tiles<T, TG, LAST, OUT_LAST, 4, 2>(a, s);
        return launch_backward_tiles<T, TG, LAST, OUT_LAST, 2, 4>(a, s);
    }
    return hipErrorInvalidValue;         // (backward_fits)
}

template <typename T, typename TG>
hipError_t launch_backward(BackwardArgs a, bool last, bool out_last, hipStream_t s) {
    a.merged = last && out_last;
    if (a.merged) {
        a.P *= a.B;
        a.B = 1;
    }
    a.tiles_item = (int)((a.P + 31) / 32);
    a.tiles = a.B * a.tiles_item;
    if (last && out_last) return launch_backward_couts<T, TG, true, true>(a, s);
    if (last) return launch_backward_couts<T, TG, true, false>(a, s);
    if (out_last) return launch_backward_couts<T, TG, false, true>(a, s);
    return launch_backward_couts<T, TG, false, false>(a, s);
}

}  // namespace
}  // namespace fno
