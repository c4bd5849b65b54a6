// Backward pass of the group norm with an activation.  With xh = (x - mean)
// rstd, z = xh w_c + b_c and g = grad_out act'(z):
//   grad_b_c = sum_{b,p} g,  grad_w_c = sum_{b,p} g xh
//   s1 = sum_group g w_c / n,  s2 = sum_group g w_c xh / n
//   grad_x = rstd (g w_c - s1 - xh s2)
// (mean and rstd depend on every x of the group: the two means take that
// back out.)  All of it follows from the sums of g and g xh over each item's
// channel, so those are what a workgroup forms:
// k_gn_bwd_fused_* keep x and grad_out in registers between the sums and
// grad_x, both read once; larger groups take k_gn_bwd_sums_* (partial sums of
// chunks), k_gn_bwd_finish (s1, s2 and the parameters' gradients) and
// k_gn_bwd_apply_*.
#include "fno_groupnorm.hpp"

namespace fno {
namespace {

// Vectors of x and of grad_out a thread keeps: 16 values of each.  (Of 16-bit
// fields twice as many would fit, but a vector of eight has eight channels'
// constants beside it, which then spill: 36 us for one 32 x 1024 item.)
template <typename TX>
constexpr int kHeld = 16 / kVec<TX>;
constexpr int64_t kFusedValues = 1024 * 16;
constexpr int kFusedThreads = 1024;

template <int ACT>
__device__ __forceinline__ float slope_times(float dy, float xh, float w, float b) {
    return dy * act_slope<ACT>(fmaf(xh, w, b));
}

// A sum with the rounding of each addition carried along (Knuth's two-sum):
// a parameter's gradient is a sum of values of either sign over a whole batch,
// often thousands of times smaller than their magnitudes' sum.
struct Compensated {
    float s, c;
    __device__ __forceinline__ void add(float v) {
        const float t = s + v, z = t - s;
        c += (s - (t - z)) + (v - z);
        s = t;
    }
    __device__ __forceinline__ float total() const { return s + c; }
};

// s1, s2 (not yet divided by n) of `groups` groups of D channels from the
// channels' sums; res[g] and res[groups + g].
__device__ __forceinline__ void group_means(const float* cg, const float* cx, const float* w, int64_t c0, int D,
                                            int groups, float* res) {
    const int t = threadIdx.x;
    int parts = 1;
    while (parts < 64 && 2 * parts * groups <= (int)blockDim.x && parts < D) parts *= 2;
    for (int g = t / parts; g < groups; g += (int)blockDim.x / parts) {
        float s1 = 0.0f, s2 = 0.0f;
        for (int d = t & (parts - 1); d < D; d += parts) {
            const float wc = or_one(w, c0 + g * D + d);
            s1 = fmaf(wc, cg[g * D + d], s1);
            s2 = fmaf(wc, cx[g * D + d], s2);
        }
        s1 = team_sum(s1, parts);
        s2 = team_sum(s2, parts);
        if ((t & (parts - 1)) == 0) {
            res[g] = s1;
            res[groups + g] = s2;
        }
    }
    __syncthreads();
}

// ---- one pass, channels last: workgroup (item, slice of cs channels) ------------
// x and grad_out in registers, read once.  256 items of 32 channels x 1024,
// float32: 39 us for 101 MB (2.6 TB/s), with the sums of every channel through
// LDS besides.
template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kFusedThreads) void k_gn_bwd_fused_last(
    const TX* __restrict__ x, const TY* __restrict__ dy, const float* __restrict__ w, const float* __restrict__ bias,
    const float* __restrict__ stats, TX* __restrict__ gx, float2* __restrict__ part, LastRows r, int slices,
    int64_t blocks) {
    constexpr int V = kVec<TX>, kHold = kHeld<TX>;
    extern __shared__ float lds[];
    const int64_t id = block_id();
    if (id >= blocks) return;
    float* buf = lds;
    float* cg = lds + r.threads * V;
    float* cx = cg + r.cs;
    float* res = cx + r.cs;
    const int groups = div_by(r.cs, r.by_D);
    const int64_t b = id / slices;
    const int c0 = (int)(id % slices) * r.cs;
    const int t = threadIdx.x, row = div_by(t, r.by_cv), slot = t - row * r.cv;
    const bool on = row < r.q;
    const int64_t base = b * r.P * r.C + c0 + slot * V;
    const float* st = stats + 2 * (b * (div_by(r.C, r.by_D)) + div_by(c0, r.by_D));

    Raw<TX, V> hx[kHold];
    Raw<TY, V> hy[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int s = row + i * r.q, n = on ? last_valid<V>(r, s, slot) : 0;
        const int64_t e = base + (int64_t)s * r.stride();
        hx[i].load(x + e, n);
        hy[i].load(dy + e, n);
    }
    float m[V], k[V], a[V], o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = mod_by(slot * V + j, r.by_cs);
        m[j] = st[2 * (div_by(c, r.by_D))];
        k[j] = st[2 * (div_by(c, r.by_D)) + 1];
        a[j] = or_one(w, c0 + c);
        o[j] = or_zero(bias, c0 + c);
    }
    // an element that does not exist reads grad_out 0 and adds nothing; its x is set to the mean, so
    // that xh is 0 however large the mean
    float sg[V] = {}, sx[V] = {};
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int n = on ? last_valid<V>(r, row + i * r.q, slot) : 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xh = j < n ? (hx[i][j] - m[j]) * k[j] : 0.0f;
            const float g = j < n ? slope_times<ACT>(hy[i][j], xh, a[j], o[j]) : 0.0f;
            sg[j] += g;
            sx[j] = fmaf(g, xh, sx[j]);
        }
    }
    last_sums(sg, buf, cg, r, 1);
    last_sums(sx, buf, cx, r, 1);
    if (part)
        for (int c = t; c < r.cs; c += blockDim.x) part[b * r.C + c0 + c] = make_float2(cg[c], cx[c]);
    if (!gx) return;
    group_means(cg, cx, w, c0, r.D, groups, res);
    if (!on) return;
    const float inv_n = 1.0f / ((float)r.P * (float)r.D);
    float s1[V], s2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int g = div_by(mod_by(slot * V + j, r.by_cs), r.by_D);
        s1[j] = res[g] * inv_n;
        s2[j] = res[groups + g] * inv_n;
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int s = row + i * r.q, n = last_valid<V>(r, s, slot);
        if (n == 0) break;
        float u[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xh = (hx[i][j] - m[j]) * k[j];
            const float g = slope_times<ACT>(hy[i][j], xh, a[j], o[j]);
            u[j] = k[j] * (fmaf(g, a[j], -s1[j]) - xh * s2[j]);
        }
        store_part(gx + base + (int64_t)s * r.stride(), n, u);
    }
}

// ---- one pass, channels first: workgroup (item, group) ----------------------------
// Every vector leaves its sums of g and g xh in LDS, for its first channel
// and, where the row length is no multiple of V, for the next one (a row is
// at least a vector long); the vectors of each channel are then added in order.
// 4096 groups of 16384 values, float32: 149 to 151 us for 805 MB (5.3 to 5.4 TB/s): memory.
template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kFusedThreads) void k_gn_bwd_fused_first(
    const TX* __restrict__ x, const TY* __restrict__ dy, const float* __restrict__ w, const float* __restrict__ bias,
    const float* __restrict__ stats, TX* __restrict__ gx, float2* __restrict__ part, int D, int P, int groups,
    FastDiv by_p, int64_t blocks) {
    constexpr int V = kVec<TX>, kHold = kHeld<TX>;
    extern __shared__ float lds[];
    const int64_t id = block_id();
    if (id >= blocks) return;
    const int n = D * P, t = threadIdx.x, step = blockDim.x * V, nv = (n + V - 1) / V;
    const bool whole = P % V == 0;
    float2* head = reinterpret_cast<float2*>(lds);
    float2* next = head + nv;
    float* cg = reinterpret_cast<float*>(whole ? next : next + nv);
    float* cx = cg + D;
    float* res = cx + D;
    const int c0 = (int)(id % groups) * D;
    const int64_t base = id * n;
    const float mean = stats[2 * id], rstd = stats[2 * id + 1];

    Raw<TX, V> hx[kHold];
    Raw<TY, V> hy[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int e = i * step + t * V, m = max(0, min(V, n - e));
        hx[i].load(x + base + e, m);
        hy[i].load(dy + base + e, m);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int e = i * step + t * V;
        if (e >= n) break;
        const int d = div_by(e, by_p), cut = (d + 1) * P - e;      // places of the vector in channel d
        float2 s = make_float2(0.0f, 0.0f), u = make_float2(0.0f, 0.0f);
        const int c1 = min(d + 1, D - 1);
        const float w0 = or_one(w, c0 + d), b0 = or_zero(bias, c0 + d);
        const float w1 = or_one(w, c0 + c1), b1 = or_zero(bias, c0 + c1);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (j >= n - e) break;
            const float xh = (hx[i][j] - mean) * rstd;
            const float g = slope_times<ACT>(hy[i][j], xh, j < cut ? w0 : w1, j < cut ? b0 : b1);
            if (j < cut) {
                s.x += g;
                s.y = fmaf(g, xh, s.y);
            } else {
                u.x += g;
                u.y = fmaf(g, xh, u.y);
            }
        }
        head[e / V] = s;
        if (!whole) next[e / V] = u;
    }
    __syncthreads();
    int parts = 1;
    while (parts < 64 && 2 * parts * D <= (int)blockDim.x) parts *= 2;
    for (int d = t / parts; d < D; d += (int)blockDim.x / parts) {
        const int lo = d * P / V, hi = ((d + 1) * P + V - 1) / V;
        float2 s = make_float2(0.0f, 0.0f);
        for (int v = lo + (t & (parts - 1)); v < hi; v += parts) {
            const float2 q = v * V < d * P ? next[v] : head[v];
            s.x += q.x;
            s.y += q.y;
        }
        s.x = team_sum(s.x, parts);
        s.y = team_sum(s.y, parts);
        if ((t & (parts - 1)) == 0) {
            cg[d] = s.x;
            cx[d] = s.y;
            if (part) part[id * D + d] = s;
        }
    }
    if (!gx) return;
    __syncthreads();
    group_means(cg, cx, w, c0, D, 1, res);
    const float inv_n = 1.0f / (float)n, s1 = res[0] * inv_n, s2 = res[1] * inv_n;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int e = i * step + t * V;
        if (e >= n) break;
        const int d = div_by(e, by_p), cut = (d + 1) * P - e;
        const int c1 = min(d + 1, D - 1);
        const float w0 = or_one(w, c0 + d), b0 = or_zero(bias, c0 + d);
        const float w1 = or_one(w, c0 + c1), b1 = or_zero(bias, c0 + c1);
        float u[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xh = (hx[i][j] - mean) * rstd, wc = j < cut ? w0 : w1;
            const float g = slope_times<ACT>(hy[i][j], xh, wc, j < cut ? b0 : b1);
            u[j] = rstd * (fmaf(g, wc, -s1) - xh * s2);
        }
        store_part(gx + base + e, min(V, n - e), u);
    }
}

// ---- one pass, items spread over workgroups --------------------------------------------
// Workgroup (item, chunk of q NV super-rows), as k_gn_once_last: x and
// grad_out stay in registers while the chunks' (s1, s2) are exchanged.  Each
// chunk's channel sums go to part[(item chunks + chunk) C + c].
//
// Vectors a thread holds of each field, at most: 16, and half as many where a
// 16-bit x meets a float32 grad_out, whose vectors of eight are 32 bytes (16 of
// each spill 24 to 28 registers).
template <typename TX, typename TY>
constexpr int kOnceVectors = kVec<TX> == kVec<TY> ? 16 : 8;
template <typename TX, typename TY>
struct OnceArgs {
    const TX* x;
    const TY* dy;
    const float *w, *bias, *stats;
    TX* gx;
    float2* part;
    uint64_t* slots;
    LastRows r;
    Once o;
    int spin;
};

template <int ACT, int NV, typename TX, typename TY>
struct OnceLast {
    static constexpr int V = kVec<TX>;
    // float32 keeps g = grad_out act'(z) in the place of grad_out: the slope is not formed twice
    static constexpr bool kKeep = std::is_same_v<TY, float>;
    typedef typename VecOf<TX, V>::type VecX;
    typedef typename VecOf<TY, V>::type VecY;
    const OnceArgs<TX, TY>& a;
    const LastRows& r;
    float *buf, *w, *s1, *s2;
    int* missing;
    int t, row, slot, groups, chunk;
    int64_t item, step;
    float m[V], k[V], b[V], wc[V];

    __device__ __forceinline__ OnceLast(const OnceArgs<TX, TY>& args, float* lds, int* flag)
        : a(args), r(args.r), buf(lds), missing(flag) {
        t = threadIdx.x;
        row = div_by(t, r.by_cv);
        slot = t - row * r.cv;
        groups = div_by(r.C, r.by_D);
        w = lds + 2 * r.threads * V;
        s1 = w + r.C;
        s2 = s1 + groups;
        item = blockIdx.x / a.o.chunks;
        chunk = (int)(blockIdx.x - item * a.o.chunks);
        step = (int64_t)r.q * r.stride();
    }
    // The constants of the thread's channels.  Asked for before the field: loads come back in order, and the first
    // vectors are worked on while the last are on their way.
    __device__ __forceinline__ void constants() {
        const float* st = a.stats + 2 * item * groups;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = channel(j), g = div_by(c, r.by_D);
            m[j] = st[2 * g];
            k[j] = st[2 * g + 1];
            b[j] = or_zero(a.bias, c);
            wc[j] = or_one(a.w, c);
        }
    }
    __device__ __forceinline__ int channel(int j) const { return mod_by(slot * V + j, r.by_cs); }
    __device__ __forceinline__ int per() const { return r.q * NV; }
    __device__ __forceinline__ int64_t base() const { return item * r.P * r.C; }
    __device__ __forceinline__ uint64_t* pairs() const { return a.slots + item * groups * a.o.chunks; }
    __device__ __forceinline__ int rows_of(int c) const {
        return row < r.q ? max(0, min(NV, (r.ns - (c * per() + row) + r.q - 1) / r.q)) : 0;
    }
    __device__ __forceinline__ int64_t at_of(int c) const { return (int64_t)(c * per() + row) * r.stride() + slot * V; }

    // The sums of chunk c, from the pairs of vectors that `each` hands over (g is left in the second where it fits).
    template <typename F>
    __device__ __forceinline__ void put(int c, bool own, F&& each) const {
        float sg[V], sx[V];
#pragma unroll
        for (int j = 0; j < V; ++j) sg[j] = sx[j] = 0.0f;
        each([&](const VecX& x, VecY& y) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = ((float)x[j] - m[j]) * k[j];
                const float g = slope_times<ACT>((float)y[j], xh, wc[j], b[j]);
                sg[j] += g;
                sx[j] = fmaf(g, xh, sx[j]);
                if constexpr (kKeep) y[j] = g;
            }
        });
        float* gs = buf;
        float* xs = buf + r.threads * V;
        __syncthreads();
        if (row == 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) w[channel(j)] = wc[j];
        }
        if (row < r.q) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                gs[t * V + j] = sg[j];
                xs[t * V + j] = sx[j];
            }
        }
        __syncthreads();
        const int rows = r.q * r.R;
        {
            const int parts = a.o.parts, part = t & (parts - 1), g = t >> __builtin_ctz(parts);
            if (g < groups) {
                float s = 0.0f, z = 0.0f;
                for (int e = part; e < rows * r.D; e += parts) {
                    const int i = div_by(e, r.by_D), ch = g * r.D + e - i * r.D;
                    s = fmaf(w[ch], gs[i * r.C + ch], s);
                    z = fmaf(w[ch], xs[i * r.C + ch], z);
                }
                s = team_sum(s, parts);
                z = team_sum(z, parts);
                if (part == 0) put_pair(pairs() + g * a.o.chunks + c, s, z);
            }
        }
        if (own && a.part) {
            int parts = 1;
            while (parts < 64 && 2 * parts * r.C <= (int)blockDim.x) parts *= 2;
            const int part = t & (parts - 1), step_c = (int)blockDim.x >> __builtin_ctz(parts);
            for (int ch = t >> __builtin_ctz(parts); ch < r.C; ch += step_c) {
                float s = 0.0f, z = 0.0f;
                for (int i = part; i < rows; i += parts) {
                    s += gs[i * r.C + ch];
                    z += xs[i * r.C + ch];
                }
                s = team_sum(s, parts);
                z = team_sum(z, parts);
                if (part == 0) a.part[(item * a.o.chunks + c) * r.C + ch] = make_float2(s, z);
            }
        }
    }
    // s1 and s2 of the item's groups, in LDS; the first chunk not there, or `chunks`
    __device__ __forceinline__ int join(int looks) const {
        const int chunks = a.o.chunks, parts = a.o.parts;
        const int part = t & (parts - 1), g = t >> __builtin_ctz(parts);
        __syncthreads();
        if (t == 0) *missing = chunks;
        __syncthreads();
        if (g < groups) {
            uint64_t v[kLooks];
            const int lost = gather_pairs(pairs() + g * chunks, chunks, part, parts, looks, v);
            if (lost < chunks) atomicMin(missing, lost);
            float s = 0.0f, z = 0.0f;
#pragma unroll
            for (int i = 0; i < kLooks; ++i) {
                if (i * parts >= chunks) break;
                if (part + i * parts < chunks) {
                    const float2 q = unpack_pair(v[i]);
                    s += q.x;
                    z += q.y;
                }
            }
            s = team_sum(s, parts);
            z = team_sum(z, parts);
            if (part == 0) {
                const float inv = 1.0f / ((float)r.P * (float)r.D);
                s1[g] = s * inv;
                s2[g] = z * inv;
            }
        }
        __syncthreads();
        return *missing;
    }
    // grad_x of this workgroup's chunk; `kept`: the second vector holds g
    template <bool KEPT, typename F>
    __device__ __forceinline__ void write(int64_t at, F&& each) const {
        float p[V], q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int g = div_by(channel(j), r.by_D);
            p[j] = s1[g];
            q[j] = s2[g];
        }
        TX* out = a.gx + base() + at;
        each([&](int i, const VecX& x, const VecY& y) {
            float u[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = ((float)x[j] - m[j]) * k[j];
                const float g = KEPT ? (float)y[j] : slope_times<ACT>((float)y[j], xh, wc[j], b[j]);
                u[j] = k[j] * (fmaf(g, wc[j], -p[j]) - xh * q[j]);
            }
            store_vec<V>(out + i * step, u);
        });
    }
};

template <int ACT, int NV, typename TX, typename TY>
__device__ __attribute__((noinline)) void once_late(OnceArgs<TX, TY> args, float* lds, int* flag, int lost) {
    typedef OnceLast<ACT, NV, TX, TY> F;
    F f(args, lds, flag);
    f.constants();
    const auto pair_at = [&](int64_t at, int i, auto&& use) {
        const int64_t e = f.base() + at + i * f.step;
        const typename F::VecX x = *reinterpret_cast<const typename F::VecX*>(args.x + e);
        typename F::VecY y = *reinterpret_cast<const typename F::VecY*>(args.dy + e);
        use(x, y);
    };
    do {
        const int n = f.rows_of(lost);
        const int64_t at = f.at_of(lost);
        f.put(lost, false, [&](auto&& take) {
#pragma unroll 1
            for (int i = 0; i < n; ++i) pair_at(at, i, take);
        });
        lost = f.join(0);
    } while (lost < args.o.chunks);
    const int64_t at = f.at_of(f.chunk);
    f.template write<false>(at, [&](auto&& to) {
#pragma unroll 1
        for (int i = 0; i < f.rows_of(f.chunk); ++i)
            pair_at(at, i, [&](const auto& x, const auto& y) { to(i, x, y); });
    });
}

// Two waves a SIMD, with 16 vectors of each field in 256 registers: 95 us for
// the 128 x 128 field (32 x 64 channels, float32) where four waves of 8
// vectors took 111 and of 4 vectors 165 (what a workgroup costs whatever it
// holds shows; not waiting for the others changed none of them).  The kernel
// alone now takes 86 us (403 MB, 4.7 TB/s); with 8 vectors of a bfloat16 field and
// a float32 grad_out 64 us (268 MB, 4.2 TB/s).
template <int ACT, int NV, typename TX, typename TY>
__global__ __launch_bounds__(kOnceThreads, 2) void k_gn_bwd_once_last(OnceArgs<TX, TY> args) {
    typedef OnceLast<ACT, NV, TX, TY> F;
    extern __shared__ float lds[];
    __shared__ int missing;
    F f(args, lds, &missing);
    f.constants();
    typename F::VecX x[NV];
    typename F::VecY y[NV];
    const int rows = f.rows_of(f.chunk);
    const int64_t at = rows ? f.at_of(f.chunk) : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t e = f.base() + at + max(0, min(i, rows - 1)) * f.step;
        x[i] = *reinterpret_cast<const typename F::VecX*>(args.x + e);
        y[i] = *reinterpret_cast<const typename F::VecY*>(args.dy + e);
    }
    f.put(f.chunk, true, [&](auto&& take) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < rows) take(x[i], y[i]);
    });
    if (!args.gx) return;
    const int lost = f.join(args.spin);
    if (lost < args.o.chunks) {
        once_late<ACT, NV, TX, TY>(args, lds, &missing, lost);
        return;
    }
    f.template write<F::kKeep>(at, [&](auto&& to) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < rows) to(i, x[i], y[i]);
    });
}

// ---- partial sums of chunks ----------------------------------------------------------
// Bound by memory: 1.07 GB in 182 us (5.9 TB/s).
// Channels last: workgroup (item, chunk); part[(b chunks + chunk) C + c].
template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kMaxSlots) void k_gn_bwd_sums_last(const TX* __restrict__ x, const TY* __restrict__ dy,
                                                                const float* __restrict__ w,
                                                                const float* __restrict__ bias,
                                                                const float* __restrict__ stats,
                                                                float2* __restrict__ part, LastRows r, int per,
                                                                int chunks, int64_t blocks) {
    constexpr int V = kVec<TX>;
    extern __shared__ float lds[];
    const int64_t id = block_id();
    if (id >= blocks) return;
    float* buf = lds;
    float* cg = lds + r.threads * V;
    float* cx = cg + r.C;
    const int64_t b = id / chunks;
    const int first = (int)(id % chunks) * per, last = min(first + per, r.ns);
    const int t = threadIdx.x, row = div_by(t, r.by_cv), slot = t - row * r.cv;
    const int64_t base = b * r.P * r.C + slot * V;
    const float* st = stats + 2 * b * (div_by(r.C, r.by_D));
    float m[V], k[V], a[V], o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = mod_by(slot * V + j, r.by_cs);
        m[j] = st[2 * (div_by(c, r.by_D))];
        k[j] = st[2 * (div_by(c, r.by_D)) + 1];
        a[j] = or_one(w, c);
        o[j] = or_zero(bias, c);
    }
    // sums of 16 rows at a time, then of those: shorter chains of additions
    float sg[V] = {}, sx[V] = {}, tg[V] = {}, tx[V] = {};
    auto fold = [&] {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            tg[j] += sg[j];
            tx[j] += sx[j];
            sg[j] = sx[j] = 0.0f;
        }
    };
    auto take = [&](const float (&u)[V], const float (&v)[V], int n) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xh = (u[j] - m[j]) * k[j];
            const float g = slope_times<ACT>(v[j], xh, a[j], o[j]);
            if (j < n) {
                sg[j] += g;
                sx[j] = fmaf(g, xh, sx[j]);
            }
        }
    };
    if (row < r.q) {
        int s = first + row;
        const int full = min(last, r.P / r.R);
        int pairs = 0;
        for (; s + r.q < full; s += 2 * r.q) {
            float u[2][V], v[2][V];
            if ((++pairs & 7) == 0) fold();
            const int64_t e = base + (int64_t)s * r.stride(), f = e + (int64_t)r.q * r.stride();
            load_vec<V>(x + e, u[0]);
            load_vec<V>(dy + e, v[0]);
            load_vec<V>(x + f, u[1]);
            load_vec<V>(dy + f, v[1]);
            take(u[0], v[0], V);
            take(u[1], v[1], V);
        }
        for (; s < last; s += r.q) {
            float u[V], v[V];
            const int n = last_valid<V>(r, s, slot);
            const int64_t e = base + (int64_t)s * r.stride();
            load_part<V>(x + e, n, u);
            load_part<V>(dy + e, n, v);
            take(u, v, n);
        }
    }
    fold();
    last_sums(tg, buf, cg, r, 1);
    last_sums(tx, buf, cx, r, 1);
    for (int c = t; c < r.C; c += blockDim.x) part[id * r.C + c] = make_float2(cg[c], cx[c]);
}

// Channels first: a team takes a row or a piece of it; part[row chunks + piece].
// 1.07 GB in 182 to 186 us (5.8 to 5.9 TB/s): memory.
template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kGnThreads) void k_gn_bwd_sums_first(const TX* __restrict__ x, const TY* __restrict__ dy,
                                                                  const float* __restrict__ w,
                                                                  const float* __restrict__ bias,
                                                                  const float* __restrict__ stats,
                                                                  float2* __restrict__ part, FirstRows r, int C, int D,
                                                                  int64_t blocks) {
    constexpr int V = kVec<TX>;
    __shared__ float red[16];
    const int64_t id = block_id();
    if (id >= blocks) return;
    const int64_t row = id / r.chunks * (kGnThreads / r.team) + threadIdx.x / r.team;
    const int piece = (int)(id % r.chunks);
    Compensated cg{}, cx{};
    if (row < r.rows) {
        const int at = piece * r.piece, end = min(at + r.piece, r.P);
        const int c = (int)(row % C);
        const float* st = stats + 2 * (row / D);
        const float m = st[0], k = st[1], a = or_one(w, c), o = or_zero(bias, c);
        const int64_t base = row * r.P;
        for (int p = at + (threadIdx.x & (r.team - 1)) * V; p < end; p += r.team * V) {
            float u[V], v[V];
            const int n = min(V, end - p);
            load_part<V>(x + base + p, n, u);
            load_part<V>(dy + base + p, n, v);
            float sg = 0.0f, sx = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = (u[j] - m) * k;
                const float g = slope_times<ACT>(v[j], xh, a, o);
                if (j < n) {
                    sg += g;
                    sx = fmaf(g, xh, sx);
                }
            }
            cg.add(sg);
            cx.add(sx);
        }
    }
    float sg = cg.total(), sx = cx.total();
    if (r.team == kGnThreads) {
        sg = block_sum(sg, red);
        sx = block_sum(sx, red);
    } else {
        sg = team_sum(sg, r.team);
        sx = team_sum(sx, r.team);
    }
    if ((threadIdx.x & (r.team - 1)) == 0 && row < r.rows) part[row * r.chunks + piece] = make_float2(sg, sx);
}

// x and grad_out of different layouts: workgroup (item, chunk of `per`
// position tiles, channel tile); the channels-last one of the two is turned
// in LDS.  part as that of x's layout.  268 MB in 57 to 60 us (4.4 to 4.7 TB/s) for 32 x 64
// x 128 x 128: memory, and the tiles' barriers.
template <int ACT, bool XLAST, typename TX, typename TY>
__global__ __launch_bounds__(kGnThreads) void k_gn_bwd_sums_cross(const TX* __restrict__ x, const TY* __restrict__ dy,
                                                                  const float* __restrict__ w,
                                                                  const float* __restrict__ bias,
                                                                  const float* __restrict__ stats,
                                                                  float2* __restrict__ part, Tiles q, int C, int P,
                                                                  int D, int per, int chunks, int64_t blocks) {
    constexpr int V = kVec<TX>, N = kTile / V / kGnThreads;
    __shared__ float tile[kTileLds];
    __shared__ float2 waves[N * kGnThreads / 64];
    const int64_t id = block_id();
    if (id >= blocks) return;
    const int64_t b = id / q.tiles_c / chunks;
    const int chunk = (int)(id / q.tiles_c % chunks), ct = (int)(id % q.tiles_c);
    const int first = chunk * per, last = min(first + per, q.tiles_p);
    const float* st = stats + 2 * b * (C / D);
    Compensated cg[N] = {}, cx[N] = {};
    Spot s{};
    for (int pt = first; pt < last; ++pt) {
        s = spot_of(q, (int64_t)pt * q.tiles_c + ct, b, C, P);
        __syncthreads();
        if constexpr (XLAST) load_last(x, tile, q, s, C);
        else load_last(dy, tile, q, s, C);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const Along<V> a(q, s, i);
            if (a.n) {
                const int c = s.c0 + a.c;
                const float m = st[2 * (c / D)], k = st[2 * (c / D) + 1], wc = or_one(w, c), bc = or_zero(bias, c);
                const int64_t e = s.item + (int64_t)c * P + s.p0 + a.p;
                const float* row = tile + a.c * (q.tp() + 1) + a.p;
                float u[V];
                if constexpr (XLAST) load_part<V>(dy + e, a.n, u);
                else load_part<V>(x + e, a.n, u);
                float sg = 0.0f, sx = 0.0f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = ((XLAST ? row[j] : u[j]) - m) * k;
                    const float g = slope_times<ACT>(XLAST ? u[j] : row[j], xh, wc, bc);
                    if (j < a.n) {
                        sg += g;
                        sx = fmaf(g, xh, sx);
                    }
                }
                cg[i].add(sg);
                cx[i].add(sx);
            }
        }
    }
    // lanes of a row (a whole wave, or a part of one), then the waves of a row
    const int lv = 12 - q.log2c - (V == 4 ? 2 : 3), lanes = min(64, 1 << lv), t = threadIdx.x;
    const auto put = [&](int c, float2 v) {
        const int64_t ch = s.c0 + c;
        part[XLAST ? (b * chunks + chunk) * C + ch : (b * C + ch) * chunks + chunk] = v;
    };
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 v = make_float2(team_sum(cg[i].total(), lanes), team_sum(cx[i].total(), lanes));
        const int c = (i * kGnThreads + t) >> lv;
        if (lv < 6) {
            if ((t & (lanes - 1)) == 0 && c < s.nc) put(c, v);
        } else if ((t & 63) == 0) {
            waves[(i * kGnThreads + t) >> 6] = v;
        }
    }
    if (lv < 6) return;
    __syncthreads();
    if (t < s.nc) {
        const int per_row = 1 << (lv - 6);
        float2 v = make_float2(0.0f, 0.0f);
        for (int k = 0; k < per_row; ++k) {
            v.x += waves[t * per_row + k].x;
            v.y += waves[t * per_row + k].y;
        }
        put(t, v);
    }
}

// Channels last, any width: workgroup (item, chunk of positions, kWideC
// channels), threads along the channels; part[(b chunks + chunk) C + c].
// 268 MB in 65 us (4 x 8192 channels x 1024, float32): scalar loads.
constexpr int kWideC = 4 * kGnThreads;
template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kGnThreads) void k_gn_bwd_sums_wide(const TX* __restrict__ x, const TY* __restrict__ dy,
                                                                 const float* __restrict__ w,
                                                                 const float* __restrict__ bias,
                                                                 const float* __restrict__ stats,
                                                                 float2* __restrict__ part, int C, int P, int D,
                                                                 int per, int chunks, int64_t blocks) {
    if (block_id() >= blocks) return;
    const int pieces = (C + kWideC - 1) / kWideC, c0 = (int)(block_id() % pieces) * kWideC;
    const int64_t id = block_id() / pieces, b = id / chunks;
    const int first = (int)(id % chunks) * per, last = min(first + per, P);
    for (int c = c0 + threadIdx.x; c < min(C, c0 + kWideC); c += kGnThreads) {
        const float* st = stats + 2 * (b * (C / D) + c / D);
        const float m = st[0], k = st[1], a = or_one(w, c), o = or_zero(bias, c);
        Compensated sg{}, sx{};
        for (int p = first; p < last; ++p) {
            const int64_t e = (b * P + p) * C + c;
            const float xh = ((float)x[e] - m) * k;
            const float g = slope_times<ACT>((float)dy[e], xh, a, o);
            sg.add(g);
            sx.add(g * xh);
        }
        part[id * C + c] = make_float2(sg.total(), sx.total());
    }
}

// ---- joining the partial sums -----------------------------------------------------------
// Partial sums of a backward pass: pair (b, chunk, c) is part[(b chunks +
// chunk) C + c] (`last`) or part[(b C + c) chunks + chunk].  They come from
// other XCDs' kernels and are far away (a microsecond), so a lane asks for
// eight at a time, and adds them in double.
struct Parts {
    const float2* part;
    int64_t B;
    int C, D, chunks;
    bool last;
    float inv_n;
    float *gw, *gb;
};

template <typename F>
__device__ __forceinline__ void sum_parts(int64_t n, int first, int step, F&& at, double& s, double& z) {
    for (int64_t k = first; k < n; k += 8 * step) {
        float2 q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = k + i * step < n ? at(k + i * step) : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s += q[i].x;
            z += q[i].y;
        }
    }
}

// s1 and s2 of group `g` (numbered over the items), added by `parts` threads:
// what those of one wave have, if it is more than a wave.
__device__ __forceinline__ float2 group_sums(const Parts& f, const float* __restrict__ w, int64_t g, int part,
                                             int parts) {
    const int groups = f.C / f.D;
    const int64_t b = g / groups;
    const int c0 = (int)(g % groups) * f.D;
    double s = 0.0, z = 0.0;
    sum_parts((int64_t)f.D * f.chunks, part, parts, [&](int64_t k) {
        const uint32_t e = (uint32_t)k, by = (uint32_t)(f.last ? f.D : f.chunks);
        const int hi = (int)(e / by), lo = (int)(e - hi * by), d = f.last ? lo : hi, ch = f.last ? hi : lo;
        const float2 q = f.part[f.last ? (b * f.chunks + ch) * f.C + c0 + d : (b * f.C + c0 + d) * f.chunks + ch];
        const float wc = or_one(w, c0 + d);
        return make_float2(wc * q.x, wc * q.y);
    }, s, z);
    parts = min(parts, 64);
    return make_float2(team_sum((float)s, parts) * f.inv_n, team_sum((float)z, parts) * f.inv_n);
}

// The parameters' gradients, over items and chunks, a workgroup for eight
// channels (`last`: their pairs share a 64-byte piece of each chunk's row) or
// for one.  `both` holds a float2 a thread.
__device__ __forceinline__ void param_sums(const Parts& f, int64_t block, float2* both) {
    const int t = threadIdx.x, threads = blockDim.x, per = f.last ? 8 : 1;
    const int64_t c = block * per + t % per;
    double s = 0.0, z = 0.0;
    if (c < f.C) {
        if (f.last) {
            sum_parts(f.B * f.chunks, t / 8, threads / 8, [&](int64_t k) { return f.part[k * f.C + c]; }, s, z);
        } else {
            sum_parts(f.B * f.chunks, t, threads,
                      [&](int64_t k) { return f.part[(k / f.chunks * f.C + c) * f.chunks + k % f.chunks]; }, s, z);
        }
    }
    both[t] = make_float2((float)s, (float)z);
    // halves added until a row of `per` is left (a row without a partner stays)
    for (int rows = threads / per; rows > 1;) {
        const int keep = (rows + 1) / 2;
        __syncthreads();
        if (t < (rows - keep) * per) {
            both[t].x += both[t + keep * per].x;
            both[t].y += both[t + keep * per].y;
        }
        rows = keep;
    }
    if (t < per && c < f.C) {
        if (f.gb) f.gb[c] = both[t].x;
        if (f.gw) f.gw[c] = both[t].y;
    }
}
inline int64_t param_blocks(const Parts& f) {
    return !f.gw && !f.gb ? 0 : f.last ? (f.C + 7) / 8 : f.C;
}

// First (with gsum) the B G groups' (s1, s2); then the parameters.  A group has
// a wave, or a workgroup (`waves` > 1) where its pairs are more than a wave asks
// for in one go: 31 us with a wave for 8 groups of 4096 pairs, 6.3 with a
// workgroup.  Latency of memory far away bounds both.
// Large workgroups: all a parameter's pairs are then asked for in one or two
// goes (2048 chunks of 64 channels: 8.1 us with 256 threads, 5.1 with 1024).
constexpr int kFinishThreads = 1024;
__global__ __launch_bounds__(kFinishThreads) void k_gn_bwd_finish(Parts f, const float* __restrict__ w,
                                                                  float2* __restrict__ gsum, int64_t ngroups,
                                                                  int waves) {
    constexpr int kWaves = kFinishThreads / 64;
    __shared__ float2 both[kFinishThreads];
    const int64_t id = block_id(), gblocks = waves == 1 ? (ngroups + kWaves - 1) / kWaves : ngroups;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (id >= gblocks) {
        if ((id - gblocks) * (f.last ? 8 : 1) < f.C) param_sums(f, id - gblocks, both);
    } else if (waves == 1) {
        const int64_t i = id * kWaves + wave;
        if (i >= ngroups) return;
        const float2 s = group_sums(f, w, i, lane, 64);
        if (lane == 0) gsum[i] = s;
    } else {
        const float2 s = group_sums(f, w, id, threadIdx.x, kFinishThreads);
        if (lane == 0) both[wave] = s;
        __syncthreads();
        if (threadIdx.x < 64) {
            const float2 v = lane < kWaves ? both[lane] : make_float2(0.0f, 0.0f);
            const float2 all = make_float2(team_sum(v.x, 64), team_sum(v.y, 64));
            if (lane == 0) gsum[id] = all;
        }
    }
}
inline int finish_waves(const Parts& f) { return (int64_t)f.D * f.chunks <= 8 * 64 ? 1 : kFinishThreads / 64; }

// With few chunks there is no k_gn_bwd_finish: the workgroups of grad_x add
// their own groups' sums (Parts::part not null), and further workgroups behind
// them the parameters' gradients.
__device__ __forceinline__ void join_groups(const Parts& f, const float* __restrict__ w, int64_t g0, int ng,
                                            float2* res) {
    const int t = threadIdx.x, threads = blockDim.x;
    int parts = 1;
    while (parts < 64 && 2 * parts * ng <= threads) parts *= 2;
    for (int i = t / parts; i < ng; i += threads / parts) {
        const float2 s = group_sums(f, w, g0 + i, t & (parts - 1), parts);
        if ((t & (parts - 1)) == 0) res[i] = s;
    }
    __syncthreads();
}

// ---- grad_x --------------------------------------------------------------------------------
// Two fields read, one written, bound by memory: 1.6 GB in 290 us (5.6 TB/s)
// in either layout; between the layouts 403 MB in 62 to 70 us (5.8 to 6.5 TB/s,
// partly from the caches) with tiles turned in LDS.
template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kMaxSlots) void k_gn_bwd_apply_last(const TX* __restrict__ x, const TY* __restrict__ dy,
                                                                 const float* __restrict__ w,
                                                                 const float* __restrict__ bias,
                                                                 const float* __restrict__ stats,
                                                                 const float2* __restrict__ gsum, TX* __restrict__ gx,
                                                                 LastRows r, Parts f, int per, int chunks,
                                                                 int64_t blocks, int64_t extra) {
    constexpr int V = kVec<TX>;
    extern __shared__ float2 joined[];
    const int64_t id = block_id();
    if (id >= blocks + extra) return;
    if (id >= blocks) {
        param_sums(f, id - blocks, joined);
        return;
    }
    const int64_t b = id / chunks;
    const int first = (int)(id % chunks) * per, last = min(first + per, r.ns);
    const int t = threadIdx.x, row = div_by(t, r.by_cv), slot = t - row * r.cv;
    const int groups = div_by(r.C, r.by_D);
    const float2* gs = gsum + b * groups;
    if (f.part) {
        join_groups(f, w, b * groups, groups, joined);
        gs = joined;
    }
    if (row >= r.q) return;
    const int64_t base = b * r.P * r.C + slot * V;
    const float* st = stats + 2 * b * groups;
    float m[V], k[V], a[V], o[V], s1[V], s2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = mod_by(slot * V + j, r.by_cs), g = div_by(c, r.by_D);
        m[j] = st[2 * g];
        k[j] = st[2 * g + 1];
        a[j] = or_one(w, c);
        o[j] = or_zero(bias, c);
        s1[j] = gs[g].x;
        s2[j] = gs[g].y;
    }
    for (int s = first + row; s < last; s += r.q) {
        float u[V], v[V];
        const int n = last_valid<V>(r, s, slot);
        const int64_t e = base + (int64_t)s * r.stride();
        load_part<V>(x + e, n, u);
        load_part<V>(dy + e, n, v);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xh = (u[j] - m[j]) * k[j];
            const float g = slope_times<ACT>(v[j], xh, a[j], o[j]);
            u[j] = k[j] * (fmaf(g, a[j], -s1[j]) - xh * s2[j]);
        }
        store_part(gx + e, n, u);
    }
}

template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kGnThreads) void k_gn_bwd_apply_first(const TX* __restrict__ x, const TY* __restrict__ dy,
                                                                   const float* __restrict__ w,
                                                                   const float* __restrict__ bias,
                                                                   const float* __restrict__ stats,
                                                                   const float2* __restrict__ gsum,
                                                                   TX* __restrict__ gx, FirstRows r, Parts f, int C,
                                                                   int D, int64_t blocks, int64_t extra) {
    constexpr int V = kVec<TX>;
    __shared__ float2 joined[kGnThreads];
    const int64_t id = block_id();
    if (id >= blocks + extra) return;
    if (id >= blocks) {
        param_sums(f, id - blocks, joined);
        return;
    }
    const int teams = kGnThreads / r.team;
    const int64_t row0 = id / r.chunks * teams, row = row0 + threadIdx.x / r.team;
    int64_t g0 = 0;
    if (f.part) {
        g0 = row0 / D;
        join_groups(f, w, g0, (int)(min(row0 + teams - 1, r.rows - 1) / D - g0) + 1, joined);
        gsum = joined;
    }
    if (row >= r.rows) return;
    const int at = (int)(id % r.chunks) * r.piece, end = min(at + r.piece, r.P);
    const int c = (int)(row % C);
    const float* st = stats + 2 * (row / D);
    const float2 gs = gsum[row / D - g0];
    const float m = st[0], k = st[1], a = or_one(w, c), o = or_zero(bias, c);
    const int64_t base = row * r.P;
    for (int p = at + (threadIdx.x & (r.team - 1)) * V; p < end; p += r.team * V) {
        float u[V], v[V];
        const int n = min(V, end - p);
        load_part<V>(x + base + p, n, u);
        load_part<V>(dy + base + p, n, v);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xh = (u[j] - m) * k;
            const float g = slope_times<ACT>(v[j], xh, a, o);
            u[j] = k * (fmaf(g, a, -gs.x) - xh * gs.y);
        }
        store_part(gx + base + p, n, u);
    }
}

template <int ACT, bool XLAST, typename TX, typename TY>
__global__ __launch_bounds__(kGnThreads) void k_gn_bwd_apply_cross(const TX* __restrict__ x, const TY* __restrict__ dy,
                                                                   const float* __restrict__ w,
                                                                   const float* __restrict__ bias,
                                                                   const float* __restrict__ stats,
                                                                   const float2* __restrict__ gsum,
                                                                   TX* __restrict__ gx, Tiles q, Parts f, int C, int P,
                                                                   int D, int64_t blocks, int64_t extra) {
    constexpr int V = kVec<TX>;
    __shared__ float tile[kTileLds];
    __shared__ float2 joined[kGnThreads];
    const int64_t id = block_id();
    if (id >= blocks + extra) return;
    if (id >= blocks) {
        param_sums(f, id - blocks, joined);
        return;
    }
    const int64_t per_item = (int64_t)q.tiles_c * q.tiles_p, b = id / per_item;
    const Spot s = spot_of(q, id % per_item, b, C, P);
    const float* st = stats + 2 * b * (C / D);
    const float2* gs = gsum + b * (C / D);
    if (f.part) {
        const int g0 = s.c0 / D;
        join_groups(f, w, b * (C / D) + g0, (s.c0 + s.nc - 1) / D - g0 + 1, joined);
        gs = joined - g0;
    }
    if constexpr (XLAST) load_last(x, tile, q, s, C);
    else load_last(dy, tile, q, s, C);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTile / V / kGnThreads; ++i) {
        const Along<V> a(q, s, i);
        if (a.n) {
            const int c = s.c0 + a.c, g0 = c / D;
            const float m = st[2 * g0], k = st[2 * g0 + 1], wc = or_one(w, c), bc = or_zero(bias, c);
            const float2 sums = gs[g0];
            const int64_t e = s.item + (int64_t)c * P + s.p0 + a.p;
            float* row = tile + a.c * (q.tp() + 1) + a.p;
            float u[V];
            if constexpr (XLAST) load_part<V>(dy + e, a.n, u);
            else load_part<V>(x + e, a.n, u);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = ((XLAST ? row[j] : u[j]) - m) * k;
                const float g = slope_times<ACT>(XLAST ? u[j] : row[j], xh, wc, bc);
                const float v = k * (fmaf(g, wc, -sums.x) - xh * sums.y);
                if constexpr (XLAST) row[j] = v;
                else u[j] = v;
            }
            if constexpr (!XLAST) store_part(gx + e, a.n, u);
        }
    }
    if constexpr (XLAST) {
        __syncthreads();
        store_last(gx, tile, q, s, C);
    }
}

template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kGnThreads) void k_gn_bwd_apply_wide(const TX* __restrict__ x, const TY* __restrict__ dy,
                                                                  const float* __restrict__ w,
                                                                  const float* __restrict__ bias,
                                                                  const float* __restrict__ stats,
                                                                  const float2* __restrict__ gsum,
                                                                  TX* __restrict__ gx, int C, int P, int D,
                                                                  int64_t blocks) {
    const int64_t id = block_id();
    if (id >= blocks) return;
    const int64_t b = id / P;
    for (int c = threadIdx.x; c < C; c += kGnThreads) {
        const int64_t g = b * (C / D) + c / D, e = id * C + c;
        const float k = stats[2 * g + 1], a = or_one(w, c);
        const float xh = ((float)x[e] - stats[2 * g]) * k;
        const float v = slope_times<ACT>((float)dy[e], xh, a, or_zero(bias, c));
        gx[e] = (TX)(k * (fmaf(v, a, -gsum[g].x) - xh * gsum[g].y));
    }
}

// ---- schedules ------------------------------------------------------------------------------
enum How { kFusedLast, kFusedFirst, kOnceLast, kSplitLast, kSplitFirst, kCross, kWide };
struct Plan {
    How how;
    bool last;                    // layout of the partial sums
    LastRows rows;
    FirstRows frows;
    Tiles tiles;
    int slices, threads, per, chunks;
    size_t lds;
    Once once;
    bool join;                    // no k_gn_bwd_finish
};

Plan plan_kernels(const GroupNorm& g) {
    const int V = vec_of(g);
    const int64_t D = g.C / g.groups, n = D * g.P;
    const int held = 16 / V;
    const int64_t capacity = kFusedValues / V;                    // vectors
    Plan p{};
    p.chunks = 1;
    const bool same = g.x_last == g.out_last;
    p.last = g.x_last;
    if (!same) {
        p.how = kCross;
        p.tiles = tiles_of(g.C, g.P);
        split_chunks(g.B * p.tiles.tiles_c, p.tiles.tiles_p, 1, 32, &p.per, &p.chunks);
        return p;
    }
    if (!p.last) {
        const int64_t vectors = (n + V - 1) / V;
        p.lds = (size_t)vectors * sizeof(float2) * (g.P % V ? 2 : 1) + sizeof(float) * (size_t)(2 * D + 2);
        if (g.P >= V && vectors <= capacity && p.lds <= kLdsMax) {
            p.how = kFusedFirst;
            p.threads = 64;
            while (p.threads < kFusedThreads && p.threads * held < vectors) p.threads *= 2;
            return p;
        }
        p.how = kSplitFirst;
        p.frows = first_rows(g.B * g.C, g.P, V, 16);
        p.chunks = p.frows.chunks;
        return p;
    }
    if (!last_rows_ok(g.C, V)) {
        p.how = kWide;
        // the partial sums of an item are C times the chunks: 16 positions a chunk or more, so that they stay a
        // small part of what is read, and few chunks where the channels fill the chip
        const int64_t most = std::max<int64_t>(1, (int64_t(1) << 22) / g.C);
        split_chunks(g.B * ((g.C + kWideC - 1) / kWideC), g.P, std::max<int64_t>(16, (g.P + most - 1) / most),
                     std::max<int64_t>(256, g.P / most + 1), &p.per, &p.chunks);
        return p;
    }
    // the narrowest slice of whole groups that is a run of 64 bytes or more, or the whole rows
    int64_t cs = D;
    while (cs < g.C && (g.C % cs != 0 || cs % V != 0 || cs * 16 / V < 64)) cs += D;
    const LastRows r = last_rows(g.C, cs, D, g.P, V, kGnThreads);
    if ((int64_t)r.ns * r.cv <= capacity) {
        int threads = 64;
        while (threads < kFusedThreads && (threads < r.cv || (int64_t)(threads / r.cv) * held < r.ns)) threads *= 2;
        p.rows = last_rows(g.C, cs, D, g.P, V, threads);
        p.lds = sizeof(float) * (size_t)(p.rows.threads * V + 2 * cs + 2 * (cs / D));
        if ((int64_t)p.rows.q * held >= p.rows.ns && p.rows.threads <= kFusedThreads && p.lds <= kLdsMax) {
            p.how = kFusedLast;
            p.slices = (int)(g.C / cs);
            return p;
        }
    }
    p.rows = last_rows(g.C, g.C, D, g.P, V, kGnThreads);
    p.lds = sizeof(float) * (size_t)(2 * p.rows.threads * V + g.C + 2 * g.groups);
    const int vectors = g.out_type == g.x_type ? kOnceVectors<float, float> : kOnceVectors<bf16, float>;
    if (p.lds <= kLdsMax && once_plan(g, p.rows, vectors, 512, &p.once)) {
        p.how = kOnceLast;
        p.chunks = p.once.chunks;
        return p;
    }
    p.how = kSplitLast;
    split_chunks(g.B, p.rows.ns, 4 * p.rows.q, 64 * p.rows.q, &p.per, &p.chunks);
    p.lds = sizeof(float) * (size_t)(p.rows.threads * V + 2 * g.C);
    return p;
}

// Joining in every workgroup of grad_x reads its item's partial sums in each: worth it while those and the
// workgroups are few.
Plan plan_backward(const GroupNorm& g) {
    Plan p = plan_kernels(g);
    const bool split = p.how == kSplitLast || p.how == kSplitFirst || p.how == kCross;
    p.join = split && g.C * p.chunks <= 2048 && g.B * g.C * g.P <= (int64_t)4096 * 4096;
    return p;
}

bool fused(const Plan& p) { return p.how == kFusedLast || p.how == kFusedFirst; }

// (s1, s2) of each group, or the slots where chunks exchange theirs
int64_t group_pairs(const GroupNorm& g, const Plan& p) {
    return g.B * g.groups * (p.how == kOnceLast ? p.once.chunks : 1);
}

}  // namespace

size_t gn_backward_workspace(const GroupNorm& g) {
    const Plan p = plan_backward(g);
    return sizeof(float2) * (size_t)(g.B * g.C * p.chunks + group_pairs(g, p));
}

int gn_backward_kernels(const GroupNorm& g, bool need_x, bool need_w, const char** names) {
    const Plan p = plan_backward(g);
    int k = 0;
    if (p.how == kOnceLast) {
        names[k++] = "gn_clear";
        names[k++] = "gn_bwd_once";
        if (need_w) names[k++] = "gn_bwd_finish";
        return k;
    }
    names[k++] = fused(p) ? "gn_bwd_fused" : p.how == kCross ? "gn_bwd_sums_cross" : "gn_bwd_sums";
    if (need_w ? !(p.join && need_x) : !fused(p) && !p.join) names[k++] = "gn_bwd_finish";
    if (need_x && !fused(p)) names[k++] = p.how == kCross ? "gn_bwd_apply_cross" : "gn_bwd_apply";
    return k;
}

hipError_t gn_backward_launch(const GroupNorm& g, const GroupNormArgs& a, int kernel, hipStream_t s) {
    const Plan p = plan_backward(g);
    const int D = (int)(g.C / g.groups), C = (int)g.C, P = (int)g.P;
    const int64_t runs = g.B * g.groups;
    float2* part = static_cast<float2*>(a.ws);
    float2* gsum = part + g.B * g.C * p.chunks;
    if (p.how == kOnceLast && kernel == 0)
        return launch_clear(reinterpret_cast<uint64_t*>(gsum), group_pairs(g, p), s);
    const bool need_w = a.grad_weight || a.grad_bias, join = p.join && a.grad_x;
    const Parts parts{part, g.B, C, D, p.chunks, p.last, 1.0f / ((float)D * (float)P), a.grad_weight, a.grad_bias};
    if (!join && kernel == (p.how == kOnceLast ? 2 : 1)) {
        const bool need_groups = !fused(p) && p.how != kOnceLast && a.grad_x;
        const int64_t ngroups = need_groups ? runs : 0, all = kFinishThreads / 64;
        const int waves = finish_waves(parts);
        const int64_t blocks = (waves == 1 ? (ngroups + all - 1) / all : ngroups) + param_blocks(parts);
        return launch_kernel(k_gn_bwd_finish, grid_of(blocks), dim3(kFinishThreads), 0, s, parts, a.weight, gsum,
                             ngroups, waves);
    }
    Parts joined = parts;             // as the kernels of grad_x get it
    if (!join) joined.part = nullptr;
    const int64_t extra = join && need_w ? param_blocks(parts) : 0;
    return with_types(g, [&](auto tx, auto ty) {
        using TX = decltype(tx);
        using TY = decltype(ty);
        const TX* x = static_cast<const TX*>(a.x);
        const TY* dy = static_cast<const TY*>(a.out);
        const float* stats = a.stats;
        TX* gx = static_cast<TX*>(a.grad_x);
        return with_act(g.act, [&](auto act) {
            constexpr int ACT = decltype(act)::value;
            if (fused(p)) {
                float2* mine = a.grad_weight || a.grad_bias ? part : nullptr;
                if (p.how == kFusedLast) {
                    const int64_t blocks = g.B * p.slices;
                    return launch_kernel(k_gn_bwd_fused_last<ACT, TX, TY>, grid_of(blocks), dim3(p.rows.threads), p.lds,
                                         s, x, dy, a.weight, a.bias, stats, gx, mine, p.rows, p.slices, blocks);
                }
                return launch_kernel(k_gn_bwd_fused_first<ACT, TX, TY>, grid_of(runs), dim3(p.threads), p.lds, s, x, dy,
                                     a.weight, a.bias, stats, gx, mine, D, P, (int)g.groups, fast_div(P), runs);
            }
            if (p.how == kOnceLast)
                return with_vectors<kOnceVectors<TX, TY>>(p.once.nv, [&](auto nv) {
                    constexpr int NV = decltype(nv)::value;
                    const OnceArgs<TX, TY> args{x,  dy,
                                                a.weight, a.bias,
                                                stats, gx,
                                                a.grad_weight || a.grad_bias ? part : nullptr,
                                                reinterpret_cast<uint64_t*>(gsum),
                                                p.rows, p.once, once_looks.load()};
                    return launch_kernel(k_gn_bwd_once_last<ACT, NV, TX, TY>, dim3((unsigned)p.once.total),
                                         dim3(p.rows.threads), p.lds, s, args);
                });
            if (kernel == 0) {
                if (p.how == kSplitLast) {
                    const int64_t blocks = g.B * p.chunks;
                    return launch_kernel(k_gn_bwd_sums_last<ACT, TX, TY>, grid_of(blocks), dim3(p.rows.threads), p.lds,
                                         s, x, dy, a.weight, a.bias, stats, part, p.rows, p.per, p.chunks, blocks);
                }
                if (p.how == kSplitFirst) {
                    const int64_t blocks = first_blocks(p.frows);
                    return launch_kernel(k_gn_bwd_sums_first<ACT, TX, TY>, grid_of(blocks), dim3(kGnThreads), 0, s, x,
                                         dy, a.weight, a.bias, stats, part, p.frows, C, D, blocks);
                }
                if (p.how == kWide) {
                    const int64_t blocks = g.B * p.chunks * ((C + kWideC - 1) / kWideC);
                    return launch_kernel(k_gn_bwd_sums_wide<ACT, TX, TY>, grid_of(blocks), dim3(kGnThreads), 0, s, x,
                                         dy, a.weight, a.bias, stats, part, C, P, D, p.per, p.chunks, blocks);
                }
                const int64_t blocks = g.B * p.chunks * p.tiles.tiles_c;
                if (g.x_last)
                    return launch_kernel(k_gn_bwd_sums_cross<ACT, true, TX, TY>, grid_of(blocks), dim3(kGnThreads), 0,
                                         s, x, dy, a.weight, a.bias, stats, part, p.tiles, C, P, D, p.per, p.chunks,
                                         blocks);
                return launch_kernel(k_gn_bwd_sums_cross<ACT, false, TX, TY>, grid_of(blocks), dim3(kGnThreads), 0, s,
                                     x, dy, a.weight, a.bias, stats, part, p.tiles, C, P, D, p.per, p.chunks, blocks);
            }
            const float2* gs = gsum;
            if (p.how == kSplitLast) {
                const int per = std::min(8 * p.rows.q, p.rows.ns), chunks = (p.rows.ns + per - 1) / per;
                const int64_t blocks = g.B * chunks;
                const size_t lds = join ? sizeof(float2) * (size_t)std::max<int64_t>(p.rows.threads, g.groups) : 0;
                return launch_kernel(k_gn_bwd_apply_last<ACT, TX, TY>, grid_of(blocks + extra), dim3(p.rows.threads),
                                     lds, s, x, dy, a.weight, a.bias, stats, gs, gx, p.rows, joined, per, chunks,
                                     blocks, extra);
            }
            if (p.how == kSplitFirst) {
                const FirstRows r = first_rows(g.B * g.C, g.P, kVec<TX>, 8);
                const int64_t blocks = first_blocks(r);
                return launch_kernel(k_gn_bwd_apply_first<ACT, TX, TY>, grid_of(blocks + extra), dim3(kGnThreads), 0, s,
                                     x, dy, a.weight, a.bias, stats, gs, gx, r, joined, C, D, blocks, extra);
            }
            if (p.how == kWide) {
                const int64_t blocks = g.B * g.P;
                return launch_kernel(k_gn_bwd_apply_wide<ACT, TX, TY>, grid_of(blocks), dim3(kGnThreads), 0, s, x, dy,
                                     a.weight, a.bias, stats, gs, gx, C, P, D, blocks);
            }
            const int64_t blocks = g.B * p.tiles.tiles_c * p.tiles.tiles_p;
            if (g.x_last)
                return launch_kernel(k_gn_bwd_apply_cross<ACT, true, TX, TY>, grid_of(blocks + extra), dim3(kGnThreads),
                                     0, s, x, dy, a.weight, a.bias, stats, gs, gx, p.tiles, joined, C, P, D, blocks,
                                     extra);
            return launch_kernel(k_gn_bwd_apply_cross<ACT, false, TX, TY>, grid_of(blocks + extra), dim3(kGnThreads), 0,
                                 s, x, dy, a.weight, a.bias, stats, gs, gx, p.tiles, joined, C, P, D, blocks, extra);
        });
    });
}

// ---- slots, empty ------------------------------------------------------------------------------
namespace {
// 2 us for 32 KiB of them, 5.3 for 64 or 128 KiB: a launch, and cold lines.
__global__ __launch_bounds__(kGnThreads) void k_gn_clear(uint64_t* slots, int64_t n) {
    const int64_t i = block_id() * kGnThreads + threadIdx.x;
    if (i < n) slots[i] = kEmpty;
}
}  // namespace
hipError_t launch_clear(uint64_t* slots, int64_t n, hipStream_t s) {
    return launch_kernel(k_gn_clear, grid_of((n + kGnThreads - 1) / kGnThreads), dim3(kGnThreads), 0, s, slots, n);
}

void set_exchange_looks(int looks) { once_looks.store(looks); }

// ---- both directions ---------------------------------------------------------------------------
int group_norm_kernels(const GroupNorm& g, const GroupNormArgs& a, bool backward, const char** names) {
    return backward ? gn_backward_kernels(g, a.grad_x, a.grad_weight || a.grad_bias, names)
                    : gn_forward_kernels(g, names);
}
size_t group_norm_workspace(const GroupNorm& g, bool backward) {
    return backward ? gn_backward_workspace(g) : gn_forward_workspace(g);
}
hipError_t launch_group_norm(const GroupNorm& g, const GroupNormArgs& a, bool backward, int kernel, hipStream_t s) {
    return backward ? gn_backward_launch(g, a, kernel, s) : gn_forward_launch(g, a, kernel, s);
}

}  // namespace fno
