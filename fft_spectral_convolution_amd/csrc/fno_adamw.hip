// AdamW over many tensors at once:
//   g' = g coef,  m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2
//   p' = p (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
// with coef the clipping factor of a given norm (1 without one), moments held
// in float32 or in 8 bits, and optionally a 16-bit copy of p'.
//
// The tensors are handed to each launch as a table in its kernel arguments
// (kAdamTable tensors a launch), cut into chunks of 4096 values, one a
// workgroup.
//
// Moments in 8 bits.  128 neighbouring values of a tensor are a block and
// share a power of two 2^e, e the exponent of the largest of them (a byte, e +
// 127).  A code is the value's own exponent below that and three bits of its
// fraction: 1 + 4 + 3 bits for m, 5 + 3 bits for v, which has no sign.  Scales
// that are powers of two make every code an exact shift of its value's bits,
// so scaling rounds nothing and divides by nothing.  The update is formed in
// double (a sum rounded to float32 first would now and then round to another
// code: one in 10^6, each an eighth of the value), and the code takes the part
// of the fraction that it drops as the probability of rounding up.  Rounding
// to nearest would not do: b2 = 0.999 moves v by at most 0.1% a step towards
// smaller values, codes are 6 to 12% apart, and v would stay where it is.
// The random bits are a hash of (seed, step, tensor, number of the value), so
// equal calls give equal bits.
#include <type_traits>

#include "fno_fields.hpp"

namespace fno {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;          // values a workgroup
constexpr int kBlock = 128;           // values of 8-bit moments that share an exponent
static_assert(kChunk % kBlock == 0, "chunks hold whole blocks");

// Tensor that holds a chunk (as in the gradient norm: the last whose first chunk is not beyond it).
__device__ __forceinline__ int tensor_of(const AdamTable& t, uint32_t chunk) {
    static_assert(kAdamTable <= 64, "one entry a lane");
    const int lane = threadIdx.x & 63;
    const uint64_t b = __ballot(lane < kAdamTable && t.first[lane < kAdamTable ? lane : 0] <= chunk);
    return __builtin_amdgcn_readfirstlane(__popcll(b) - 1);
}

template <typename F>
__device__ __forceinline__ void with_type(int type, F&& f) {
    if (type == kTypeBf16) {
        f(bf16{});
    } else if (type == kTypeF16) {
        f(f16{});
    } else {
        f(0.0f);          // complex values as pairs
    }
}

// What one step needs besides the tensors, the same for all of them.
struct Step {
    float decay, size, inv_c2, eps, coef;      // 1 - lr wd, lr / (1 - b1^t), (1 - b2^t)^-1/2
    float inv_c2_small;                        // 2^-32 of that
    double b1, b2;
    uint32_t step;
};
__device__ Step make_step(const AdamOptions& o) {
    Step s;
    const double lr = o.lr_dev ? (double)*o.lr_dev : o.lr;
    double c1 = o.c1, c2 = o.c2;
    s.step = (uint32_t)o.step;
    if (o.step_dev) {              // a step number that a captured graph finds in memory
        const long long t = *o.step_dev;
        c1 = -expm1((double)t * o.log_b1);
        c2 = -expm1((double)t * o.log_b2);
        s.step = (uint32_t)t;
    }
    s.decay = (float)(1.0 - lr * o.weight_decay);
    s.size = (float)(lr / c1);
    s.inv_c2 = (float)(1.0 / sqrt(c2));
    s.inv_c2_small = s.inv_c2 * 0x1p-32f;
    s.eps = (float)o.eps;
    s.coef = 1.0f;
    if (o.norm) {                  // the factor of the clipping call: min(1, max_norm / (norm + 1e-6))
        const double c = (double)o.max_norm / ((double)*o.norm + 1e-6);
        s.coef = c > 1.0 ? 1.0f : (float)c;
    }
    s.b1 = o.b1;
    s.b2 = o.b2;
    return s;
}

// The device's root and reciprocal, good to 1 ulp: a few last bits of the update, which is
// a small part of p.  The root takes subnormal numbers for zero, so small v are scaled.
__device__ __forceinline__ float new_param(float p, float m, float v, const Step& s) {
    const bool small = v < 0x1p-96f;
    const float root = __builtin_amdgcn_sqrtf(v * (small ? 0x1p64f : 1.0f));
    const float denom = fmaf(root, small ? s.inv_c2_small : s.inv_c2, s.eps);
    return fmaf(-s.size * m, __builtin_amdgcn_rcpf(denom), p * s.decay);
}

template <int N, typename T>
__device__ __forceinline__ void load_some(const T* p, float (&v)[N], int n) {
    if (n == N) {
        load_vec<N>(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = j < n ? (float)p[j] : 0.0f;
    }
}
template <int N, typename T>
__device__ __forceinline__ void store_some(T* p, const float (&v)[N], int n) {
    if (n == N) {
        store_vec<N>(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < n) p[j] = (T)v[j];
    }
}

// 16 bits of a copy beside the parameter
template <int N>
__device__ __forceinline__ void store_copy(void* copy, int type, int64_t at, const float (&v)[N], int n) {
    if (!copy) return;
    if (type == kTypeBf16) {
        store_some(static_cast<bf16*>(copy) + at, v, n);
    } else {
        store_some(static_cast<f16*>(copy) + at, v, n);
    }
}

// ---- moments in 32 bits ---------------------------------------------------------
template <typename TP, typename TG>
__device__ __forceinline__ void chunk32(const AdamTable& t, int i, int64_t at, int n, const Step& s) {
    const TP* p = static_cast<const TP*>(t.p[i]) + at;
    TP* po = static_cast<TP*>(t.po[i]) + at;
    const TG* g = static_cast<const TG*>(t.g[i]) + at;
    const float* m = static_cast<const float*>(t.m[i]) + at;
    const float* v = static_cast<const float*>(t.v[i]) + at;
    float* mo = static_cast<float*>(t.mo[i]) + at;
    float* vo = static_cast<float*>(t.vo[i]) + at;
    const float b1 = (float)s.b1, b2 = (float)s.b2, a1 = (float)(1.0 - s.b1), a2 = (float)(1.0 - s.b2);
    auto update = [&](float (&pv)[4], const float (&gv)[4], float (&mv)[4], float (&vv)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float q = gv[j] * s.coef;
            mv[j] = fmaf(b1, mv[j], a1 * q);
            vv[j] = fmaf(b2, vv[j], a2 * (q * q));
            pv[j] = new_param(pv[j], mv[j], vv[j], s);
        }
    };
    constexpr int kStep = 4 * kThreads;
    if (n == kChunk) {
        // all of a chunk's loads in flight two vectors of each field at a time
#pragma unroll
        for (int c = 0; c < kChunk; c += 2 * kStep) {
            float pv[2][4], gv[2][4], mv[2][4], vv[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int k = c + u * kStep + 4 * threadIdx.x;
                load_vec<4>(p + k, pv[u]);
                load_vec<4>(g + k, gv[u]);
                load_vec<4>(m + k, mv[u]);
                load_vec<4>(v + k, vv[u]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int k = c + u * kStep + 4 * threadIdx.x;
                update(pv[u], gv[u], mv[u], vv[u]);
                store_vec<4>(po + k, pv[u]);
                store_vec<4>(mo + k, mv[u]);
                store_vec<4>(vo + k, vv[u]);
                store_copy(t.copy[i], t.ctype[i], at + k, pv[u], 4);
            }
        }
        return;
    }
    for (int k = 4 * threadIdx.x; k < n; k += kStep) {
        const int left = min(4, n - k);
        float pv[4], gv[4], mv[4], vv[4];
        load_some(p + k, pv, left);
        load_some(g + k, gv, left);
        load_some(m + k, mv, left);
        load_some(v + k, vv, left);
        update(pv, gv, mv, vv);
        store_some(po + k, pv, left);
        store_some(mo + k, mv, left);
        store_some(vo + k, vv, left);
        store_copy(t.copy[i], t.ctype[i], at + k, pv, left);
    }
}

// ---- moments in 8 bits ------------------------------------------------------------
// A bijection of 32-bit words whose output bits each depend on all input bits:
// two rounds of shift, exclusive or and product.  The factors are the leading
// fraction bits of the square roots of 2 and 3.
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x6A09E667u;
    x = (x ^ (x >> 15)) * 0xBB67AE85u;
    return x ^ (x >> 16);
}

constexpr int kTopM = 14, kTopV = 30;         // exponent codes below a block's largest value
constexpr int kLeastM = 1, kLeastV = 31;      // least exponent byte: every value is a float32, v's a normal one

template <bool SIGNED>
__device__ __forceinline__ float decode8(uint32_t code, float scale) {
    constexpr uint32_t top = SIGNED ? kTopM : kTopV, all = SIGNED ? 127 : 255;
    const uint32_t c = code & all;
    const uint32_t bits = (c << 20) + ((127 - top) << 23) | (SIGNED ? (code & 128) << 24 : 0);
    const float y = __builtin_bit_cast(float, bits) * scale;
    return c == 0 ? 0.0f : c == all ? __builtin_nanf("") : y;
}
__device__ __forceinline__ float exp8(uint8_t e) { return __builtin_bit_cast(float, (uint32_t)e << 23); }

__device__ __forceinline__ uint32_t high(double d) { return (uint32_t)(__builtin_bit_cast(uint64_t, d) >> 32); }

// Exponent byte of a block from the largest exponent field of its finite values.
template <bool SIGNED>
__device__ __forceinline__ int exp_byte(uint32_t f) {
    const int field = (int)f;
    return field == 0 ? 0 : max(SIGNED ? kLeastM : kLeastV, min(254, field - 1023 + 127));
}
// Code of d: `up` (17 bits) is added to the 17 bits of the high word that the code drops.
template <bool SIGNED>
__device__ __forceinline__ uint32_t encode8(double d, int e, uint32_t up) {
    constexpr int top = SIGNED ? kTopM : kTopV;
    const uint32_t h = high(d), a = h & 0x7fffffffu;
    int c = ((int)(a - ((uint32_t)(e - 127) << 20) + up) >> 17) - ((1023 - top) << 3);
    // A block's largest value may round up to 2^(e + 1), but not beyond float32.  A second moment that is
    // not zero stays so: its root divides a first moment that may have stayed, too.
    c = max(SIGNED ? 0 : 1, min((top + 1) * 8 - (e == 254), c));
    if constexpr (SIGNED) c |= c ? (int)(h >> 31) << 7 : 0;
    c = a == 0 ? 0 : c;
    return a >= 0x7ff00000u ? (SIGNED ? 127 : 255) : c;
}

// Largest of 16 neighbouring lanes, in each of them.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = dpp_max<kDppXor1>(v);
    v = dpp_max<kDppXor2>(v);
    v = dpp_max<kDppHalfMirror>(v);
    return dpp_max<kDppMirror>(v);
}
__device__ __forceinline__ uint32_t finite_high(double d) {
    const uint32_t h = high(d) & 0x7fffffffu;
    return h >= 0x7ff00000u ? 0 : h;
}

__device__ __forceinline__ void unpack8(const uint8_t* p, uint32_t (&c)[8]) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = ((j < 4 ? q.x : q.y) >> (8 * (j & 3))) & 0xff;
}
__device__ __forceinline__ void pack8(uint8_t* p, const uint32_t (&c)[8]) {
    uint2 q;
    q.x = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
    q.y = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
    *reinterpret_cast<uint2*>(p) = q;
}

// Eight values a lane, so 16 lanes hold a block.
template <typename TP, typename TG>
__device__ __forceinline__ void chunk8(const AdamTable& t, int i, int64_t at, int n, const Step& s, uint32_t key) {
    const TP* p = static_cast<const TP*>(t.p[i]) + at;
    TP* po = static_cast<TP*>(t.po[i]) + at;
    const TG* g = static_cast<const TG*>(t.g[i]) + at;
    const int64_t exps = (t.n[i] + kBlock - 1) / kBlock * kBlock;      // where the blocks' exponents lie
    const uint8_t* m = static_cast<const uint8_t*>(t.m[i]);
    const uint8_t* v = static_cast<const uint8_t*>(t.v[i]);
    uint8_t* mo = static_cast<uint8_t*>(t.mo[i]);
    uint8_t* vo = static_cast<uint8_t*>(t.vo[i]);
    key = mix32(key + (uint32_t)(at >> 32));
    const double a1 = 1.0 - s.b1, a2 = 1.0 - s.b2;
    auto vectors = [&](int k, auto all) {
        constexpr bool kAll = decltype(all)::value;          // no place is behind the tensor's end
        const int left = kAll ? 8 : max(0, min(8, n - k));
        const int64_t block = (at + k) / kBlock;
        float pv[8], gv[8];
        uint32_t mc[8], vc[8];
        load_some(p + k, pv, left);
        load_some(g + k, gv, left);
        unpack8(m + at + k, mc);
        unpack8(v + at + k, vc);
        const float ms = exp8(m[exps + block]), vs = exp8(v[exps + block]);
        double md[8], vd[8];
        uint32_t me = 0, ve = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double q = (double)(gv[j] * s.coef);
            md[j] = fma(s.b1, (double)decode8<true>(mc[j], ms), a1 * q);
            vd[j] = fma(s.b2, (double)decode8<false>(vc[j], vs), a2 * (q * q));
            if (!kAll && j >= left) md[j] = vd[j] = 0.0;     // places behind the end hold zeros
            me = max(me, high(md[j]) & 0x7fffffffu);
            ve = max(ve, high(vd[j]) & 0x7fffffffu);
        }
        // a block with infinities or NaN takes the exponent of its finite values
        if (max(me, ve) >= 0x7ff00000u) {
            me = ve = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                me = max(me, finite_high(md[j]));
                ve = max(ve, finite_high(vd[j]));
            }
        }
        const int mx = exp_byte<true>(row_max(me) >> 20), vx = exp_byte<false>(row_max(ve) >> 20);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t r = mix32((uint32_t)(at + k + j) ^ key);
            mc[j] = encode8<true>(md[j], mx, 2 * (r & 0xffff) + 1);
            vc[j] = encode8<false>(vd[j], vx, 2 * (r >> 16) + 1);
            pv[j] = new_param(pv[j], (float)md[j], (float)vd[j], s);
        }
        store_some(po + k, pv, left);
        pack8(mo + at + k, mc);
        pack8(vo + at + k, vc);
        if ((threadIdx.x & 15) == 0) {
            mo[exps + block] = (uint8_t)mx;
            vo[exps + block] = (uint8_t)vx;
        }
        store_copy(t.copy[i], t.ctype[i], at + k, pv, left);
    };
    const int whole = (n + kBlock - 1) / kBlock * kBlock;
    if (n == whole) {
        for (int k = 8 * threadIdx.x; k < whole; k += 8 * kThreads) vectors(k, std::true_type{});
    } else {
        for (int k = 8 * threadIdx.x; k < whole; k += 8 * kThreads) vectors(k, std::false_type{});
    }
}

// A table's moments are all of 32 bits or all of 8.  67 million floats of a model with
// spectral weights: 32 bits 335 to 340 us, 1.88 GB at 5.5 TB/s, memory (407 with one vector
// of each field in flight and one kernel for both kinds); 8 bits 230 to 240 us, 1.09
// GB at 4.6 TB/s beside 100 vector instructions a value, a fifth of them the random bits.  11
// small tensors: 4.9 us, a launch.
template <int BITS>
__global__ __launch_bounds__(kThreads, BITS == 8 ? 3 : 4) void k_adamw(AdamTable t, uint32_t nchunks, AdamOptions o) {
    const Step s = make_step(o);
    for (uint32_t c = blockIdx.x; c < nchunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const int64_t at = (int64_t)(c - t.first[i]) * kChunk;
        const int n = (int)min((int64_t)kChunk, t.n[i] - at);
        uint32_t key = mix32(mix32((uint32_t)o.seed) + (uint32_t)(o.seed >> 32));
        key = mix32(mix32(key + s.step) + (uint32_t)t.number[i]);
        with_type(t.ptype[i], [&](auto a) {
            with_type(t.gtype[i], [&](auto b) {
                if constexpr (BITS == 8) {
                    chunk8<decltype(a), decltype(b)>(t, i, at, n, s, key);
                } else {
                    chunk32<decltype(a), decltype(b)>(t, i, at, n, s);
                }
            });
        });
    }
}

// The values that 8-bit moments stand for: 67 million, 160 us, 677 MB at 4.2 TB/s.
__global__ __launch_bounds__(kThreads) void k_adamw_moments(AdamTable t, uint32_t nchunks) {
    for (uint32_t c = blockIdx.x; c < nchunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const int64_t at = (int64_t)(c - t.first[i]) * kChunk;
        const int n = (int)min((int64_t)kChunk, t.n[i] - at);
        const int64_t exps = (t.n[i] + kBlock - 1) / kBlock * kBlock;
        const uint8_t* m = static_cast<const uint8_t*>(t.m[i]);
        const uint8_t* v = static_cast<const uint8_t*>(t.v[i]);
        float* mo = static_cast<float*>(t.mo[i]) + at;
        float* vo = static_cast<float*>(t.vo[i]) + at;
        for (int k = 8 * threadIdx.x; k < n; k += 8 * kThreads) {
            const int left = min(8, n - k);
            const int64_t block = (at + k) / kBlock;
            const float ms = exp8(m[exps + block]), vs = exp8(v[exps + block]);
            uint32_t mc[8], vc[8];
            unpack8(m + at + k, mc);
            unpack8(v + at + k, vc);
            float a[8], b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] = decode8<true>(mc[j], ms);
                b[j] = decode8<false>(vc[j], vs);
            }
            store_some(mo + k, a, left);
            store_some(vo + k, b, left);
        }
    }
}

}  // namespace

int64_t adam_moment_bytes(int64_t n) {
    const int64_t blocks = (n + kBlock - 1) / kBlock;
    return (blocks * kBlock + blocks + 15) / 16 * 16;
}

uint32_t adam_table_chunks(AdamTable& t, int count) {
    uint64_t c = 0;
    for (int i = 0; i < kAdamTable; ++i) {
        t.first[i] = i < count ? (uint32_t)c : UINT32_MAX;
        if (i < count) c += (uint64_t)((t.n[i] + kChunk - 1) / kChunk);
    }
    return (uint32_t)c;
}

hipError_t launch_adamw(const AdamTable& t, uint32_t nchunks, const AdamOptions& o, hipStream_t s) {
    const dim3 grid(nchunks < 1u << 22 ? nchunks : 1u << 22), block(kThreads);
    return o.bits == 8 ? launch_kernel(k_adamw<8>, grid, block, 0, s, t, nchunks, o)
                       : launch_kernel(k_adamw<32>, grid, block, 0, s, t, nchunks, o);
}
hipError_t launch_adamw_moments(const AdamTable& t, uint32_t nchunks, hipStream_t s) {
    return launch_kernel(k_adamw_moments, dim3(nchunks < 1u << 22 ? nchunks : 1u << 22), dim3(kThreads), 0, s, t,
                         nchunks);
}

}  // namespace fno
