// Device-side pieces of the channel products (fno_channels_kernel.hpp,
// fno_channels_bwd.hpp, fno_channels_grad.hip): operands of the matrix instructions, the splitting of
// float32 into them, and the tiles of fields they are loaded from.
//
// All products run on v_mfma_f32_32x32x16_{bf16,f16}.  A lane l holds, of
// either operand, row (column) l % 32 and 8 neighbouring k from 8 (l / 32) on;
// of the result, column l % 32 and the rows 8 (r / 4) + 4 (l / 32) + r % 4 for
// r < 16.  The order of k and of rows is ours to choose as long as both
// operands agree: channels are dealt to the result's rows such that a lane's 16
// values are 16 neighbouring channels (row_channel), so that fields of either
// layout are read and written from registers as they lie.
//
// float32 values take three bfloat16 parts, each the rounding of what the ones
// before it leave: a part leaves up to 2^-8 of a value, two 2^-17, three nothing.
// Of the nine products of parts the six largest are formed; what the other three
// would add is up to 2 2^-25 + 2^-34 of the product, which is what a float32 product's
// rounding takes.  The 16-bit instructions do 16 times the float32 one's work in
// the same time, so six of them still take 3/8 of it.  A part of an infinity, or of
// a value above bfloat16's largest (3.39e38), is an infinity and the rest then a
// NaN: such inputs give a NaN where float32 sums might give an infinity.
#pragma once

#include <algorithm>

#include "fno_fields.hpp"

namespace fno {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// Channel of a 32-channel tile that row m of the result stands for.
__host__ __device__ __forceinline__ constexpr int row_channel(int m) {
    return 16 * ((m >> 2) & 1) + 4 * (m >> 3) + (m & 3);
}

// An operand of type T: parts of type E.
template <typename T>
struct Operand;
template <>
struct Operand<float> {
    typedef __bf16 E;
    typedef bf16x8 V;
    static constexpr int type = kTypeF32, parts = 3;
};
template <>
struct Operand<bf16> {
    typedef __bf16 E;
    typedef bf16x8 V;
    static constexpr int type = kTypeBf16, parts = 1;
};
template <>
struct Operand<f16> {
    typedef _Float16 E;
    typedef f16x8 V;
    static constexpr int type = kTypeF16, parts = 1;
};

template <typename V, int N>
struct Frag {
    V part[N];
};

// Parts of eight values.
template <typename V, int N>
__device__ __forceinline__ Frag<V, N> split(const float (&v)[8]) {
    Frag<V, N> f;
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f.part[k][i] = r[i];
            if (k + 1 < N) r[i] -= (float)f.part[k][i];
        }
    }
    return f;
}

// c += a b over the products of parts i and j that matter, i + j <= MOST, the smallest first.
template <int MOST, typename V, int NA, int NB>
__device__ __forceinline__ f32x16 mfma_upto(const Frag<V, NA>& a, const Frag<V, NB>& b, f32x16 c) {
#pragma unroll
    for (int s = MOST; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) c = mfma(a.part[i], b.part[s - i], c);
    return c;
}

// ---- activations ----------------------------------------------------------------------
// As act_value, in fewer instructions, which the products of 16-bit fields with
// many output channels are bound by: gelu(z) = max(z, 0) - |z| Phi(-|z|), and
// log2 Phi(-a) is a smooth function that a polynomial gives without a
// division: least squares of the error times Phi^1/2, made level, on [0, 6]; it
// falls on up to 12, where Phi is 2^-97 or less.  Degree 8: gelu within 9e-8, and
// of its own value within 5e-7 down to z = -1, 4e-4 down to -5.5; degree 6, for results
// rounded to 16 bits: 2.2e-7, 1.4e-6 and 7e-4.  Below -5.5, where gelu is less than
// 1.1e-7 in size, within 1e-10, which is not a small part of it any more.
template <int ACT, bool FINE>
__device__ __forceinline__ float product_act(float z) {
    if constexpr (ACT == kActGelu) {
        const float a = fminf(fabsf(z), 12.0f);
        float q;
        if constexpr (FINE) {
            q = -8.72182852e-07f;
            q = fmaf(q, a, 1.44495389e-05f);
            q = fmaf(q, a, -6.05394889e-05f);
            q = fmaf(q, a, -0.000458409078f);
            q = fmaf(q, a, 0.00750667136f);
            q = fmaf(q, a, -0.0528182127f);
            q = fmaf(q, a, -0.459096968f);
            q = fmaf(q, a, -1.15111935f);
            q = fmaf(q, a, -0.999999702f);
        } else {
            q = 3.2875083e-05f;
            q = fmaf(q, a, -0.000760217314f);
            q = fmaf(q, a, 0.00802443828f);
            q = fmaf(q, a, -0.0532797612f);
            q = fmaf(q, a, -0.458904028f);
            q = fmaf(q, a, -1.15114868f);
            q = fmaf(q, a, -0.999998987f);
        }
        return fmaf(-a, __builtin_amdgcn_exp2f(q), z < 0.0f ? 0.0f : z);       // (a NaN stays one)
    }
    return act_value<ACT>(z);
}

// A run of positions of one item that a wave works on: 32 NT of them, of
// which lane n % 32's j-th is p0 + pn n + pj j.
struct Tile {
    int64_t item;        // of which item (0 where all positions are one run)
    int64_t p0;
    int pn, pj;
    bool full;           // no position is behind the item's end
};

template <typename F>
__device__ __forceinline__ void with_field_type(int type, F&& f) {
    if (type == kTypeBf16) {
        f(bf16{});
    } else if (type == kTypeF16) {
        f(f16{});
    } else {
        f(0.0f);
    }
}

// Addresses are a base that all lanes share and 32-bit byte offsets.  Where
// something lies outside the field (a ragged tile), values are moved one by one
// through a buffer resource that ends with the field, places outside it at
// offset kOutside: such loads return zero and such stores are dropped, without a branch.
constexpr uint32_t kOutside = 0x80000000u;

template <typename T>
__device__ __forceinline__ T buffer_load(__amdgpu_buffer_rsrc_t rs, uint32_t at) {
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(rs, (int)at, 0, 0));
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(rs, (int)at, 0, 0));
    }
}
template <typename T>
__device__ __forceinline__ void buffer_store(__amdgpu_buffer_rsrc_t rs, uint32_t at, T v) {
    if constexpr (sizeof(T) == 4) {
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), rs, (int)at, 0, 0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), rs, (int)at, 0, 0);
    }
}
// Offsets that are the same for every tile are formed again where they are
// used: dozens of them kept from tile to tile would take the registers of the products.
__device__ __forceinline__ void per_tile(uint32_t& lane_offset, uint32_t& step) {
    step = __builtin_amdgcn_readfirstlane(step);
    asm volatile("" : "+v"(lane_offset), "+s"(step));
}
template <typename T>
__device__ __forceinline__ T* from(T* base, uint32_t bytes) {
    return reinterpret_cast<T*>(reinterpret_cast<char*>(base) + bytes);
}
template <typename T>
__device__ __forceinline__ const T* from(const T* base, uint32_t bytes) {
    return reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + bytes);
}

// 16 of a lane's values of a 32-channel part of a result tile, as one of NT
// chunks (few registers are busy at a time), and their places in a field.
// Channels last: chunk j holds position j, z[r] channel c0 + 16 (lane / 32) + r.
// Channels first: chunk q holds 16 / NT channels, z[NT i + j] is channel
// c0 + 16 (lane / 32) + 16 / NT q + i at position j.
template <bool LAST, int NT>
__device__ __forceinline__ constexpr int chunk_pos(int q, int i) { return LAST ? q : i % NT; }
template <bool LAST, int NT>
__device__ __forceinline__ constexpr int chunk_row(int q, int i) { return LAST ? i : 16 / NT * q + i / NT; }

// A chunk's values as they lie in the field.  Those of channels that do not
// exist are made zero where they are used: earlier would wait for the load.
template <typename T>
struct Values {
    T v[16] __attribute__((aligned(16)));

    // NT = 1: of the 16 channels of the lane's half of the part at c0
    __device__ __forceinline__ void keep(int C, int c0) {
        if (c0 + 32 <= C) return;
        const int channels = C - c0 - 16 * (int)((threadIdx.x & 63) >> 5);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = i < channels ? v[i] : (T)0.0f;
    }
};

// Bytes of LDS that a wave turns channels-last results in: 32 positions of 32
// channels, rows 16 bytes longer than that, so that those of neighbouring lanes start on other banks.
constexpr int kTurnBytes = 32 * (32 * 4 + 16);

template <typename T, bool LAST, int NT>
struct Places {
    int64_t start;           // elements from the field's start to the part's, the same in all lanes
    uint32_t left;           // bytes from there to the field's (channels first: the item's) end, or enough; 0 behind it
    uint32_t at, step;       // bytes: the lane's first channel and position; from a position (LAST) or channel to the next
    int channels;            // of the lane's half of the part that exist
    int part;                // of the part that exist
    int positions;           // of the tile that exist
    int C;
    int first, pn, pj;       // the lane's first position in the tile; from lane to lane, from one of its own to the next
    bool full;               // all positions exist
    bool readable;           // channels last: rows may be read to the part's end

    __device__ __forceinline__ Places(const Tile& t, int C_, int64_t P, int64_t items, int c0) {
        const int lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
        C = C_;
        start = t.item * P * C + (LAST ? t.p0 * C + c0 : c0 * P + t.p0);
        const int64_t more = ((LAST ? (P - t.p0) * C - c0 : (C - c0) * P - t.p0)) * (int64_t)sizeof(T);
        left = (uint32_t)max((int64_t)0, min(more, (int64_t)kOutside));
        pn = t.pn;
        pj = t.pj;
        first = n * pn;
        at = (LAST ? (uint32_t)(first * C + 16 * h) : (uint32_t)(16 * h * P + first)) * (uint32_t)sizeof(T);
        step = (uint32_t)(LAST ? pj * C : P) * (uint32_t)sizeof(T);
        per_tile(at, step);
        part = C - c0;
        channels = part - 16 * h;
        positions = (int)min(P - t.p0, (int64_t)32 * NT);
        full = t.full;
        readable = full && (c0 + 32 <= C || t.item + 1 < items || t.p0 + 32 * NT + 32 <= P);
    }
    __device__ __forceinline__ uint32_t place(int q, int i) const {
        const int j = chunk_pos<LAST, NT>(q, i), r = chunk_row<LAST, NT>(q, i);
        const bool in = r < channels && first + j * pj < positions;
        return in ? at + (LAST ? j * step + r * (uint32_t)sizeof(T) : r * step + j * (uint32_t)sizeof(T)) : kOutside;
    }

    // (values of channels that do not exist may be anything)
    __device__ __forceinline__ void load(const void* field, int q, float (&z)[16]) const {
        const T* f = static_cast<const T*>(field) + start;
        if (LAST ? readable : full) {
            if constexpr (LAST) {
                constexpr int V = 16 / sizeof(T);
#pragma unroll
                for (int k = 0; k < 16; k += V) {
                    float v[V];
                    load_vec<V>(from(f, at + q * step) + k, v);
#pragma unroll
                    for (int i = 0; i < V; ++i) z[k + i] = v[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; i += NT) {
                    const int r = chunk_row<LAST, NT>(q, i);
                    float v[NT];
                    load_vec<NT>(from(f, r < channels ? at + r * step : (uint32_t)first * (uint32_t)sizeof(T)), v);
#pragma unroll
                    for (int j = 0; j < NT; ++j) z[i + j] = v[j];
                }
            }
        } else {
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(f, left);
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = (float)buffer_load<T>(rs, place(q, i));
        }
    }

    // As load, but as the field holds the values.
    __device__ __forceinline__ void fetch(const void* field, int q, Values<T>& z) const {
        const T* f = static_cast<const T*>(field) + start;
        if (LAST ? readable : full) {
            if constexpr (LAST) {
                typedef typename VecOf<T, 8>::type V8;
#pragma unroll
                for (int k = 0; k < 16; k += 8)
                    *reinterpret_cast<V8*>(z.v + k) = *reinterpret_cast<const V8*>(from(f, at + q * step) + k);
            } else {
                typedef typename VecOf<T, NT>::type VN;
#pragma unroll
                for (int i = 0; i < 16; i += NT) {
                    const int r = chunk_row<LAST, NT>(q, i);
                    *reinterpret_cast<VN*>(z.v + i) = *reinterpret_cast<const VN*>(
                        from(f, r < channels ? at + r * step : (uint32_t)first * (uint32_t)sizeof(T)));
                }
            }
        } else {
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(f, left);
#pragma unroll
            for (int i = 0; i < 16; ++i) z.v[i] = buffer_load<T>(rs, place(q, i));
        }
    }

    // Channels last, lanes hold 16 channels of a position: the part is turned in `turn` (this wave's), so
    // that neighbouring lanes write neighbouring 16 bytes of a row.
    __device__ __forceinline__ void store(void* field, int q, const float (&z)[16], unsigned char* turn) const {
        T* f = static_cast<T*>(field) + start;
        if constexpr (LAST) {
            const int lane = threadIdx.x & 63;
            constexpr int V = 16 / sizeof(T), row = 32 * sizeof(T) + 16, lanes = 32 / V;
            typedef T VT __attribute__((ext_vector_type(V)));
            VT* mine = reinterpret_cast<VT*>(turn + (lane & 31) * row + (lane >> 5) * 16 * sizeof(T));
#pragma unroll
            for (int k = 0; k < 16 / V; ++k) {
                VT v;
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = (T)z[k * V + i];
                mine[k] = v;
            }
            __builtin_amdgcn_wave_barrier();
            const int c = lane % lanes * V;
#pragma unroll
            for (int k = 0; k < 32; k += 64 / lanes) {
                const int n = k + lane / lanes, p = n * pn + q * pj;
                const VT v = *reinterpret_cast<const VT*>(turn + n * row + c * sizeof(T));
                T* o = f + (uint32_t)(p * C + c);
                if (p < positions && c + V <= part) {
                    *reinterpret_cast<typename VecOf<T, V>::type*>(o) = v;
                } else if (p < positions) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (c + i < part) o[i] = v[i];
                }
            }
            __builtin_amdgcn_wave_barrier();
        } else if (full) {
#pragma unroll
            for (int i = 0; i < 16; i += NT) {
                const int r = chunk_row<LAST, NT>(q, i);
                float v[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) v[j] = z[i + j];
                if (r < channels) store_vec<NT>(from(f, at + r * step), v);
            }
        } else {
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(f, left);
#pragma unroll
            for (int i = 0; i < 16; ++i) buffer_store<T>(rs, place(q, i), (T)z[i]);
        }
    }
};

// ---- input tiles ------------------------------------------------------------------
// 16 channels from k0 on of a tile's positions, as they are loaded: channels
// first, NT positions of each of the lane's 8 channels; channels last, 8
// channels of each of its NT positions.  Channels that do not exist may hold
// anything until keep() makes them zero, where they are used.
template <typename T, bool LAST, int NT>
struct Raw {
    T v[LAST ? NT : 8][LAST ? 8 : NT] __attribute__((aligned(16)));

    __device__ __forceinline__ void keep(int C, int k0) {
        if (k0 + 16 <= C) return;
        const int more = C - k0 - 8 * (int)((threadIdx.x & 63) >> 5);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                T& q = v[LAST ? j : i][LAST ? i : j];
                q = i < more ? q : (T)0.0f;
            }
    }
};

template <typename T, bool LAST, int NT>
__device__ __forceinline__ void load_raw(Raw<T, LAST, NT>& raw, const void* field, const Tile& t, int C, int64_t P,
                                         int64_t items, int k0) {
    const int lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
    const T* x = static_cast<const T*>(field) + (t.item * P * C + (LAST ? t.p0 * C + k0 : k0 * P + t.p0));
    const int more = C - k0 - 8 * h;          // channels that exist from the lane's first on
    constexpr uint32_t S = sizeof(T);
    if constexpr (LAST) {
        typedef typename VecOf<T, 8>::type V8;
        uint32_t at = (uint32_t)(n * t.pn * C + 8 * h) * S, step = (uint32_t)(t.pj * C) * S;
        per_tile(at, step);
        // a row's tail may be read into the next rows, but not behind the field
        if (t.full && (k0 + 16 <= C || t.item + 1 < items || t.p0 + 32 * NT + 16 <= P)) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
                *reinterpret_cast<V8*>(raw.v[j]) = *reinterpret_cast<const V8*>(from(x, at + j * step));
        } else {
            const int64_t bytes = ((P - t.p0) * C - k0) * (int64_t)S;
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(x, (uint32_t)min(bytes, (int64_t)kOutside));
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    raw.v[j][i] = buffer_load<T>(rs, i < more ? at + j * step + i * S : kOutside);
        }
    } else {
        typedef typename VecOf<T, NT>::type VN;
        uint32_t step = (uint32_t)P * S, at = 8 * h * step + (uint32_t)(n * t.pn) * S;
        per_tile(at, step);
        if (t.full && k0 + 16 <= C) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<VN*>(raw.v[i]) = *reinterpret_cast<const VN*>(from(x, at + i * step));
        } else if (t.full) {
#pragma unroll
            for (int i = 0; i < 8; ++i)        // channels that do not exist: channel k0
                *reinterpret_cast<VN*>(raw.v[i]) =
                    *reinterpret_cast<const VN*>(from(x, i < more ? at + i * step : (uint32_t)(n * t.pn) * S));
        } else {
            const int64_t bytes = ((C - k0) * P - t.p0) * (int64_t)S;
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(x, (uint32_t)min(bytes, (int64_t)kOutside));
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    raw.v[i][j] = buffer_load<T>(rs, n * t.pn + j < P - t.p0 ? at + i * step + j * S : kOutside);
        }
    }
}

// The operand of position j.
template <int N, typename T, bool LAST, int NT>
__device__ __forceinline__ Frag<typename Operand<T>::V, N> operand(const Raw<T, LAST, NT>& raw, int j) {
    typedef typename Operand<T>::V V;
    if constexpr (Operand<T>::parts == 1) {
        Frag<V, 1> f;
#pragma unroll
        for (int i = 0; i < 8; ++i) f.part[0][i] = LAST ? raw.v[j][i] : raw.v[i][j];
        return f;
    } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = LAST ? raw.v[j][i] : raw.v[i][j];
        return split<V, N>(v);
    }
}

// ---- sums over positions -------------------------------------------------------------
// Parts of x and W (those of g are three), and the products formed, i + j up to these: for z,
// for grad_x (rounded to x's type), for grad_W.
template <typename T>
struct Scheme;
template <>
struct Scheme<float> {
    static constexpr int x = 3, z = 2, gx = 2, gw = 2;
};
template <>
struct Scheme<bf16> {
    static constexpr int x = 1, z = 0, gx = 1, gw = 2;
};
template <>
struct Scheme<f16> {
    static constexpr int x = 2, z = 2, gx = 1, gw = 2;
};

// Step s (of two) of the operand of 16 values.
template <int N, typename T>
__device__ __forceinline__ Frag<bf16x8, N> step_of(const T* v, int s) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)v[8 * s + i];
    return split<bf16x8, N>(f);
}

// What a product with the identity must not see: 0 times an infinity or NaN takes all 32 channels of a
// position along.  Such a value of g makes its row of grad_weight and its entry of grad_bias infinite or NaN, one
// of x its column; here it is set to zero and its channel is marked, whose sums leave as NaN.  For every tile
// this would cost 5% of a backward pass, so it is done only where sums show such a value, in another
// pass over their tiles.
template <int N>
__device__ __forceinline__ void set_apart(Frag<bf16x8, N> (&a)[2], uint32_t* marked) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool bad = !(fabsf((float)a[s].part[0][i]) < __builtin_inff());
            __hip_atomic_fetch_or(marked + 16 * h + 8 * s + i, bad ? 1u : 0u, __ATOMIC_RELAXED,
                                  __HIP_MEMORY_SCOPE_WORKGROUP);
#pragma unroll
            for (int p = 0; p < N; ++p) a[s].part[p][i] = bad ? (__bf16)0.0f : a[s].part[p][i];
        }
}

// A 32 x 32 part of an operand, turned: lanes hold what was its steps' k.  Returns the sum of the lane's values.
template <int N>
__device__ __forceinline__ float turned(const Frag<bf16x8, N> (&a)[2], const bf16x8 (&one)[2],
                                        Frag<bf16x8, N> (&out)[2]) {
    float sum = 0.0f;
#pragma unroll
    for (int p = 0; p < N; ++p) {
        f32x16 d;
#pragma unroll
        for (int r = 0; r < 16; ++r) d[r] = 0.0f;
        d = mfma(a[0].part[p], one[0], d);
        d = mfma(a[1].part[p], one[1], d);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            out[r >> 3].part[p][r & 7] = d[r];
            sum += d[r];
        }
    }
    return sum;
}

// Whether any of a wave's sums is not finite.
template <int MO, int MI>
__device__ __forceinline__ bool any_not_finite(const f32x16 (&dw)[MO][MI], const float (&db)[MO]) {
    float m[4] = {};                        // 0, or a NaN from then on
#pragma unroll
    for (int mo = 0; mo < MO; ++mo) {
        m[0] = fmaf(db[mo], 0.0f, m[0]);
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int r = 0; r < 16; ++r) m[r & 3] = fmaf(dw[mo][mi][r], 0.0f, m[r & 3]);
    }
    return __builtin_amdgcn_ballot_w64((m[0] + m[1]) + (m[2] + m[3]) != 0.0f) != 0;
}

// Sums of g x (and of g) that four waves of a workgroup hold, joined one after the
// other, so in a fixed order: rows o0.., columns i0.. of part [Cout][Cin] and, of the
// first columns' workgroup, the sums of g behind it.  join holds MO MI 1024 floats, sums 32 MO; marked_o and
// marked_i are the marks of these rows and columns, looked at where *spoilt is not 0 (null: not).
template <int MO, int MI>
__device__ __forceinline__ void join_sums(const f32x16 (&dw)[MO][MI], const float (&db)[MO], float* join, float* sums,
                                          const uint32_t* spoilt, const uint32_t* marked_o, const uint32_t* marked_i,
                                          float* part, int o0, int i0, int Cout, int Cin) {
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int k = 0; k < 4; ++k) {
        __syncthreads();
        if (wave != k) continue;
#pragma unroll
        for (int mo = 0; mo < MO; ++mo) {
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float* q = join + ((mo * MI + mi) * 16 + r) * 64 + lane;
                    *q = k ? *q + dw[mo][mi][r] : dw[mo][mi][r];
                }
            const float s = swap_add<32>(db[mo]);
            if (h == 0) sums[32 * mo + lane] = k ? sums[32 * mo + lane] + s : s;
        }
    }
    __syncthreads();
    const bool look = spoilt && __builtin_amdgcn_readfirstlane(*spoilt);
    for (int q = threadIdx.x; q < MO * MI * 1024; q += 256) {
        const int l = q & 63, r = (q >> 6) & 15, mi = (q >> 10) % MI, mo = (q >> 10) / MI;
        const int o = 32 * mo + 8 * (r >> 2) + 4 * (l >> 5) + (r & 3), i = 32 * mi + (l & 31);
        const bool marked = look && (marked_o[o] | marked_i[i]);
        if (o0 + o < Cout && i0 + i < Cin)
            part[(int64_t)(o0 + o) * Cin + i0 + i] = marked ? __builtin_nanf("") : join[q];
    }
    if (i0 == 0)
        for (int o = threadIdx.x; o < 32 * MO && o0 + o < Cout; o += 256)
            part[(int64_t)Cin * Cout + o0 + o] = look && marked_o[o] ? __builtin_nanf("") : sums[o];
}

// ---- the product's kernel (fno_channels_kernel.hpp) ---------------------------------
struct ProductArgs {
    const void *x, *w;
    const float* bias;
    const void* branch;      // of out's type and layout, null for none
    void* out;
    const void* grad;        // slope mode: grad_out, of out's type and layout
    float* g;                // slope mode: grad_out act'(z), in out's layout
    int64_t B, P;            // items and positions, as tiles see them
    int Cin, Cout;
    int act;
    bool branch_after, merged, slope, transposed;
    int w_type;
    int tiles_item;          // tiles of an item
    int64_t tiles;
    int cout_tiles;          // workgroups over the output channels
    int groups;              // workgroups over the positions
    int chunk, nks;          // steps of 16 input channels: in LDS at a time, in all
};

// Parts that a product's weight is held in: it is of x's type, beside a float32 x and a 16-bit result of the result's.
constexpr int weight_parts(int x_type, int out_type) {
    return x_type != kTypeF32 || out_type == kTypeBf16 ? 1 : out_type == kTypeF16 ? 2 : 3;
}
// Steps of 16 channels that are loaded before they are used: 64 channels of 16
// bits, 32 of 32 bits.  Chunks of staged weights are whole numbers of them.
constexpr int steps_ahead(int x_type) { return x_type == kTypeF32 ? 2 : 4; }
constexpr int positions_a_wave(bool merged) { return merged ? 32 : 64; }

// The form of the kernel that a product takes.
struct ProductPlan {
    int mt;          // 32-channel parts of the output a wave: 1, 2 or 4
    int waves;       // a workgroup: 4 or 8
    int nks, chunk;  // steps of 16 input channels: in all, in LDS at a time
};
inline ProductPlan plan_product(const ProductArgs& a, int x_type, int out_type, bool merged) {
    const int width = positions_a_wave(merged);
    const int64_t runs = merged ? 1 : a.B, length = merged ? a.B * a.P : a.P;
    const int64_t groups = (runs * ((length + width - 1) / width) + 3) / 4;
    ProductPlan p;
    // As many output channels a wave as there are, up to 128, so that x is read once; fewer where
    // that would leave half of the CUs without a workgroup, since a wave's latency is all there is
    // then (one position, 256 -> 256 bfloat16: 13.6 us with 32 channels a wave, 27.0 with 128; 512
    // positions, 128 -> 256 float32: 13.0 and 36.8; 4 x 1024 positions, 64 -> 64 float32: 10.7 with 32, 15.0 with 64).
    p.mt = a.Cout > 64 && groups * ((a.Cout + 127) / 128) >= 128  ? 4
           : a.Cout > 32 && groups * ((a.Cout + 63) / 64) >= 128 ? 2
                                                                 : 1;
    p.nks = (a.Cin + 15) / 16;
    const int step = weight_parts(x_type, out_type) * p.mt * 1024;          // bytes of weights for 16 input channels
    // 60 KiB leave room for two workgroups of four waves a CU; one of eight has twice that
    const bool wide = (int64_t)p.nks * step > 60 * 1024;
    const int most = (wide ? 120 : 60) * 1024 / step, ahead = steps_ahead(x_type);
    p.waves = wide ? 8 : 4;
    p.chunk = p.nks <= most ? p.nks : most / ahead * ahead;
    return p;
}
// By type of x; out is of out_type (x's or float32; any for float32).
hipError_t launch_product_f32(const ProductArgs& a, bool last, bool out_last, int out_type, hipStream_t s);
hipError_t launch_product_bf16(const ProductArgs& a, bool last, bool out_last, int out_type, hipStream_t s);
hipError_t launch_product_f16(const ProductArgs& a, bool last, bool out_last, int out_type, hipStream_t s);

// ---- the backward pass in one kernel (fno_channels_bwd.hpp) --------------------------
struct BackwardArgs {
    const void *x, *w;
    const float* bias;
    const void *branch, *grad;     // branch only where it is inside the activation
    void *grad_x, *grad_branch;    // null where not asked for
    float* part;                   // [groups][Cout Cin + Cout]: sums of g x and of g; null where not asked for
    int64_t B, P;
    int Cin, Cout, act;
    bool merged;
    int tiles_item, groups;
    int64_t tiles;
};
// What a wave's registers hold: up to 64 channels, of 16-bit fields 128 on one side.  (float32, 32 x 64 x 64
// positions: 64 -> 128 takes 238 us in one kernel and 144 in four, 128 -> 64 99 and 117; 78 -> 15, channels
// last, 56445 positions, 129 and 63.)
inline bool backward_fits(int Cin, int Cout, int x_type) {
    return std::max(Cin, Cout) <= (x_type == kTypeF32 ? 64 : 128) && std::min(Cin, Cout) <= 64;
}
hipError_t launch_backward_f32(const BackwardArgs& a, bool last, bool out_last, hipStream_t s);
hipError_t launch_backward_bf16(const BackwardArgs& a, bool last, bool out_last, hipStream_t s);
hipError_t launch_backward_bf16_f32(const BackwardArgs& a, bool last, bool out_last, hipStream_t s);
hipError_t launch_backward_f16(const BackwardArgs& a, bool last, bool out_last, hipStream_t s);
hipError_t launch_backward_f16_f32(const BackwardArgs& a, bool last, bool out_last, hipStream_t s);


// ---- gradient of the weight alone (fno_channels_grad.hip) ------------------------------
struct WeightGradArgs {
    const void *x, *g;
    float* part;                   // [splits][Cout Cin + Cout]: sums of g x and of g
    int64_t B, P, tiles;
    int Cin, Cout, tiles_item, splits;
    bool merged;
};
// 64 x 64 channels a workgroup, in `splits` shares of the positions
hipError_t launch_channel_weight_grad(WeightGradArgs a, int x_type, int g_type, bool x_last, bool g_last,
                                      hipStream_t s);

}  // namespace fno
