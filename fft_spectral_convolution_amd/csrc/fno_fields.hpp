// Device-side helpers of the field operators (group norm, gradient norm):
// element types, vector loads and stores, activations and block sums.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "fno_device.hpp"
#include "fno_internal.hpp"

namespace fno {

using bf16 = __bf16;
using f16 = _Float16;

// ---- element types ----------------------------------------------------------
// All arithmetic is in float; a 16-bit output is rounded once, to nearest
// even, when it is stored.  Vectors are only aligned to their elements (the
// device's vector loads and stores take any such address), so that rows of
// odd length and slices of packed buffers need no other path.
template <typename T, int N>
struct VecOf {
    typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};
template <typename T>
struct VecOf<T, 1> {
    typedef T type;
};

template <int N, typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[N]) {
    const typename VecOf<T, N>::type q = *reinterpret_cast<const typename VecOf<T, N>::type*>(p);
    if constexpr (N == 1) {
        v[0] = (float)q;
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = (float)q[j];
    }
}
// Outputs go past the caches (non-temporal), as those of the transforms do.
template <int N, typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[N]) {
    typename VecOf<T, N>::type q;
    if constexpr (N == 1) {
        q = (T)v[0];
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = (T)v[j];
    }
    __builtin_nontemporal_store(q, reinterpret_cast<typename VecOf<T, N>::type*>(p));
}

// ---- activations ---------------------------------------------------------------
// The vector instructions per value count: a 16-bit field is read and written
// at the memory's rate in about 40 of them.
//
// gelu(z) = z Phi(z) = max(z, 0) - |z| Phi(-|z|), with
//   Phi(-|z|) = erfc(a) / 2 = t exp(-a^2 + P(t)) / 2,  a = |z| / sqrt 2, t = 1 / (1 + a / 2),
// P the fit of epi_erfc (Numerical Recipes, "erfcc").  The exponential is a
// power of two: P's coefficients carry log2 e, the constant one also the
// factor 1/2.  18 instructions (a division and Phi itself: 30).  The device's
// reciprocal and power of two are good to 1 ulp.
constexpr float kLog2e = 1.44269504088896341f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == kActGelu) {
        constexpr double L = 1.44269504088896341;
        const float t = __builtin_amdgcn_rcpf(fmaf(0.353553390593273762f, fabsf(z), 1.0f));
        float p = (float)(0.17087277 * L);
        p = fmaf(p, t, (float)(-0.82215223 * L));
        p = fmaf(p, t, (float)(1.48851587 * L));
        p = fmaf(p, t, (float)(-1.13520398 * L));
        p = fmaf(p, t, (float)(0.27886807 * L));
        p = fmaf(p, t, (float)(-0.18628806 * L));
        p = fmaf(p, t, (float)(0.09678418 * L));
        p = fmaf(p, t, (float)(0.37409196 * L));
        p = fmaf(p, t, (float)(1.00002368 * L));
        p = fmaf(p, t, (float)(-1.26551223 * L - 1.0));
        const float r = t * __builtin_amdgcn_exp2f(fmaf(-0.5f * kLog2e * z, z, p));
        // (the bound keeps infinity times 0 out of gelu(infinity))
        return fmaf(-fminf(fabsf(z), 3e38f), r, fmaxf(z, 0.0f));
    }
    // z / (1 + e^-z): e^-z overflows to infinity for z < -88, where the quotient is 0, its limit
    if constexpr (ACT == kActSilu) return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
    return z;
}
// gelu'(z) = Phi(z) + z phi(z),  silu'(z) = s (1 + z (1 - s)), s = 1 / (1 + e^-z).
// Phi here by Abramowitz and Stegun 7.1.26 (absolute error of erf below
// 1.5e-7, all a slope near 1 needs; the coefficients halved), which shares its
// exponential with phi.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == kActGelu) {
        const float e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z);
        const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f * 0.707106781186547524f, fabsf(z), 1.0f));
        float p = 0.5f * 1.061405429f;
        p = fmaf(p, t, 0.5f * -1.453152027f);
        p = fmaf(p, t, 0.5f * 1.421413741f);
        p = fmaf(p, t, 0.5f * -0.284496736f);
        p = fmaf(p, t, 0.5f * 0.254829592f);
        const float r = p * t * e;
        return fmaf(z * 0.398942280401432678f, e, z >= 0.0f ? 1.0f - r : r);
    }
    if constexpr (ACT == kActSilu) {
        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    return 1.0f;
}

// ---- sums over lanes and blocks ---------------------------------------------------
// Adding across a wave takes one or two vector instructions a step: data
// moved within rows of 16 lanes by DPP, across them by the lane swaps (a
// shuffle through LDS costs ten times that, which small calls feel).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
constexpr int kDppXor1 = 0xb1, kDppXor2 = 0x4e, kDppHalfMirror = 0x141, kDppMirror = 0x140;

// v plus the value of the lane 16 or 32 away: the swap exchanges the odd rows
// (halves) of one register with the even ones of the other.  The results are
// copied out before they are read as floats: a bit cast of a vector's element
// itself reads the first one.
template <int N>
__device__ __forceinline__ float swap_add(float v) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    uint32_t x, y;
    if constexpr (N == 16) {
        const auto q = __builtin_amdgcn_permlane16_swap(a, a, false, false);
        x = q[0];
        y = q[1];
    } else {
        const auto q = __builtin_amdgcn_permlane32_swap(a, a, false, false);
        x = q[0];
        y = q[1];
    }
    return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}

// Sum over the lanes of each aligned team of `parts` (a power of two, at most
// 64, the same in every lane), in every lane.
__device__ __forceinline__ float team_sum(float v, int parts) {
    if (parts > 1) v += dpp<kDppXor1>(v);
    if (parts > 2) v += dpp<kDppXor2>(v);
    if (parts > 4) v += dpp<kDppHalfMirror>(v);      // lanes of a quad hold the same value by now
    if (parts > 8) v += dpp<kDppMirror>(v);
    if (parts > 16) v = swap_add<16>(v);
    if (parts > 32) v = swap_add<32>(v);
    return v;
}
__device__ __forceinline__ float wave_sum(float v) { return team_sum(v, 64); }
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}
// Sum over a block of whole waves (at most 16); `red` holds 16 values and may
// be reused after the next barrier.  Every thread gets the sum.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* red) {
    v = wave_sum(v);
    const int nw = blockDim.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    T s = red[0];
    for (int i = 1; i < nw; ++i) s += red[i];
    return s;
}

// Quotient by a small divisor without a division: exact for n d < 2^32.
struct FastDiv {
    uint32_t d, m, one;       // one: all bits where d is 1
};
inline FastDiv fast_div(int d) {
    return d == 1 ? FastDiv{1, 0, ~0u} : FastDiv{(uint32_t)d, (uint32_t)((1ull << 32) / d + 1), 0};
}
__device__ __forceinline__ int div_by(int n, const FastDiv& f) {
    return (int)(__umulhi((uint32_t)n, f.m) + ((uint32_t)n & f.one));
}
__device__ __forceinline__ int mod_by(int n, const FastDiv& f) { return n - div_by(n, f) * (int)f.d; }

}  // namespace fno
