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
// gelu(z) = z Phi(z), Phi(z) = erfc(-z / sqrt 2) / 2 by the fit of epi_erfc
// with the device's reciprocal (1 ulp) in place of a division: 21 vector
// instructions against 30, which counts where a 16-bit field is read and
// written at the memory's rate.  Slopes:
//   gelu'(z) = Phi(z) + z phi(z),  silu'(z) = s (1 + z (1 - s)), s = sigmoid(z).
// sigmoid(z) = 1 / (1 + e^-z): e^-z overflows to infinity for z < -88, where
// the quotient is 0, its limit.
__device__ __forceinline__ float phi_cdf(float z) {
    const float a = 0.707106781186547524f * fabsf(z);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.5f, a, 1.0f));
    float p = 0.17087277f;
    p = fmaf(p, t, -0.82215223f);
    p = fmaf(p, t, 1.48851587f);
    p = fmaf(p, t, -1.13520398f);
    p = fmaf(p, t, 0.27886807f);
    p = fmaf(p, t, -0.18628806f);
    p = fmaf(p, t, 0.09678418f);
    p = fmaf(p, t, 0.37409196f);
    p = fmaf(p, t, 1.00002368f);
    p = fmaf(p, t, -1.26551223f);
    const float r = 0.5f * t * __expf(fmaf(-a, a, p));    // Phi(-|z|)
    return z >= 0.0f ? 1.0f - r : r;
}
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == kActGelu) return z * phi_cdf(z);
    if constexpr (ACT == kActSilu) return z * sigmoid(z);
    return z;
}
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == kActGelu) return fmaf(z, 0.398942280401432678f * __expf(-0.5f * z * z), phi_cdf(z));
    if constexpr (ACT == kActSilu) {
        const float s = sigmoid(z);
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    return 1.0f;
}

// ---- block sums -----------------------------------------------------------------
// Sum over a wave in a fixed order, the same value in every lane.
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
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

}  // namespace fno
