// Global norm of many gradients, and clipping by it:
//   norm = (sum_t sum_i |g_ti|^2)^1/2,  g' = g min(1, max_norm / (norm + 1e-6)).
//
// The tensors are handed to each launch as a table in its kernel arguments
// (kGradTable tensors a launch), cut into chunks of 16 KiB.  Squares are
// summed in double: the square of a float neither overflows nor vanishes
// there, and the norm of 10^9 values is as good as its inputs.
#include <algorithm>

#include "fno_fields.hpp"

namespace fno {
namespace {

constexpr int kThreads = 256;
constexpr int kChunkBytes = 16384;
constexpr int kPartBlocks = 2048;     // partial sums a launch leaves

__device__ __forceinline__ int64_t chunk_elems(int type) {
    return kChunkBytes / (type == kTypeBf16 || type == kTypeF16 ? 2 : 4);
}

// Tensor that holds a chunk: the last whose first chunk is not beyond it
// (empty tensors own no chunk and share their successor's first).
__device__ __forceinline__ int tensor_of(const GradTable& t, uint32_t chunk) {
    static_assert(kGradTable == 128, "two entries a lane");
    const int lane = threadIdx.x & 63;
    const uint64_t lo = __ballot(t.first[lane] <= chunk);
    const uint64_t hi = __ballot(t.first[lane + 64] <= chunk);
    return __builtin_amdgcn_readfirstlane(__popcll(lo) + __popcll(hi) - 1);
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

template <typename T>
__device__ __forceinline__ double sum_squares(const T* __restrict__ p, int64_t n, int t, int threads) {
    constexpr int V = 16 / sizeof(T);
    double s = 0.0;
    const int64_t nv = n / V;
    int64_t i = t;
    for (; i + 3 * threads < nv; i += 4 * threads) {          // four loads in flight: 16 KiB a workgroup
        float v[4][V];
#pragma unroll
        for (int k = 0; k < 4; ++k) load_vec<V>(p + (i + k * threads) * V, v[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) s = fma((double)v[k][j], (double)v[k][j], s);
    }
    for (; i < nv; i += threads) {
        float v[V];
        load_vec<V>(p + i * V, v);
#pragma unroll
        for (int j = 0; j < V; ++j) s = fma((double)v[j], (double)v[j], s);
    }
    for (i = nv * V + t; i < n; i += threads) s = fma((double)(float)p[i], (double)(float)p[i], s);
    return s;
}

template <typename T>
__device__ __forceinline__ void scale_by(const T* p, T* q, int64_t n, float coef, int t, int threads) {
    constexpr int V = 16 / sizeof(T);
    const int64_t nv = n / V;
    for (int64_t i = t; i < nv; i += threads) {
        float v[V];
        load_vec<V>(p + i * V, v);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= coef;
        store_vec<V>(q + i * V, v);
    }
    for (int64_t i = nv * V + t; i < n; i += threads) q[i] = (T)((float)p[i] * coef);
}

// part[blockIdx.x] = sum of squares of this block's chunks.  268 MB in 46 us (5.8
// TB/s); 56 with 1024 workgroups and no loads batched.  Memory bounds it.
__global__ __launch_bounds__(kThreads) void k_grad_sumsq(GradTable t, uint32_t nchunks, double* __restrict__ part) {
    __shared__ double red[16];
    double s = 0.0;
    for (uint32_t c = blockIdx.x; c < nchunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const int64_t ce = chunk_elems(t.type[i]), at = (int64_t)(c - t.first[i]) * ce;
        const int64_t n = min(ce, t.n[i] - at);
        with_type(t.type[i], [&](auto e) {
            s += sum_squares(static_cast<const decltype(e)*>(t.src[i]) + at, n, threadIdx.x, kThreads);
        });
    }
    s = block_sum(s, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// min(1, max_norm / (norm + 1e-6)); a NaN norm gives NaN.
__device__ __forceinline__ float clip_coef(double norm, float max_norm) {
    const double c = (double)max_norm / (norm + 1e-6);
    return c > 1.0 ? 1.0f : (float)c;
}

// One block: the norm from the partial sums (or as given), and the factor.  4.7 to 5.0
// us, a launch and the latency of the sums: workgroups that leave them to the
// last of them would need a counter that someone clears.
__global__ __launch_bounds__(kThreads) void k_grad_finish(const double* __restrict__ part, int nparts,
                                                          const float* __restrict__ given, float max_norm,
                                                          float* __restrict__ norm, float* __restrict__ coef) {
    __shared__ double red[16];
    double s = 0.0;
    for (int i = threadIdx.x; i < nparts; i += kThreads) s += part[i];
    s = block_sum(s, red);
    if (threadIdx.x == 0) {
        const double v = given ? (double)*given : sqrt(s);
        if (norm) *norm = (float)v;
        if (coef) *coef = clip_coef(v, max_norm);
    }
}

// At most kGradSmallChunks chunks: everything in one workgroup, a wave a chunk.
// The second read comes from the caches.  11 tensors of 17 KB: 7 to 8 us, latency.
__global__ __launch_bounds__(1024) void k_grad_small(GradTable t, uint32_t nchunks, float max_norm, bool scale,
                                                     float* __restrict__ norm) {
    __shared__ double red[16];
    const uint32_t wave = threadIdx.x >> 6;
    const int lane = threadIdx.x & 63;
    double s = 0.0;
    for (uint32_t c = wave; c < nchunks; c += 16) {
        const int i = tensor_of(t, c);
        const int64_t ce = chunk_elems(t.type[i]), at = (int64_t)(c - t.first[i]) * ce;
        const int64_t n = min(ce, t.n[i] - at);
        with_type(t.type[i], [&](auto e) {
            s += sum_squares(static_cast<const decltype(e)*>(t.src[i]) + at, n, lane, 64);
        });
    }
    const double v = sqrt(block_sum(s, red));
    if (threadIdx.x == 0) *norm = (float)v;
    if (!scale) return;
    const float k = clip_coef(v, max_norm);
    for (uint32_t c = wave; c < nchunks; c += 16) {
        const int i = tensor_of(t, c);
        if (k == 1.0f && t.src[i] == t.dst[i]) continue;
        const int64_t ce = chunk_elems(t.type[i]), at = (int64_t)(c - t.first[i]) * ce;
        const int64_t n = min(ce, t.n[i] - at);
        with_type(t.type[i], [&](auto e) {
            scale_by(static_cast<const decltype(e)*>(t.src[i]) + at, static_cast<decltype(e)*>(t.dst[i]) + at, n, k,
                     lane, 64);
        });
    }
}

// One chunk a block.  A tensor clipped in place by a factor of 1 is left as
// it is: every value times 1 is itself.  537 MB moved in 78 us (6.9 TB/s, part
// of the gradients still in the memory-side cache).
__global__ __launch_bounds__(kThreads) void k_grad_scale(GradTable t, uint32_t nchunks, const float* __restrict__ coef) {
    const float k = *coef;
    for (uint32_t c = blockIdx.x; c < nchunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        if (k == 1.0f && t.src[i] == t.dst[i]) continue;
        const int64_t ce = chunk_elems(t.type[i]), at = (int64_t)(c - t.first[i]) * ce;
        const int64_t n = min(ce, t.n[i] - at);
        with_type(t.type[i], [&](auto e) {
            scale_by(static_cast<const decltype(e)*>(t.src[i]) + at, static_cast<decltype(e)*>(t.dst[i]) + at, n, k,
                     threadIdx.x, kThreads);
        });
    }
}

}  // namespace

uint32_t grad_table_chunks(GradTable& t, int count) {
    uint64_t c = 0;
    for (int i = 0; i < kGradTable; ++i) {
        t.first[i] = i < count ? (uint32_t)c : UINT32_MAX;
        if (i >= count) continue;
        const int64_t ce = kChunkBytes / (t.type[i] == kTypeBf16 || t.type[i] == kTypeF16 ? 2 : 4);
        c += (uint64_t)((t.n[i] + ce - 1) / ce);
    }
    return (uint32_t)c;
}

int grad_sumsq_blocks(uint32_t nchunks) { return (int)std::min<uint32_t>(nchunks, kPartBlocks); }

size_t grad_norm_workspace(int64_t count) {
    const size_t launches = (size_t)(count + kGradTable - 1) / kGradTable;
    return 256 + launches * kPartBlocks * sizeof(double);
}

hipError_t launch_grad_sumsq(const GradTable& t, uint32_t nchunks, double* part, hipStream_t s) {
    return launch_kernel(k_grad_sumsq, dim3(grad_sumsq_blocks(nchunks)), dim3(kThreads), 0, s, t, nchunks, part);
}
hipError_t launch_grad_small(const GradTable& t, uint32_t nchunks, float max_norm, bool scale, float* norm,
                             hipStream_t s) {
    return launch_kernel(k_grad_small, dim3(1), dim3(1024), 0, s, t, nchunks, max_norm, scale, norm);
}
hipError_t launch_grad_finish(const double* part, int nparts, const float* given, float max_norm, float* norm,
                              float* coef, hipStream_t s) {
    return launch_kernel(k_grad_finish, dim3(1), dim3(kThreads), 0, s, part, nparts, given, max_norm, norm, coef);
}
hipError_t launch_grad_scale(const GradTable& t, uint32_t nchunks, const float* coef, hipStream_t s) {
    // one chunk a workgroup (a dimension of the grid holds fewer than 2^32 threads)
    return launch_kernel(k_grad_scale, dim3(std::min<uint32_t>(nchunks, 1u << 22)), dim3(kThreads), 0, s, t, nchunks,
                         coef);
}

}  // namespace fno
