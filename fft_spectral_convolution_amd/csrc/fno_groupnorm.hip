// Group norm with an activation:
//   mean = sum x / n,  var = sum (x - mean)^2 / n,  rstd = (var + eps)^-1/2
//   out = act((x - mean) rstd w_c + b_c)
// over the n = P D values of a group (D = C / groups channels of all P
// positions).
//
// A group that fits a workgroup's registers is read once (k_gn_fused_*): mean,
// then the squares about it, then the output from the kept values.  A larger
// one is read twice: k_gn_stats_* leaves (mean, sum of squares about it) of
// each chunk, k_gn_finish joins them (Chan, Golub and LeVeque's pairwise
// update, all chunks at once), and k_gn_apply_* writes the output.
#include "fno_groupnorm.hpp"

namespace fno {
namespace {

// Vectors a thread keeps in the one-workgroup kernels: 32 values.  (Of a
// 16-bit field twice as many would fit, but a vector of eight has eight
// channels' constants beside it, which then spill.)
template <typename TX>
constexpr int kHeld = 32 / kVec<TX>;
constexpr int64_t kFusedValues = 1024 * 32;
constexpr int kFusedThreads = 1024;

// ---- one pass, channels last -----------------------------------------------------
// Workgroup (item, slice of cs channels), values in registers: read once, the
// mean before the squares.  256 items of 32 channels x 1024, float32: 20 us
// (67 MB, 3.3 TB/s); memory, and two sums through LDS a workgroup.
template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kFusedThreads) void k_gn_fused_last(const TX* __restrict__ x,
                                                                const float* __restrict__ w,
                                                                const float* __restrict__ bias,
                                                                TY* __restrict__ out, float* __restrict__ stats,
                                                                LastRows r, int slices, int64_t blocks, float eps) {
    constexpr int V = kVec<TX>, kHold = kHeld<TX>;
    extern __shared__ float lds[];
    const int64_t id = block_id();
    if (id >= blocks) return;
    float* buf = lds;
    float* mean = lds + r.threads * V;
    const int groups = div_by(r.cs, r.by_D);
    float* rstd = mean + groups;
    const int64_t b = id / slices;
    const int c0 = (int)(id % slices) * r.cs;
    const int t = threadIdx.x, row = div_by(t, r.by_cv), slot = t - row * r.cv;
    const bool on = row < r.q;
    const int64_t base = b * r.P * r.C + c0 + slot * V;
    const float n_group = (float)r.P * (float)r.D, inv_n = 1.0f / n_group;

    Raw<TX, V> held[kHold];
    float sum[V] = {};
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int s = row + i * r.q;
        held[i].load(x + base + (int64_t)s * r.stride(), on ? last_valid<V>(r, s, slot) : 0);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += held[i][j];
    float m[V], a[V], o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = c0 + mod_by(slot * V + j, r.by_cs);
        a[j] = or_one(w, c);
        o[j] = or_zero(bias, c);
    }
    last_sums(sum, buf, mean, r, r.D);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        m[j] = mean[div_by(mod_by(slot * V + j, r.by_cs), r.by_D)] / n_group;
        sum[j] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int n = on ? last_valid<V>(r, row + i * r.q, slot) : 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float d = held[i][j] - m[j];
            sum[j] = fmaf(j < n ? d : 0.0f, d, sum[j]);
        }
    }
    last_sums(sum, buf, rstd, r, r.D);
    for (int g = t; g < groups; g += blockDim.x) {
        float* st = stats + 2 * (b * (div_by(r.C, r.by_D)) + div_by(c0, r.by_D) + g);
        st[0] = mean[g] / n_group;
        st[1] = rsqrtf(fmaf(rstd[g], inv_n, eps));
    }
    if (!on) return;
#pragma unroll
    for (int j = 0; j < V; ++j)
        a[j] *= rsqrtf(fmaf(rstd[div_by(mod_by(slot * V + j, r.by_cs), r.by_D)], inv_n, eps));
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int s = row + i * r.q, n = last_valid<V>(r, s, slot);
        if (n == 0) break;
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = act_value<ACT>(fmaf(held[i][j] - m[j], a[j], o[j]));
        store_part(out + base + (int64_t)s * r.stride(), n, y);
    }
}

// ---- one pass, channels first ------------------------------------------------------
// Workgroup (item, group): D rows of P values, one run of memory, read once.
// 1024 groups of 32768 values, float32: 58 to 60 us, 4.5 to 4.6 TB/s where a copy has 5.1.
template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kFusedThreads) void k_gn_fused_first(const TX* __restrict__ x,
                                                                 const float* __restrict__ w,
                                                                 const float* __restrict__ bias,
                                                                 TY* __restrict__ out, float* __restrict__ stats,
                                                                 int D, int P, int groups, FastDiv by_p, int64_t blocks,
                                                                 float eps) {
    constexpr int V = kVec<TX>, kHold = kHeld<TX>;
    __shared__ float red[16];
    const int64_t id = block_id();
    if (id >= blocks) return;
    const int n = D * P, t = threadIdx.x, step = blockDim.x * V;
    const int c0 = (int)(id % groups) * D;
    const int64_t base = id * n;
    const float inv_n = 1.0f / (float)n;

    Raw<TX, V> held[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int e = i * step + t * V;
        held[i].load(x + base + e, max(0, min(V, n - e)));
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kHold; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) sum += held[i][j];
    const float mean = block_sum(sum, red) / (float)n;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int left = n - (i * step + t * V);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float d = held[i][j] - mean;
            sum = fmaf(j < left ? d : 0.0f, d, sum);
        }
    }
    const float rstd = rsqrtf(fmaf(block_sum(sum, red), inv_n, eps));
    if (t == 0) {
        stats[2 * id] = mean;
        stats[2 * id + 1] = rstd;
    }
    const bool whole = P % V == 0;        // a vector lies in one channel
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int e = i * step + t * V, left = n - e;
        if (left <= 0) break;
        float y[V];
        int c = c0 + div_by(e, by_p);
        float a = rstd * or_one(w, c), o = or_zero(bias, c);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (!whole && j && j < left) {
                c = c0 + div_by(e + j, by_p);
                a = rstd * or_one(w, c);
                o = or_zero(bias, c);
            }
            y[j] = act_value<ACT>(fmaf(held[i][j] - mean, a, o));
        }
        store_part(out + base + e, min(V, left), y);
    }
}

// ---- statistics of chunks ------------------------------------------------------------
// A thread sums its values less the first of them, and their squares: what
// is subtracted lies within the spread of the thread's own values, so the
// squares lose nothing to a level far from zero.
struct Running {
    float pivot, s, q;
    __device__ __forceinline__ void add(float v) {
        const float d = v - pivot;
        s += d;
        q = fmaf(d, d, q);
    }
    __device__ __forceinline__ float mean(float n) const { return pivot + s / n; }
    // (one rounding: where q has passed float32's range, it stays infinite instead of infinity less infinity)
    __device__ __forceinline__ float squares(float n) const { return fmaxf(fmaf(-s, s / n, q), 0.0f); }
};

// The first of two reads, bound by memory: 537 MB in 95 us (5.6 TB/s).
// Workgroup (item, chunk of `per` super-rows); part[(b chunks + chunk) groups + g].
template <typename TX>
__global__ __launch_bounds__(kMaxSlots) void k_gn_stats_last(const TX* __restrict__ x, float2* __restrict__ part,
                                                             LastRows r, int per, int chunks, int64_t blocks) {
    constexpr int V = kVec<TX>;
    extern __shared__ float lds[];
    const int64_t id = block_id();
    if (id >= blocks) return;
    float* buf = lds;
    float* mean = lds + r.threads * V;
    const int groups = div_by(r.C, r.by_D);
    float* sq = mean + groups;
    const int64_t b = id / chunks;
    const int first = (int)(id % chunks) * per, last = min(first + per, r.ns);
    const int t = threadIdx.x, row = div_by(t, r.by_cv), slot = t - row * r.cv;
    const bool on = row < r.q;
    const TX* p = x + b * r.P * r.C + slot * V;
    // positions of this chunk
    const float n = (float)min((int64_t)per * r.R, r.P - (int64_t)first * r.R) * (float)r.D;

    Running run[V] = {};
    float cnt = 0.0f;
    int s = first + row;
    const int full = min(last, r.P / r.R);
    if (on && s < full) {
        // eight loads on their way at once; those past the end repeat the last and are not counted
        bool fresh = true;
        for (; s < full; s += 8 * r.q) {
            Raw<TX, V> u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                u[i].load(p + (int64_t)(s + i * r.q < full ? s + i * r.q : s) * r.stride(), V);
            if (fresh) {
#pragma unroll
                for (int j = 0; j < V; ++j) run[j].pivot = u[0][j];
                fresh = false;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (s + i * r.q < full) {
#pragma unroll
                    for (int j = 0; j < V; ++j) run[j].add(u[i][j]);
                    cnt += 1.0f;
                }
        }
        // where the loop would have gone next
        s = first + row + (full - 1 - first - row) / r.q * r.q + r.q;
    }
    // the incomplete super-row: values that some of the vector's places lack
    float num[V];
    const int tail = on && s < last && s >= full ? last_valid<V>(r, s, slot) : 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        num[j] = cnt;
        if (j < tail) {
            const float v = (float)p[(int64_t)s * r.stride() + j];
            if (cnt == 0.0f) run[j] = Running{v, 0.0f, 0.0f};
            else run[j].add(v);
            num[j] += 1.0f;
        }
    }
    float val[V];
#pragma unroll
    for (int j = 0; j < V; ++j) val[j] = num[j] > 0.0f ? num[j] * run[j].mean(num[j]) : 0.0f;
    last_sums(val, buf, mean, r, r.D);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float d = num[j] > 0.0f ? run[j].mean(num[j]) - mean[div_by(mod_by(slot * V + j, r.by_cs), r.by_D)] / n : 0.0f;
        val[j] = num[j] > 0.0f ? fmaf(num[j] * d, d, run[j].squares(num[j])) : 0.0f;
    }
    last_sums(val, buf, sq, r, r.D);
    for (int g = t; g < groups; g += blockDim.x) part[id * groups + g] = make_float2(mean[g] / n, sq[g]);
}

// Bound by memory: 537 MB in 89 us (6.0 TB/s).
// Workgroup (group's run of memory, chunk of `per` values); part[run chunks + chunk].
template <typename TX>
__global__ __launch_bounds__(kGnThreads) void k_gn_stats_first(const TX* __restrict__ x, float2* __restrict__ part,
                                                               int64_t run_len, int per, int chunks, int64_t blocks) {
    constexpr int V = kVec<TX>;
    __shared__ float red[16];
    const int64_t id = block_id();
    if (id >= blocks) return;
    const int64_t run_id = id / chunks, at = (id % chunks) * per;
    const int n = (int)min((int64_t)per, run_len - at);
    const TX* p = x + run_id * run_len + at;
    constexpr int kStep = kGnThreads * V;
    const int t = threadIdx.x, full = n / kStep * kStep;
    Running run{};
    float cnt = 0.0f;
    if (t < n) run.pivot = (float)p[min(t * V, n - 1)];
    int e = t * V;
    for (; e + 3 * kStep < full; e += 4 * kStep) {
        float u[4][V];
#pragma unroll
        for (int i = 0; i < 4; ++i) load_vec<V>(p + e + i * kStep, u[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) run.add(u[i][j]);
        cnt += 4.0f * V;
    }
    for (; e < n; e += kStep) {
        float u[V];
        const int m = min(V, n - e);
        load_part<V>(p + e, m, u);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < m) run.add(u[j]);
        cnt += (float)m;
    }
    const float mine = cnt > 0.0f ? run.mean(cnt) : 0.0f;
    const float mean = block_sum(cnt * mine, red) / (float)n;
    const float d = mine - mean;
    const float sq = block_sum(cnt > 0.0f ? fmaf(cnt * d, d, run.squares(cnt)) : 0.0f, red);
    if (t == 0) part[id] = make_float2(mean, sq);
}

// One workgroup a group: joins its chunks' statistics.  Chunk i of group (b, g)
// is part[(b G + g) chunks + i] (channels first) or part[(b chunks + i) G + g];
// all chunks hold `per` values but the last.  A thread asks for eight pairs at
// a time (they come from far away) and keeps the first eight for the squares:
// latency bounds it, 5 us for 8 groups of 1024 chunks.
__global__ __launch_bounds__(kGnThreads) void k_gn_finish(const float2* __restrict__ part, float* __restrict__ stats,
                                                          int64_t total, int groups, int chunks, bool last, int64_t per,
                                                          int64_t n, float eps) {
    __shared__ float red[16];
    const int64_t i = block_id();
    if (i >= total) return;
    const float2* p = part + (last ? i / groups * chunks * groups + i % groups : i * chunks);
    const int step = last ? groups : 1;
    const auto load = [&](int k0, float2(&q)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int k = k0 + e * kGnThreads;
            q[e] = k < chunks ? p[(int64_t)k * step] : make_float2(0.0f, 0.0f);
        }
    };
    const auto values = [&](int k) { return k < chunks ? (float)min(per, n - k * per) : 0.0f; };
    const auto sums = [&](int k0, const float2(&q)[8]) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(values(k0 + e * kGnThreads), q[e].x, s);
        return s;
    };
    const int t = threadIdx.x;
    float2 q[8], far[8];
    load(t, q);
    float sum = sums(t, q);
    for (int k = t + 8 * kGnThreads; k < chunks; k += 8 * kGnThreads) {
        load(k, far);
        sum += sums(k, far);
    }
    const float mean = block_sum(sum, red) / (float)n;
    const auto squares = [&](int k0, const float2(&v)[8]) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = v[e].x - mean;
            s += fmaf(values(k0 + e * kGnThreads) * d, d, v[e].y);
        }
        return s;
    };
    float sq = squares(t, q);
    for (int k = t + 8 * kGnThreads; k < chunks; k += 8 * kGnThreads) {
        load(k, far);
        sq += squares(k, far);
    }
    sq = block_sum(sq, red);
    if (t == 0) {
        stats[2 * i] = mean;
        stats[2 * i + 1] = rsqrtf(sq / (float)n + eps);
    }
}

// ---- one pass, items spread over workgroups ----------------------------------------------
// Workgroup (item, chunk of q NV super-rows).  Vectors are whole (P is a
// multiple of R); rows past the end of an item are read as the thread's last
// one and left out.
constexpr int kOnceVectors = 16;      // of a thread, at most
template <typename TX, typename TY>
struct OnceArgs {
    const TX* x;
    const float *w, *bias;
    TY* out;
    float* stats;
    uint64_t* slots;
    LastRows r;
    Once o;
    float eps;
    int spin;
};

template <int ACT, int NV, bool TURN, typename TX, typename TY>
struct OnceLast {
    static constexpr int V = kVec<TX>;
    // TURN: out is channels first; kTurn vectors a thread go through LDS at a time, so that a channel's run in out is
    // kTurn q positions long
    static constexpr int kTurn = NV < 4 ? NV : 4;
    typedef typename VecOf<TX, V>::type Vec;
    const OnceArgs<TX, TY>& a;
    const LastRows& r;
    float *buf, *counts, *mean, *sq;
    int* missing;
    int t, row, slot, groups, chunk;
    int64_t item, step;
    float w[V], b[V];

    // The constants of the thread's channels.  Four each are asked for long before `write` uses them; eight would cost
    // registers that hold the field (they spill: 60 us instead of 48 for the 128 x 128 field in 16 bits).
    static constexpr bool kEarly = V <= 4;
    __device__ __forceinline__ void constants() {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = mod_by(slot * V + j, r.by_cs);
            w[j] = or_one(a.w, c);
            b[j] = or_zero(a.bias, c);
        }
    }
    __device__ __forceinline__ OnceLast(const OnceArgs<TX, TY>& args, float* lds, int* flag)
        : a(args), r(args.r), buf(lds), missing(flag) {
        t = threadIdx.x;
        row = div_by(t, r.by_cv);
        slot = t - row * r.cv;
        groups = div_by(r.C, r.by_D);
        counts = lds + once_buffer(r.threads, V, r.C, TURN ? kTurn : 0, r.q * r.R);
        mean = counts + r.q;
        sq = mean + groups;
        item = blockIdx.x / a.o.chunks;
        chunk = (int)(blockIdx.x - item * a.o.chunks);
        step = (int64_t)r.q * r.stride();
    }
    __device__ __forceinline__ int per() const { return r.q * NV; }
    __device__ __forceinline__ const TX* x_item() const { return a.x + item * r.P * r.C; }
    __device__ __forceinline__ uint64_t* pairs() const { return a.slots + item * groups * a.o.chunks; }
    __device__ __forceinline__ float values_of(int k) const {
        return (float)min(per(), r.ns - k * per()) * (float)(r.R * r.D);
    }
    // rows of chunk k that this thread holds, and the element of the first
    __device__ __forceinline__ int rows_of(int k) const {
        return row < r.q ? max(0, min(NV, (r.ns - (k * per() + row) + r.q - 1) / r.q)) : 0;
    }
    __device__ __forceinline__ int64_t at_of(int k) const { return (int64_t)(k * per() + row) * r.stride() + slot * V; }
    // Chunk k's mean and squares about it, of each group, to its slots.  `rows` vectors that `each` hands over one
    // by one (twice): every thread leaves its own mean and squares in LDS; after one barrier a team of lanes joins a
    // group's (their mean first, then the squares about that).
    template <typename F>
    __device__ __forceinline__ void put(int k, int rows, F&& each) const {
        float m[V], q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) m[j] = 0.0f;
        each([&](const Vec& h) {
#pragma unroll
            for (int j = 0; j < V; ++j) m[j] += (float)h[j];
        });
        const float inv_rows = rows ? __builtin_amdgcn_rcpf((float)rows) : 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            // the quotient to the last bit or so: the reciprocal's error is put right once
            const float sum = m[j];
            m[j] = sum * inv_rows;
            m[j] = fmaf(fmaf(-(float)rows, m[j], sum), inv_rows, m[j]);
            q[j] = 0.0f;
        }
        each([&](const Vec& h) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = (float)h[j] - m[j];
                q[j] = fmaf(d, d, q[j]);
            }
        });
        __syncthreads();
        float* means = buf;
        float* squares = buf + r.threads * V;
        if (row < r.q) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                means[t * V + j] = m[j];
                squares[t * V + j] = q[j];
            }
            if (slot == 0) counts[row] = (float)rows;
        }
        __syncthreads();
        const int parts = a.o.parts, part = t & (parts - 1), g = t >> __builtin_ctz(parts);
        if (g < groups) {
            const int entries = r.q * r.R * r.D;
            float sum = 0.0f;
            for (int e = part; e < entries; e += parts) {
                const int i = div_by(e, r.by_D);
                sum = fmaf(counts[div_by(i, r.by_R)], means[i * (r.C - r.D) + g * r.D + e], sum);
            }
            const float mu = team_sum(sum, parts) / values_of(k);
            sum = 0.0f;
            for (int e = part; e < entries; e += parts) {
                const int i = div_by(e, r.by_D), at = i * (r.C - r.D) + g * r.D + e;
                const float d = means[at] - mu;
                sum += fmaf(counts[div_by(i, r.by_R)] * d, d, squares[at]);
            }
            sum = team_sum(sum, parts);
            if (part == 0) put_pair(pairs() + g * a.o.chunks + k, mu, sum);
        }
    }
    // mean and 1 / deviation of the item's groups, in LDS, from all its chunks; the first chunk not there, or `chunks`
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
            const float n = (float)r.P * (float)r.D;
            const float whole = values_of(0), rest = values_of(chunks - 1);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kLooks; ++i) {
                if (i * parts >= chunks) break;
                const int k = part + i * parts;
                const float m = k + 1 < chunks ? whole : rest;
                if (k < chunks) sum = fmaf(m, unpack_pair(v[i]).x, sum);
            }
            const float mu = team_sum(sum, parts) / n;
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kLooks; ++i) {
                if (i * parts >= chunks) break;
                const int k = part + i * parts;
                const float2 q = unpack_pair(v[i]);
                const float m = k + 1 < chunks ? whole : rest;
                if (k < chunks) sum += fmaf(m * (q.x - mu), q.x - mu, q.y);
            }
            sum = team_sum(sum, parts);
            if (part == 0) {
                mean[g] = mu;
                sq[g] = rsqrtf(sum / n + a.eps);
            }
        }
        __syncthreads();
        return *missing;
    }
    // The output of this workgroup's chunk from its vectors: get(i) is vector i < rows.
    template <typename F>
    __device__ __forceinline__ void write(int64_t at, int rows, F&& get) {
        if constexpr (!kEarly) constants();
        if (chunk == 0)
            for (int i = t; i < groups; i += blockDim.x) {
                a.stats[2 * (item * groups + i)] = mean[i];
                a.stats[2 * (item * groups + i) + 1] = sq[i];
            }
        float m[V], k[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int g = div_by(mod_by(slot * V + j, r.by_cs), r.by_D);
            m[j] = mean[g];
            k[j] = sq[g] * w[j];
        }
        if constexpr (!TURN) {
            TY* y = a.out + item * r.P * r.C + at;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < rows) {
                    const Vec h = get(i);
                    float u[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) u[j] = act_value<ACT>(fmaf((float)h[j] - m[j], k[j], b[j]));
                    store_vec<V>(y + i * step, u);
                }
        } else {
            constexpr int VY = kVec<TY>;
            const int span = kTurn * r.q * r.R, ld = span + 1;       // positions in LDS at a time
            int place[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = slot * V + j, ch = mod_by(e, r.by_cs);
                place[j] = ch * ld + div_by(e, r.by_cs) + row * r.R;
            }
            TY* y = a.out + item * r.P * r.C;
#pragma unroll
            for (int i0 = 0; i0 < NV; i0 += kTurn) {
                const int p0 = (chunk * per() + i0 * r.q) * r.R, np = min(span, r.P - p0);
                if (np <= 0) break;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kTurn; ++i)
                    if (i0 + i < rows) {
                        const Vec h = get(i0 + i);
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            buf[place[j] + i * r.q * r.R] = act_value<ACT>(fmaf((float)h[j] - m[j], k[j], b[j]));
                    }
                __syncthreads();
                const int runs = (np + VY - 1) / VY;                 // vectors of a channel
                const FastDiv by_runs{(uint32_t)runs, runs == 1 ? 0u : 0xffffffffu / (uint32_t)runs + 1u, runs == 1 ? ~0u : 0u};
#pragma unroll 4
                for (int e = t; e < r.C * runs; e += blockDim.x) {
                    const int ch = div_by(e, by_runs), p = (e - ch * runs) * VY;
                    float u[VY];
#pragma unroll
                    for (int j = 0; j < VY; ++j) u[j] = buf[ch * ld + p + j];
                    store_part(y + (int64_t)ch * r.P + p0 + p, min(VY, np - p), u);
                }
            }
        }
    }
};

// Where others' sums stayed out: their chunks from memory, in the same order,
// then this workgroup's own again.  A call, so that the kernel's own registers
// are not allotted around it; its frame costs every lane 200 to 290 bytes of
// scratch, touched only here.
template <int ACT, int NV, bool TURN, typename TX, typename TY>
__device__ __attribute__((noinline)) void once_late(OnceArgs<TX, TY> args, float* lds, int* flag, int lost) {
    typedef OnceLast<ACT, NV, TURN, TX, TY> F;
    F f(args, lds, flag);
    if constexpr (F::kEarly) f.constants();
    do {
        const TX* p = f.x_item() + f.at_of(lost);
        const int n = f.rows_of(lost);
        f.put(lost, n, [&](auto&& take) {
#pragma unroll 1
            for (int i = 0; i < n; ++i) take(*reinterpret_cast<const typename F::Vec*>(p + i * f.step));
        });
        lost = f.join(0);
    } while (lost < args.o.chunks);
    const int64_t at = f.at_of(f.chunk);
    f.write(at, f.rows_of(f.chunk),
            [&](int i) { return *reinterpret_cast<const typename F::Vec*>(f.x_item() + at + i * f.step); });
}

// Four waves a SIMD, each with 16 vectors a thread in its registers: 65 us for
// the 128 x 128 field (32 x 64 channels, float32) where 8 vectors took 83; 62
// with the channels' constants asked for before the join; the kernel alone now
// takes 58 (268 MB, 4.6 TB/s), with 4 to 6 of its 128 registers spilled, and 46 to
// 47 from bfloat16 to a channels-first float32 field (4.3 TB/s).  Memory bounds it, and that a workgroup loads, joins and
// stores in turn.
template <int ACT, int NV, bool TURN, typename TX, typename TY>
__global__ __launch_bounds__(kOnceThreads, 4) void k_gn_once_last(OnceArgs<TX, TY> args) {
    typedef OnceLast<ACT, NV, TURN, TX, TY> F;
    extern __shared__ float lds[];
    __shared__ int missing;
    F f(args, lds, &missing);
    typename F::Vec cur[NV];
    const int rows = f.rows_of(f.chunk);
    const int64_t at = rows ? f.at_of(f.chunk) : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        cur[i] = *reinterpret_cast<const typename F::Vec*>(f.x_item() + at + max(0, min(i, rows - 1)) * f.step);
    if constexpr (F::kEarly) f.constants();
    f.put(f.chunk, rows, [&](auto&& take) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < rows) take(cur[i]);
    });
    const int lost = f.join(args.spin);
    if (lost < args.o.chunks) {
        once_late<ACT, NV, TURN, TX, TY>(args, lds, &missing, lost);
        return;
    }
    f.write(at, rows, [&](int i) { return cur[i]; });
}

// ---- chunks joined by the kernel that writes the output ------------------------------------
// With few chunks every workgroup of the output joins those of its own groups
// (a launch less: 3.5 us of a small call); `part` is null where k_gn_finish
// has done it.  `most` groups at most are a workgroup's: the lanes that share a
// group, and so the order of its sum, follow from that and the chunks and not
// from how many groups a workgroup has, so that all those that hold a part of a
// group see the same bits.
struct Join {
    const float2* part;
    int chunks, groups, most;
    bool last;
    int64_t per, n;
    float eps;
};
// (mean, 1 / deviation) of groups g0 .. g0 + ng - 1 (numbered over the items),
// to res[2 i], res[2 i + 1] in LDS; those from i = `own` on also to stats (one
// workgroup for each group).
__device__ __forceinline__ void join_chunks(const Join& f, int64_t g0, int ng, float* res, int own,
                                            float* __restrict__ stats) {
    const int t = threadIdx.x, threads = blockDim.x;
    int parts = 1;
    while (parts < 64 && 2 * parts * f.most <= threads && parts < f.chunks) parts *= 2;
    const int part = t & (parts - 1);
    for (int i = t / parts; i < ng; i += threads / parts) {
        const int64_t g = g0 + i;
        const float2* p = f.part + (f.last ? g / f.groups * f.chunks * f.groups + g % f.groups : g * f.chunks);
        const int step = f.last ? f.groups : 1;
        float sum = 0.0f;
#pragma unroll 4
        for (int k = part; k < f.chunks; k += parts)
            sum = fmaf((float)min(f.per, f.n - k * f.per), p[(int64_t)k * step].x, sum);
        const float mean = team_sum(sum, parts) / (float)f.n;
        sum = 0.0f;
#pragma unroll 4
        for (int k = part; k < f.chunks; k += parts) {
            const float2 q = p[(int64_t)k * step];
            const float d = q.x - mean;
            sum += fmaf((float)min(f.per, f.n - k * f.per) * d, d, q.y);
        }
        sum = team_sum(sum, parts);
        if (part == 0) {
            const float rstd = rsqrtf(sum / (float)f.n + f.eps);
            res[2 * i] = mean;
            res[2 * i + 1] = rstd;
            if (i >= own) {
                stats[2 * g] = mean;
                stats[2 * g + 1] = rstd;
            }
        }
    }
    __syncthreads();
}

// ---- output, the layout kept ------------------------------------------------------------
// Bound by memory: 537 MB read and written in 185 us (5.8 TB/s) by both.  A
// thread keeps its channels' constants; eight vectors a thread.
template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kMaxSlots) void k_gn_apply_last(const TX* __restrict__ x, const float* __restrict__ w,
                                                             const float* __restrict__ bias, float* stats,
                                                             TY* __restrict__ out, LastRows r, Join f, int per,
                                                             int chunks, int64_t blocks) {
    constexpr int V = kVec<TX>;
    extern __shared__ float joined[];
    const int64_t id = block_id();
    if (id >= blocks) return;
    const int64_t b = id / chunks;
    const int first = (int)(id % chunks) * per, last = min(first + per, r.ns);
    const int t = threadIdx.x, row = div_by(t, r.by_cv), slot = t - row * r.cv;
    const int groups = div_by(r.C, r.by_D);
    const float* st = stats + 2 * b * groups;
    if (f.part) {
        join_chunks(f, b * groups, groups, joined, first == 0 ? 0 : groups, stats);
        st = joined;
    }
    if (row >= r.q) return;
    const int64_t base = b * r.P * r.C + slot * V;
    float m[V], a[V], o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = mod_by(slot * V + j, r.by_cs), g = div_by(c, r.by_D);
        m[j] = st[2 * g];
        a[j] = st[2 * g + 1] * or_one(w, c);
        o[j] = or_zero(bias, c);
    }
    int s = first + row;
    for (; s + r.q < min(last, r.P / r.R); s += 2 * r.q) {
        float u[2][V], y[V];
        const int64_t e = base + (int64_t)s * r.stride(), f = e + (int64_t)r.q * r.stride();
        load_vec<V>(x + e, u[0]);
        load_vec<V>(x + f, u[1]);
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = act_value<ACT>(fmaf(u[0][j] - m[j], a[j], o[j]));
        store_vec<V>(out + e, y);
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = act_value<ACT>(fmaf(u[1][j] - m[j], a[j], o[j]));
        store_vec<V>(out + f, y);
    }
    for (; s < last; s += r.q) {
        float u[V];
        const int n = last_valid<V>(r, s, slot);
        const int64_t e = base + (int64_t)s * r.stride();
        load_part<V>(x + e, n, u);
#pragma unroll
        for (int j = 0; j < V; ++j) u[j] = act_value<ACT>(fmaf(u[j] - m[j], a[j], o[j]));
        store_part(out + e, n, u);
    }
}

template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kGnThreads) void k_gn_apply_first(const TX* __restrict__ x, const float* __restrict__ w,
                                                               const float* __restrict__ bias, float* stats,
                                                               TY* __restrict__ out, FirstRows r, Join f, int C, int D,
                                                               int64_t blocks) {
    constexpr int V = kVec<TX>;
    extern __shared__ float joined[];
    const int64_t id = block_id();
    if (id >= blocks) return;
    const int teams = kGnThreads / r.team;
    const int64_t row0 = id / r.chunks * teams, row = row0 + threadIdx.x / r.team;
    const int at = (int)(id % r.chunks) * r.piece, end = min(at + r.piece, r.P);
    const float* st = stats + 2 * (row / D);
    if (f.part) {
        // the workgroup with the first row of a group, and the first piece of it, stores its statistics
        const int64_t g0 = row0 / D, g1 = min(row0 + teams - 1, r.rows - 1) / D;
        const int ng = (int)(g1 - g0) + 1;
        join_chunks(f, g0, ng, joined, at ? ng : row0 % D ? 1 : 0, stats);
        st = joined + 2 * (row / D - g0);
    }
    if (row >= r.rows) return;
    const int c = (int)(row % C);
    const float m = st[0], a = st[1] * or_one(w, c), o = or_zero(bias, c);
    const int64_t base = row * r.P;
    for (int p = at + (threadIdx.x & (r.team - 1)) * V; p < end; p += r.team * V) {
        float u[V];
        const int n = min(V, end - p);
        load_part<V>(x + base + p, n, u);
#pragma unroll
        for (int j = 0; j < V; ++j) u[j] = act_value<ACT>(fmaf(u[j] - m, a, o));
        store_part(out + base + p, n, u);
    }
}

// ---- output in the other layout -----------------------------------------------------------
// Tiles turned in LDS, so that both sides are whole vectors: 268 MB moved in 43
// us (6.2 TB/s, the field partly in the caches from the statistics) for 32 x 64
// x 128 x 128, channels first to last.
template <int ACT, bool XLAST, typename TX, typename TY>
__global__ __launch_bounds__(kGnThreads) void k_gn_apply_cross(const TX* __restrict__ x, const float* __restrict__ w,
                                                               const float* __restrict__ bias, float* stats,
                                                               TY* __restrict__ out, Tiles q, Join f, int C, int P,
                                                               int D, int64_t blocks) {
    constexpr int V = kVec<TX>;
    __shared__ float tile[kTileLds];
    __shared__ float joined[2 * kMaxTileChannels];
    const int64_t id = block_id();
    if (id >= blocks) return;
    const int64_t per_item = (int64_t)q.tiles_c * q.tiles_p, b = id / per_item;
    const Spot s = spot_of(q, id % per_item, b, C, P);
    const float* st = stats + 2 * b * (C / D);
    if (f.part) {
        // the tile with the first channel of a group, and the first positions, stores its statistics
        const int g0 = s.c0 / D, ng = (s.c0 + s.nc - 1) / D - g0 + 1;
        join_chunks(f, b * (C / D) + g0, ng, joined, s.p0 ? ng : s.c0 % D ? 1 : 0, stats);
        st = joined - 2 * g0;
    }
    if constexpr (XLAST) {
        load_last(x, tile, q, s, C);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kTile / V / kGnThreads; ++i) {
        const Along<V> a(q, s, i);
        if (a.n) {
            const int c = s.c0 + a.c;
            const float m = st[2 * (c / D)], k = st[2 * (c / D) + 1] * or_one(w, c), o = or_zero(bias, c);
            const int64_t e = s.item + (int64_t)c * P + s.p0 + a.p;
            float* row = tile + a.c * (q.tp() + 1) + a.p;
            float u[V];
            if constexpr (XLAST) {
#pragma unroll
                for (int j = 0; j < V; ++j) u[j] = row[j];
            } else {
                load_part<V>(x + e, a.n, u);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) u[j] = act_value<ACT>(fmaf(u[j] - m, k, o));
            if constexpr (XLAST) {
                store_part(out + e, a.n, u);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) row[j] = u[j];
            }
        }
    }
    if constexpr (!XLAST) {
        __syncthreads();
        store_last(out, tile, q, s, C);
    }
}

// ---- channels last, too wide for a workgroup ------------------------------------------------
// Workgroup (item, chunk of `per` positions, group), reading runs of D values,
// twice (the second time from the caches); part[(b chunks + chunk) G + g].
// 134 MB in 78 us (4 x 8192 channels x 1024): scalar loads and their indexes.
// One workgroup a group took 3.5 ms.
template <typename TX>
__global__ __launch_bounds__(kGnThreads) void k_gn_stats_wide(const TX* __restrict__ x, float2* __restrict__ part,
                                                              int64_t C, int D, FastDiv by_D, int64_t P, int per,
                                                              int chunks, int64_t blocks) {
    __shared__ double red[16];
    const int64_t id = block_id();
    if (id >= blocks) return;
    const int64_t G = C / D, row = id / G, first = row % chunks * per;
    const TX* p = x + (row / chunks * P + first) * C + id % G * D;
    const int n = (int)min((int64_t)per, P - first) * D;
    const auto at = [&](int i) {
        // per D <= 65536 where per > 1: the division is exact
        const int r = per == 1 ? 0 : div_by(i, by_D);
        return (float)p[r * C + (i - r * D)];
    };
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += kGnThreads) sum += at(i);
    const float mean = (float)(block_sum(sum, red) / n);
    double sq = 0.0;
    for (int i = threadIdx.x; i < n; i += kGnThreads) {
        const float d = at(i) - mean;
        sq += d * d;
    }
    sq = block_sum(sq, red);
    if (threadIdx.x == 0) part[id] = make_float2(mean, (float)sq);
}

// Workgroup (row): C values of one position.  268 MB moved in 56 us (4.8 TB/s).
template <int ACT, typename TX, typename TY>
__global__ __launch_bounds__(kGnThreads) void k_gn_apply_wide(const TX* __restrict__ x, const float* __restrict__ w,
                                                              const float* __restrict__ bias,
                                                              const float* __restrict__ stats, TY* __restrict__ out,
                                                              int64_t C, int D, int64_t P, int64_t blocks) {
    const int64_t id = block_id();
    if (id >= blocks) return;
    const float* st = stats + 2 * (id / P) * (C / D);
    for (int64_t c = threadIdx.x; c < C; c += kGnThreads) {
        const int64_t g = c / D;
        const float xh = ((float)x[id * C + c] - st[2 * g]) * st[2 * g + 1];
        out[id * C + c] = (TY)act_value<ACT>(fmaf(xh, or_one(w, c), or_zero(bias, c)));
    }
}

// ---- schedules ------------------------------------------------------------------------------
enum Stats { kFusedLast, kFusedFirst, kOnceLast, kSplitLast, kSplitFirst, kWide };
struct Plan {
    Stats how;
    LastRows rows;                // fused or split, channels last
    int slices;                   // fused, channels last
    int threads;                  // fused, channels first
    int per, chunks;              // split: super-rows or values a chunk
    int64_t parts;                // float2 of workspace
    Once once;
    bool join;                    // split: the output's workgroups join the chunks
};

// Joining in every workgroup of the output reads `groups` times the chunks' pairs in each: worth it while those are
// few and the workgroups too.
bool joins(const GroupNorm& g, int chunks) {
    return (int64_t)chunks * g.groups <= 1024 && g.B * g.C * g.P <= (int64_t)4096 * 4096;
}

// Groups that a workgroup of the output has a part of, at most.
int join_most(const GroupNorm& g) {
    const int64_t D = g.C / g.groups;
    if (g.x_last == g.out_last)
        // channels first: 256 threads' rows are fewer values than a group that does not fit a workgroup
        return g.x_last ? (int)g.groups : 2;
    // a tile of 64 channels; where borders of groups are none of tiles, it can begin and end within one
    if (g.C <= kMaxTileChannels) return (int)g.groups;
    return kMaxTileChannels % D == 0 ? (int)(kMaxTileChannels / D) : (int)((kMaxTileChannels - 2) / D + 2);
}

size_t once_lds(const GroupNorm& g, const Plan& p) {
    const LastRows& r = p.rows;
    const int turn = g.x_last != g.out_last ? std::min(p.once.nv, 4) : 0;
    return sizeof(float) * (size_t)(once_buffer(r.threads, vec_of(g), r.C, turn, r.q * r.R) + r.q + 2 * g.groups);
}

Plan plan_forward(const GroupNorm& g) {
    const int V = vec_of(g);
    const int64_t D = g.C / g.groups, n = D * g.P;
    const int held = 32 / V;
    const bool same = g.x_last == g.out_last;
    const bool last = g.x_last;
    Plan p{};
    if (!last) {
        if (same && n <= kFusedValues) {
            p.how = kFusedFirst;
            const int64_t vectors = (n + V - 1) / V;
            p.threads = 64;
            while (p.threads < kFusedThreads && p.threads * held < vectors) p.threads *= 2;
            return p;
        }
        p.how = kSplitFirst;
        split_chunks(g.B * g.groups, n, 4 * kGnThreads * V, 64 * kGnThreads * V, &p.per, &p.chunks);
        p.parts = g.B * g.groups * p.chunks;
        p.join = joins(g, p.chunks);
        return p;
    }
    if (!last_rows_ok(g.C, V)) {
        p.how = kWide;
        split_chunks(g.B * g.groups, g.P, std::max<int64_t>(1, 4096 / D), std::max<int64_t>(1, 65536 / D), &p.per,
                     &p.chunks);
        p.parts = g.B * p.chunks * g.groups;
        return p;
    }
    if (same) {
        // the narrowest slice of whole groups that is a run of 64 bytes or more, or the whole rows
        int64_t cs = D;
        while (cs < g.C && (g.C % cs != 0 || cs % V != 0 || cs * 16 / V < 64)) cs += D;
        const LastRows r = last_rows(g.C, cs, D, g.P, V, kGnThreads);
        const int64_t vectors = (int64_t)r.ns * r.cv;
        if (vectors <= kFusedValues / V) {
            int threads = 64;
            while (threads < kFusedThreads && (threads < r.cv || (int64_t)(threads / r.cv) * held < r.ns)) threads *= 2;
            p.rows = last_rows(g.C, cs, D, g.P, V, threads);
            if ((int64_t)p.rows.q * held >= p.rows.ns && p.rows.threads <= kFusedThreads) {
                p.how = kFusedLast;
                p.slices = (int)(g.C / cs);
                return p;
            }
        }
    }
    p.rows = last_rows(g.C, g.C, D, g.P, V, kGnThreads);
    if (once_plan(g, p.rows, kOnceVectors, 1024, &p.once)) {
        if (once_lds(g, p) <= kLdsMax) {
            p.how = kOnceLast;
            p.parts = p.once.total * g.groups;
            return p;
        }
    }
    p.how = kSplitLast;
    p.rows = last_rows(g.C, g.C, D, g.P, V, kGnThreads);
    split_chunks(g.B, p.rows.ns, 4 * p.rows.q, 64 * p.rows.q, &p.per, &p.chunks);
    p.parts = g.B * p.chunks * g.groups;
    p.join = joins(g, p.chunks);
    return p;
}

}  // namespace

size_t gn_forward_workspace(const GroupNorm& g) { return sizeof(float2) * (size_t)plan_forward(g).parts; }

int gn_forward_kernels(const GroupNorm& g, const char** names) {
    const Plan p = plan_forward(g);
    const bool same = g.x_last == g.out_last;
    const char* apply = same ? "gn_apply" : "gn_apply_cross";
    if (p.how == kFusedLast || p.how == kFusedFirst) {
        names[0] = "gn_fused";
        return 1;
    }
    if (p.how == kOnceLast) {
        names[0] = "gn_clear";
        names[1] = "gn_once";
        return 2;
    }
    const bool two = p.join;
    names[0] = p.how == kWide ? "gn_stats_wide" : "gn_stats";
    names[1] = two ? apply : "gn_finish";
    names[2] = apply;
    return two ? 2 : 3;
}

hipError_t gn_forward_launch(const GroupNorm& g, const GroupNormArgs& a, int kernel, hipStream_t s) {
    const Plan p = plan_forward(g);
    const int D = (int)(g.C / g.groups), C = (int)g.C, P = (int)g.P;
    const int64_t n = (int64_t)D * P, runs = g.B * g.groups;
    float2* part = static_cast<float2*>(a.ws);
    return with_types(g, [&](auto tx, auto ty) {
        using TX = decltype(tx);
        using TY = decltype(ty);
        constexpr int V = kVec<TX>;
        const TX* x = static_cast<const TX*>(a.x);
        TY* out = static_cast<TY*>(a.out);
        float* stats = a.stats;
        const bool last = p.how == kSplitLast || p.how == kWide;
        const int64_t per = last ? (int64_t)p.per * (p.how == kWide ? 1 : p.rows.R) * D : p.per;
        const Join join{p.join ? part : nullptr, p.chunks, (int)g.groups, join_most(g), last, per, n, g.eps};
        const size_t lds = sizeof(float) * (size_t)(p.rows.threads * V + 2 * (D ? p.rows.cs / D : 0));
        if (kernel == 0 && p.how == kOnceLast)
            return launch_clear((uint64_t*)part, p.parts, s);
        if (kernel == 0 && p.how == kSplitLast) {
            const int64_t blocks = g.B * p.chunks;
            return launch_kernel(k_gn_stats_last<TX>, grid_of(blocks), dim3(p.rows.threads), lds, s, x, part, p.rows,
                                 p.per, p.chunks, blocks);
        }
        if (kernel == 0 && p.how == kSplitFirst) {
            const int64_t blocks = runs * p.chunks;
            return launch_kernel(k_gn_stats_first<TX>, grid_of(blocks), dim3(kGnThreads), 0, s, x, part, n, p.per,
                                 p.chunks, blocks);
        }
        if (kernel == 0 && p.how == kWide) {
            const int64_t blocks = runs * p.chunks;
            return launch_kernel(k_gn_stats_wide<TX>, grid_of(blocks), dim3(kGnThreads), 0, s, x, part, g.C, D,
                                 fast_div(D), g.P, p.per, p.chunks, blocks);
        }
        if (kernel == 1 && p.how != kOnceLast && !p.join) {
            return launch_kernel(k_gn_finish, grid_of(runs), dim3(kGnThreads), 0, s, (const float2*)part,
                                 a.stats, runs, (int)g.groups, p.chunks, last, per, n, g.eps);
        }
        return with_act(g.act, [&](auto act) {
            constexpr int ACT = decltype(act)::value;
            if (p.how == kFusedLast) {
                const int64_t blocks = g.B * p.slices;
                return launch_kernel(k_gn_fused_last<ACT, TX, TY>, grid_of(blocks), dim3(p.rows.threads), lds, s, x,
                                     a.weight, a.bias, out, a.stats, p.rows, p.slices, blocks, g.eps);
            }
            if (p.how == kOnceLast)
                return with_vectors<kOnceVectors>(p.once.nv, [&](auto nv) {
                    const OnceArgs<TX, TY> args{x,      a.weight, a.bias, out, a.stats, (uint64_t*)part,
                                                p.rows, p.once,   g.eps,  once_looks.load()};
                    constexpr int NV = decltype(nv)::value;
                    const bool turn = g.x_last != g.out_last;
                    const auto kernel_of = turn ? k_gn_once_last<ACT, NV, true, TX, TY>
                                                : k_gn_once_last<ACT, NV, false, TX, TY>;
                    return launch_kernel(kernel_of, dim3((unsigned)p.once.total), dim3(p.rows.threads),
                                         once_lds(g, p), s, args);
                });
            if (p.how == kFusedFirst)
                return launch_kernel(k_gn_fused_first<ACT, TX, TY>, grid_of(runs), dim3(p.threads), 0, s, x, a.weight,
                                     a.bias, out, a.stats, D, P, (int)g.groups, fast_div(P), runs, g.eps);
            if (g.x_last != g.out_last) {
                const Tiles q = tiles_of(C, P);
                const int64_t blocks = g.B * q.tiles_c * q.tiles_p;
                if (g.x_last)
                    return launch_kernel(k_gn_apply_cross<ACT, true, TX, TY>, grid_of(blocks), dim3(kGnThreads), 0, s,
                                         x, a.weight, a.bias, stats, out, q, join, C, P, D, blocks);
                return launch_kernel(k_gn_apply_cross<ACT, false, TX, TY>, grid_of(blocks), dim3(kGnThreads), 0, s, x,
                                     a.weight, a.bias, stats, out, q, join, C, P, D, blocks);
            }
            if (p.how == kSplitLast) {
                // eight vectors a thread: 32 KiB of a 16-byte-vector field a workgroup
                const int per = std::min(8 * p.rows.q, p.rows.ns), chunks = (p.rows.ns + per - 1) / per;
                const int64_t blocks = g.B * chunks;
                return launch_kernel(k_gn_apply_last<ACT, TX, TY>, grid_of(blocks), dim3(p.rows.threads),
                                     p.join ? sizeof(float) * 2 * (size_t)g.groups : 0, s, x, a.weight, a.bias, stats,
                                     out, p.rows, join, per, chunks, blocks);
            }
            if (p.how == kSplitFirst) {
                const FirstRows r = first_rows(g.B * g.C, g.P, V, 8);
                const int64_t blocks = first_blocks(r);
                return launch_kernel(k_gn_apply_first<ACT, TX, TY>, grid_of(blocks), dim3(kGnThreads),
                                     p.join ? sizeof(float) * 2 * kGnThreads : 0, s, x, a.weight, a.bias, stats, out,
                                     r, join, C, D, blocks);
            }
            const int64_t blocks = g.B * g.P;
            return launch_kernel(k_gn_apply_wide<ACT, TX, TY>, grid_of(blocks), dim3(kGnThreads), 0, s, x, a.weight,
                                 a.bias, (const float*)stats, out, g.C, D, g.P, blocks);
        });
    });
}

}  // namespace fno
