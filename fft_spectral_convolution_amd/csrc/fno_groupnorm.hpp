// Shared by the forward and backward group norm kernels: how a field is cut
// into vectors, rows and chunks, and the sums over a workgroup's part of it.
#pragma once

#include <algorithm>
#include <atomic>

#include "fno_fields.hpp"

namespace fno {

constexpr int kGnThreads = 256;
constexpr size_t kLdsMax = 65536;      // dynamic LDS of a workgroup, here

// Vector width of a field: 16 bytes.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// Workgroups are counted in up to two grid dimensions: a dimension holds
// fewer than 2^32 threads, and a field may have more groups than that.
inline dim3 grid_of(int64_t blocks) {
    constexpr int64_t kRow = 1 << 20;
    return blocks <= kRow ? dim3((unsigned)blocks) : dim3((unsigned)kRow, (unsigned)((blocks + kRow - 1) / kRow));
}
__device__ __forceinline__ int64_t block_id() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// ---- channels last ------------------------------------------------------------
// An item is P rows of C channels.  A workgroup covers `cs` neighbouring
// channels (all C of them, or a slice of whole groups).  Where C is no
// multiple of the vector width V, rows are taken R = V / gcd(C, V) at a time:
// R rows are a whole number of vectors, and a vector at place `slot` of such a
// super-row holds the channels (slot V + j) mod C whatever the super-row, so
// that each thread keeps its slot, and the constants of its channels stay in
// registers.  Only the last super-row of an item can be incomplete.
struct LastRows {
    int C, cs, D;          // channels, those of a slice, those of a group
    int P;                 // positions
    int R;                 // rows of a super-row (1 where cs < C)
    int cv;                // vectors of a super-row
    int q;                 // super-rows a workgroup takes at a time
    int threads;           // cv q, rounded up to whole waves
    int ns;                // super-rows of an item
    FastDiv by_cv, by_cs, by_D, by_R;
    __host__ __device__ int stride() const { return cs < C ? C : C * R; }   // elements from one to the next
};

inline int gcd_of(int a, int b) {
    while (b) {
        const int t = a % b;
        a = b;
        b = t;
    }
    return a;
}

inline LastRows last_rows(int64_t C, int64_t cs, int64_t D, int64_t P, int V, int threads) {
    LastRows r;
    r.C = (int)C;
    r.cs = (int)cs;
    r.D = (int)D;
    r.P = (int)P;
    const int g = gcd_of((int)std::min<int64_t>(cs, INT32_MAX), V);
    r.R = V / g;
    r.cv = (int)(cs / g);
    r.q = std::max(1, threads / r.cv);
    r.threads = (r.cv * r.q + 63) / 64 * 64;
    r.ns = (int)((P + r.R - 1) / r.R);
    r.by_cv = fast_div(r.cv);
    r.by_cs = fast_div(r.cs);
    r.by_D = fast_div(r.D);
    r.by_R = fast_div(r.R);
    return r;
}

constexpr int kMaxSlots = 512;    // slots a workgroup covers; wider items take the one-group-a-workgroup kernels
inline bool last_rows_ok(int64_t C, int V) { return C / gcd_of((int)std::min<int64_t>(C, INT32_MAX), V) <= kMaxSlots; }

// Elements of a thread's vector in super-row s that exist (all V but in the
// last super-row).
template <int V>
__device__ __forceinline__ int last_valid(const LastRows& r, int s, int slot) {
    if (s >= r.ns) return 0;
    if (r.R == 1) return V;
    const int64_t left = (int64_t)r.P * r.C - ((int64_t)s * r.R * r.C + slot * V);
    return left >= V ? V : left > 0 ? (int)left : 0;
}

// Loads n <= N elements, zeros beyond.
template <int N, typename T>
__device__ __forceinline__ void load_part(const T* p, int n, float (&v)[N]) {
    if (n == N) {
        load_vec<N>(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = j < n ? (float)p[j] : 0.0f;
    }
}
template <int N, typename T>
__device__ __forceinline__ void store_part(T* p, int n, const float (&v)[N]) {
    if (n == N) {
        store_vec<N>(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < n) p[j] = (T)v[j];
    }
}

// A vector as it lies in memory: values kept in registers between the passes
// of a kernel stay in their own type.
template <typename T, int N>
struct Raw {
    typename VecOf<T, N>::type q;
    __device__ __forceinline__ void load(const T* p, int n) {
        if (n == N) {
            q = *reinterpret_cast<const typename VecOf<T, N>::type*>(p);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) q[j] = j < n ? p[j] : (T)0.0f;
        }
    }
    __device__ __forceinline__ float operator[](int j) const { return (float)q[j]; }
};

// Sums of `val` (V values a thread) over the rows of a workgroup's super-rows
// and over `width` neighbouring channels: res[c / width].  width is D for
// group sums, 1 for channel sums.  buf holds threads * V floats.  Lanes
// `parts` at a time share a result, in an order that depends on the sizes
// alone.  buf may be reused after the next barrier, res is complete on return.
template <int V>
__device__ __forceinline__ void last_sums(const float (&val)[V], float* buf, float* res, const LastRows& r, int width) {
    const int t = threadIdx.x, active = r.cv * r.q;
    __syncthreads();
    if (t < active) {
#pragma unroll
        for (int j = 0; j < V; ++j) buf[t * V + j] = val[j];
    }
    __syncthreads();
    const FastDiv by_width = width == 1 ? FastDiv{1, 0, ~0u} : r.by_D;
    const int count = width == 1 ? r.cs : div_by(r.cs, r.by_D), entries = r.q * r.R * width;
    int parts = 1;
    while (parts < 64 && 2 * parts * count <= (int)blockDim.x) parts *= 2;
    const int part = t & (parts - 1), step = (int)blockDim.x >> __builtin_ctz(parts);
#pragma unroll 1
    for (int g = t >> __builtin_ctz(parts); g < count; g += step) {
        float s = 0.0f;
#pragma unroll 2
        for (int k = part; k < entries; k += parts) {
            const int row = div_by(k, by_width);
            s += buf[row * (r.cs - width) + g * width + k];
        }
        s = team_sum(s, parts);
        if (part == 0) res[g] = s;
    }
    __syncthreads();
}

// Chunks of a two-pass reduction over items of `units` each: about 2048
// workgroups in all, of min_per to max_per units.  The upper end bounds the
// chain of additions in a thread to a few hundred.
inline void split_chunks(int64_t items, int64_t units, int64_t min_per, int64_t max_per, int* per, int* chunks) {
    const int64_t want = std::max<int64_t>(1, 2048 / items);
    const int64_t p = std::min(std::min(std::max((units + want - 1) / want, min_per), max_per), units);
    *per = (int)p;
    *chunks = (int)((units + p - 1) / p);
}

// ---- one pass over items larger than a workgroup ------------------------------------
// An item's chunks are spread over workgroups that keep their values in
// registers, exchange two numbers a group and chunk through memory, and then
// write the output.  A pair travels as one 64-bit atomic, so nothing needs
// ordering: a slot holds kEmpty until its pair is there.  A workgroup does
// not depend on the others' progress: when a pair is not there after `spin`
// looks, it forms that chunk's sums itself and stores them, the same bits.
constexpr uint64_t kEmpty = ~0ull;
constexpr int kOnceThreads = 512, kLooks = 8;

__device__ __forceinline__ uint64_t pack_pair(float a, float b) {
    // NaNs of any payload become the one that kEmpty is not
    const uint32_t x = a == a ? __builtin_bit_cast(uint32_t, a) : 0x7fc00000u;
    const uint32_t y = b == b ? __builtin_bit_cast(uint32_t, b) : 0x7fc00000u;
    return (uint64_t)x << 32 | y;
}
__device__ __forceinline__ float2 unpack_pair(uint64_t v) {
    return make_float2(__builtin_bit_cast(float, (uint32_t)(v >> 32)), __builtin_bit_cast(float, (uint32_t)v));
}
__device__ __forceinline__ void put_pair(uint64_t* slot, float a, float b) {
    __hip_atomic_store(slot, pack_pair(a, b), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t look(const uint64_t* slot) {
    return __hip_atomic_load(slot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Fills v[i] with slots[part + i parts], i < kLooks, part + i parts < n;
// returns the first of those places that stayed empty, or n.
__device__ __forceinline__ int gather_pairs(const uint64_t* slots, int n, int part, int parts, int spin,
                                            uint64_t (&v)[kLooks]) {
#pragma unroll
    for (int i = 0; i < kLooks; ++i) v[i] = kEmpty;
    int missing = n;
    for (int tries = 0; tries <= spin; ++tries) {
        missing = n;
#pragma unroll
        for (int i = kLooks - 1; i >= 0; --i) {
            const int k = part + i * parts;
            if (k < n && v[i] == kEmpty) {
                v[i] = look(slots + k);
                if (v[i] == kEmpty) missing = k;
            }
        }
        if (missing == n) break;
        __builtin_amdgcn_s_sleep(1);
    }
    return missing;
}

// How an item is cut: `chunks` of q nv super-rows; `parts` lanes look for a
// group's pairs.
struct Once {
    int nv, chunks, parts;
    int64_t total;
};

// Whether a one-pass kernel serves the field, and how.  An item must fit half
// the workgroups that run at once, and its pairs the looks of a workgroup.
inline bool once_plan(const GroupNorm& g, const LastRows& r, int vectors, int running, Once* o) {
    if (r.threads > kOnceThreads || r.P % r.R) return false;
    o->parts = 1;
    while (o->parts < 64 && 2 * o->parts * g.groups <= r.threads) o->parts *= 2;
    if (o->parts * g.groups > r.threads) return false;
    const int64_t most = std::min(running / 2, o->parts * kLooks);
    // vectors a thread: as many as `vectors`, fewer where that would leave CUs without work
    const auto chunks_of = [&](int nv) { return (r.ns + (int64_t)r.q * nv - 1) / ((int64_t)r.q * nv); };
    o->nv = vectors;
    while (o->nv > 2 && g.B * chunks_of(o->nv) < 512 && chunks_of(o->nv / 2) <= most) o->nv /= 2;
    const int64_t chunks = chunks_of(o->nv);
    if (chunks > most || g.B * chunks >= 1 << 22) return false;
    o->chunks = (int)chunks;
    o->total = g.B * chunks;
    return true;
}

// Floats of LDS of k_gn_once_last's exchange: two values of each of a
// workgroup's elements, or `turn` vectors a thread turned to channel rows.
__host__ __device__ inline int once_buffer(int threads, int V, int C, int turn, int positions) {
    const int pairs = 2 * threads * V, turned = turn ? C * (turn * positions + 1) : 0;
    return pairs > turned ? pairs : turned;
}

// MOST: the vectors that once_plan was given
template <int MOST, typename F>
hipError_t with_vectors(int nv, F&& f) {
    switch (nv) {
        case MOST: return f(std::integral_constant<int, MOST>{});
        case MOST / 2: return f(std::integral_constant<int, MOST / 2>{});
        case 2: return f(std::integral_constant<int, 2>{});
        default: return f(std::integral_constant<int, 4>{});     // MOST is 8 or 16
    }
}

// Looks for another workgroup's sums before a workgroup forms them itself: at
// most some milliseconds.  fno_set_exchange_looks sets another count.
inline std::atomic<int> once_looks{kExchangeLooks};

// ---- channels first ------------------------------------------------------------
// Rows (b, c) of P positions.  A team of `team` threads (a power of two, at
// most the workgroup) takes a row, or one of its `chunks` pieces.
struct FirstRows {
    int64_t rows;          // B C
    int P, team, chunks, piece;
};
inline FirstRows first_rows(int64_t rows, int64_t P, int V, int vectors) {
    FirstRows r{rows, (int)P, 1, 1, (int)P};
    while (r.team < 64 && (int64_t)2 * r.team * V * 2 <= P) r.team *= 2;
    if (P >= (int64_t)2 * kGnThreads * V) {
        r.team = kGnThreads;
        r.piece = (int)std::min<int64_t>(P, (int64_t)kGnThreads * V * vectors);
        r.chunks = (int)((P + r.piece - 1) / r.piece);
    }
    return r;
}
inline int64_t first_blocks(const FirstRows& r) {
    const int per = kGnThreads / r.team;
    return (r.rows + per - 1) / per * r.chunks;
}

// ---- one layout to the other ----------------------------------------------------
// Tiles of 2^log2c channels and tp = 4096 / 2^log2c positions, turned in LDS
// (a row per channel, of odd length: lanes along channels and lanes along
// positions both fall on different banks).  The arithmetic is done along the
// positions, where a vector lies in one channel.  The channels-last side is
// read and written as runs: with up to 64 channels a tile's positions are one
// run of memory, whatever C is; of wider fields a tile takes 64 channels.
constexpr int kTile = 4096, kMaxTileChannels = 64;
constexpr int kTileLds = kTile + kMaxTileChannels;     // 2^log2c (tp + 1)
struct Tiles {
    int log2c, tiles_p, tiles_c;
    FastDiv by_c;                                      // the run's channels
    __host__ __device__ int tc() const { return 1 << log2c; }
    __host__ __device__ int tp() const { return kTile >> log2c; }
};
inline Tiles tiles_of(int64_t C, int64_t P) {
    Tiles t{0, 0, 0, {}};
    while (t.tc() < kMaxTileChannels && t.tc() < C) ++t.log2c;
    t.tiles_p = (int)((P + t.tp() - 1) / t.tp());
    t.tiles_c = (int)((C + t.tc() - 1) / t.tc());
    t.by_c = fast_div((int)std::min<int64_t>(C, kMaxTileChannels));
    return t;
}
// Where a tile lies: item, channels c0 .. c0 + nc - 1, positions p0 .. p0 + np - 1.
struct Spot {
    int64_t item;
    int c0, p0, nc, np;
};

// Calls f(element of the channels-last field, place in the tile of each of
// its V values, how many there are) for a thread's vectors of the tile.
template <int V, typename F>
__device__ __forceinline__ void last_side(const Tiles& q, const Spot& s, int C, F&& f) {
    const int ld = q.tp() + 1;
    if (q.tiles_c == 1) {
        const int n = s.np * C;
#pragma unroll
        for (int i = 0; i < kTile / V / kGnThreads; ++i) {
            const int e = (i * kGnThreads + (int)threadIdx.x) * V;
            if (e < n) {
                int place[V], p = div_by(e, q.by_c), c = e - p * C;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    place[j] = c * ld + p;
                    if (++c == C) {
                        c = 0;
                        ++p;
                    }
                }
                f(s.item + (int64_t)s.p0 * C + e, place, min(V, n - e));
            }
        }
    } else {
        constexpr int kPer = kMaxTileChannels / V;         // vectors of a position
#pragma unroll
        for (int i = 0; i < kTile / V / kGnThreads; ++i) {
            const int v = i * kGnThreads + (int)threadIdx.x, p = v / kPer, c = v % kPer * V;
            if (p < s.np && c < s.nc) {
                int place[V];
#pragma unroll
                for (int j = 0; j < V; ++j) place[j] = (c + j) * ld + p;
                f(s.item + (int64_t)(s.p0 + p) * C + s.c0 + c, place, min(V, s.nc - c));
            }
        }
    }
}
template <typename T>
__device__ __forceinline__ void load_last(const T* x, float* tile, const Tiles& q, const Spot& s, int C) {
    constexpr int V = kVec<T>;
    last_side<V>(q, s, C, [&](int64_t e, const int(&place)[V], int n) {
        float u[V];
        load_part<V>(x + e, n, u);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < n) tile[place[j]] = u[j];
    });
}
template <typename T>
__device__ __forceinline__ void store_last(T* out, const float* tile, const Tiles& q, const Spot& s, int C) {
    constexpr int V = kVec<T>;
    last_side<V>(q, s, C, [&](int64_t e, const int(&place)[V], int n) {
        float u[V];
#pragma unroll
        for (int j = 0; j < V; ++j) u[j] = j < n ? tile[place[j]] : 0.0f;
        store_part(out + e, n, u);
    });
}
__device__ __forceinline__ Spot spot_of(const Tiles& q, int64_t tile_id, int64_t b, int C, int P) {
    const int ct = (int)(tile_id % q.tiles_c), pt = (int)(tile_id / q.tiles_c);
    Spot s{b * (int64_t)P * C, ct << q.log2c, pt * q.tp(), 0, 0};
    s.nc = min(q.tc(), C - s.c0);
    s.np = min(q.tp(), P - s.p0);
    return s;
}
// A thread's vectors along the positions: i < kTile / V / kGnThreads.
template <int V>
struct Along {
    int c, p, n;          // channel and position in the tile, values (0: none)
    __device__ __forceinline__ Along(const Tiles& q, const Spot& s, int i) {
        const int lv = 12 - q.log2c - (V == 4 ? 2 : 3), v = i * kGnThreads + (int)threadIdx.x;
        c = v >> lv;
        p = (v & ((1 << lv) - 1)) * V;
        n = c < s.nc ? max(0, min(V, s.np - p)) : 0;
    }
};

__device__ __forceinline__ float or_one(const float* w, int64_t c) { return w ? w[c] : 1.0f; }
__device__ __forceinline__ float or_zero(const float* b, int64_t c) { return b ? b[c] : 0.0f; }

template <typename F>
hipError_t with_types(const GroupNorm& g, F&& f) {
    switch (g.x_type * 4 + g.out_type) {
        case kTypeF32 * 4 + kTypeF32: return f(float{}, float{});
        case kTypeBf16 * 4 + kTypeBf16: return f(bf16{}, bf16{});
        case kTypeBf16 * 4 + kTypeF32: return f(bf16{}, float{});
        case kTypeF16 * 4 + kTypeF16: return f(f16{}, f16{});
        default: return f(f16{}, float{});
    }
}
template <typename F>
hipError_t with_act(int act, F&& f) {
    switch (act) {
        case kActGelu: return f(std::integral_constant<int, kActGelu>{});
        case kActSilu: return f(std::integral_constant<int, kActSilu>{});
        default: return f(std::integral_constant<int, kActNone>{});
    }
}
inline int vec_of(const GroupNorm& g) { return g.x_type == kTypeF32 ? 4 : 8; }

// Empties the slots of a one-pass kernel.
hipError_t launch_clear(uint64_t* slots, int64_t n, hipStream_t s);

// Forward and backward halves of launch_group_norm and its queries.
int gn_forward_kernels(const GroupNorm& g, const char** names);
size_t gn_forward_workspace(const GroupNorm& g);
hipError_t gn_forward_launch(const GroupNorm& g, const GroupNormArgs& a, int kernel, hipStream_t s);
int gn_backward_kernels(const GroupNorm& g, bool need_x, bool need_w, const char** names);
size_t gn_backward_workspace(const GroupNorm& g);
hipError_t gn_backward_launch(const GroupNorm& g, const GroupNormArgs& a, int kernel, hipStream_t s);

}  // namespace fno
