// Log-sum-exp, entropy, log probabilities of given tokens and the top
// alternatives of rows of logits, in one pass over them.
//
//   y = (x - m) s,  S = sum e^y,  lse = m s + log S,
//   log p(t) = y_t - log S,  entropy = log S - sum(e^y y) / S      (m = max x)
//
// HBM bound: the logits, once.  A row is one block's, or is cut into slices for
// a cluster of up to eight, whose blocks leave their parts in shared memory for
// the first of them to join: no workspace, one launch.  A thread takes groups of
// four 16-byte vectors and keeps its own base b for the exponentials, 2^4 above a
// group's maximum and moved only when a value lies 2^4 above it, so that the
// running maximum costs a maximum and a test per group.  (Not further: sum(e^y y)
// against b turns into that against m by sum * (b - m), which cancels.)  A block
// walks over rows and has the next one's first vectors under way while it joins its
// threads' parts.
//
// The k largest: every group's maximum stays in shared memory.  The threads form
// teams, and the k-th largest of the teams' maxima is a value that k values reach;
// the few groups that do are read again (from L2), a vector a thread, and their
// values that do are ranked by counting.
//
// Measured: 2048 rows of 131072 bf16 87 us without alternatives (6.2 TB/s, 91 % of
// the card's copy rate) and 103 with 20 of them (5.2 TB/s: four blocks a
// multiprocessor rank at about the same time, and 3.4 rows a block are a last round
// for a third of them; 70 % of the issue slots are taken); 121 rows of 100003 fp32, a
// third of them masked with -inf, a third with the lowest value, 19 us; 1 row of
// 32000 7.0, of which the alternatives are 3.
#include "csa2_common.cuh"
#include "csa2_timer.cuh"

#include <atomic>
#include <cfloat>
#include <climits>
#include <type_traits>

namespace csa2 {

constexpr int kLThreads = 256;     // of a block; 128 or 64 for many short rows
constexpr int kLGroup = 4;         // vectors of a group
constexpr int kLMaxTurns = 65;     // groups of a thread: 2^21 fp32 values in eight slices, and a vector for where a row begins
constexpr int kLTop = CSA2_LOGPROBS_TOP;
constexpr int kLHits = 512;        // groups that are read again at once
// Teams: 32 of 8 threads for up to kLFew alternatives, 128 of 2 for more (threads that
// far apart, so that neighbours' values fall into different ones).  Of random values,
// 30 of 256 threads' maxima reach the 20th largest of 32 teams', 75 the 64th of 128.
constexpr int kLFew = 24;
constexpr int kLMaxCluster = 8;
constexpr float kLFloor = -160.f;  // exponents below it are nothing in fp32
constexpr float kLReach = 4.f;     // a thread's base: this far above a maximum, moved for a value this far above it

struct LogArgs {
    const uint8_t* x;
    const int64_t* tokens;
    float* logprobs;
    float* lse;
    float* entropy;
    int32_t* ids;
    float* best;
    Status* st;
    int64_t stride, n;  // elements; rows
    int32_t vocab, given, top, slice;  // vectors of a slice
    float scale;        // of the logits
};

template <int NT>
struct LogSmem {
    static constexpr int NC = NT == kLThreads ? kLMaxCluster : 1;
    static constexpr int kCands = NT == kLThreads ? 1024 : 512;  // values that are ranked
    unsigned long long cand[kCands];   // (key of the value, ~index): larger values, then lower indices, are larger
    unsigned long long list[kLTop];    // the slice's largest, in order
    float max, sum, tilt;              // of the slice: m, S, sum(e^y y)
    int bad, listed, n_cand, n_ties, n_hits;
    uint32_t keys[NT];                 // of the threads' maxima
    uint16_t hits[kLHits];
    float red[3][NT / 32];
    int redi[NT / 32];
    // the first block's join
    unsigned long long all[NC][kLTop];
    int all_n[NC];
    float all_f[NC][3];
    int all_bad;
};

__device__ __forceinline__ unsigned long long ranked(float v, int32_t index) {
    return (static_cast<unsigned long long>(float_key(v)) << 32) | uint32_t(~uint32_t(index));
}
__device__ __forceinline__ float nan_max(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float exp2_of(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two floats in a register pair: half of the issue slots.
__device__ __forceinline__ uint64_t both(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void each(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t add_both(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul_both(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_both(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// sum += v with what the sum's rounding leaves behind in `rest` (a long tail next
// to a large term would vanish one by one: 2^-25 of the sum each, and twenty times
// that of the entropy).
__device__ __forceinline__ void add_kept(float& sum, float& rest, float v) {
    const float y = v + rest, t = sum + y;
    rest = y - (t - sum);
    sum = t;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }
// The same variable of another block of the cluster.
template <typename T>
__device__ __forceinline__ uint32_t peer(const T* p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t peer_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ unsigned long long peer_u64(uint32_t a) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t nan_max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A thread's sums against its base: y = x c - base in the log2 domain (c the scale
// times log2 e, a product inside one fused operation; base a whole number, so that
// it is exact), sum = sum 2^y, tilt = sum 2^y y.  Where |x c| passes 2^22 (masks of
// the type's lowest value alone, before anything else) y = (x - raw) c instead.
struct LogPart {
    float base = __builtin_nanf(""), raw = 0.f, floor = 0.f;  // floor: values that far down are nothing
    float sum = 0.f, sum_rest = 0.f, tilt = 0.f, tilt_rest = 0.f;
    bool plain = true;
    // How far x lies above the base, log2 domain (NaN before there is one).
    __device__ __forceinline__ float over(float x, float c) const { return plain ? fmaf(x, c, -base) : (x - raw) * c; }
    __device__ __forceinline__ void move(float m, float c) {
        const float b = rintf(m * c) + kLReach;
        const bool to_plain = fabsf(b) <= 0x1p22f;
        const float d = sum == 0.f ? 0.f : plain && to_plain ? base - b : (to_plain ? fmaf(m, c, -b) : 0.f) - over(m, c);
        const float f = sum == 0.f ? 0.f : exp2_of(d);
        tilt = f == 0.f ? 0.f : f * fmaf(sum, d, tilt);
        sum = f == 0.f ? 0.f : f * sum;
        sum_rest *= f, tilt_rest *= f;
        plain = to_plain;
        base = b;
        raw = fmaxf(m, -FLT_MAX);
        floor = (b + kLFloor) / c;
    }
};

// Rows begin anywhere: vectors are the 16-byte pieces of memory that hold the
// row, `head` elements of the first one lie before it.
template <typename T>
struct RowView {
    static constexpr int E = 16 / sizeof(T);
    const uint8_t* base;  // of vector 0
    int32_t head, vocab;
    __device__ __forceinline__ RowView(const LogArgs& a, int64_t row) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) + row * a.stride * int64_t(sizeof(T));
        head = int32_t(at & 15) / int32_t(sizeof(T));
        base = reinterpret_cast<const uint8_t*>(at & ~uintptr_t(15));
        vocab = a.vocab;
    }
    __device__ __forceinline__ int32_t vectors() const { return (head + vocab + E - 1) / E; }
    // E values of vector v; what lies outside the row is -inf
    __device__ __forceinline__ uint4 load(int32_t v) const {
        const int32_t i0 = v * E - head;
        if (i0 >= 0 && i0 + E <= vocab) return __ldg(reinterpret_cast<const uint4*>(base) + v);
        uint32_t w[4];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = i0 + e >= 0 && i0 + e < vocab ? __ldg(reinterpret_cast<const uint32_t*>(base) + 4 * int64_t(v) + e) : 0xFF800000u;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t two[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int32_t i = i0 + 2 * e + k;
                    two[k] = i >= 0 && i < vocab ? __ldg(reinterpret_cast<const uint16_t*>(base) + 8 * int64_t(v) + 2 * e + k) : 0xFF80u;
                }
                w[e] = two[0] | (two[1] << 16);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // Of a group's words (2 E pairs of values): the largest value (NaN if one is), values below a floor raised to it, a pair.
    static __device__ __forceinline__ float most(const uint32_t (&w)[4 * kLGroup]) {
        if constexpr (sizeof(T) == 4) {
            float m[2] = {__uint_as_float(w[0]), __uint_as_float(w[1])};
#pragma unroll
            for (int e = 2; e < 4 * kLGroup; ++e) m[e & 1] = nan_max(m[e & 1], __uint_as_float(w[e]));
            return nan_max(m[0], m[1]);
        } else {
            uint32_t m[2] = {w[0], w[1]};
#pragma unroll
            for (int e = 2; e < 4 * kLGroup; ++e) m[e & 1] = nan_max_bf16x2(m[e & 1], w[e]);
            m[0] = nan_max_bf16x2(m[0], m[1]);
            return nan_max(bf16_lo(m[0]), bf16_hi(m[0]));
        }
    }
    static __device__ __forceinline__ void at_least(uint32_t (&w)[4 * kLGroup], float floor) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < 4 * kLGroup; ++e) w[e] = __float_as_uint(fmaxf(__uint_as_float(w[e]), floor));
        } else {
            const uint32_t f = __float_as_uint(floor), b = (f + (f >> 31 ? 0xFFFFu : 0u)) >> 16, two = b | (b << 16);  // rounded down
#pragma unroll
            for (int e = 0; e < 4 * kLGroup; ++e) w[e] = nan_max_bf16x2(w[e], two);
        }
    }
    static __device__ __forceinline__ uint64_t pair(const uint32_t (&w)[4 * kLGroup], int e) {
        if constexpr (sizeof(T) == 4) return both(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
        else return both(bf16_lo(w[e]), bf16_hi(w[e]));
    }
    static __device__ __forceinline__ void values(const uint4& v, float (&x)[E]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(T) == 4) {
                x[e] = __uint_as_float(w[e]);
            } else {
                x[2 * e] = bf16_lo(w[e]);
                x[2 * e + 1] = bf16_hi(w[e]);
            }
        }
    }
};

// The sum of v over the block's earlier threads, and over all of them.
template <int NT>
__device__ __forceinline__ int block_before(LogSmem<NT>& S, int v, int& all) {
    const int lane = lane_id(), warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();  // the last use of redi
    if (lane == 31) S.redi[warp] = inc;
    __syncthreads();
    int before = inc - v;
    all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += S.redi[w];
        all += S.redi[w];
    }
    return before;
}

// The k largest of the slice, in order, to S.list (fewer where fewer are above -inf).
template <int NT, typename T>
__device__ void top_of_slice(LogSmem<NT>& S, const float* groups, const RowView<T>& row, int32_t v0, int32_t v1, int turns, float mine, int k) {
    constexpr int E = RowView<T>::E;
    const int tid = threadIdx.x;
    const int lane = tid & 31;
    S.keys[tid] = mine > -INFINITY ? float_key(mine) : 0u;
    if (tid == 0) S.n_hits = S.n_cand = S.n_ties = 0;
    __syncthreads();
    // the k-th largest of the teams' maxima (0 where fewer have any), by every warp
    uint32_t bar = 0;
    auto reach = [&](auto teams) {
        constexpr int N = decltype(teams)::value / 32;
        uint32_t own[N];
        int n[N] = {};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            own[i] = S.keys[32 * i + lane];
#pragma unroll
            for (int j = i + N; j < NT / 32; j += N) {
                const uint32_t u = S.keys[32 * j + lane];
                own[i] = own[i] > u ? own[i] : u;
            }
        }
#pragma unroll 8
        for (int j = 0; j < 32; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t u = __shfl_sync(0xffffffffu, own[i], j);
#pragma unroll
                for (int e = 0; e < N; ++e) n[e] += u >= own[e];
            }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (n[i] >= k && own[i] > bar) bar = own[i];
        bar = __reduce_max_sync(0xffffffffu, bar);
    };
    if (k <= kLFew) reach(std::integral_constant<int, 32>());
    else reach(std::integral_constant<int, (NT < 128 ? NT : 128)>());
    const uint32_t low = float_key(-INFINITY) + 1;  // -inf is no alternative
    if (bar < low) bar = low;
    // The values at the bar or above; where they are too many for the lists, or many and most of them equal, as where a mask
    // leaves less than k above its own value, those above it.  (They are ranked in n^2 steps: 1000 of them by 256 threads
    // took 25 us a row.)
    int n;
    uint32_t from = bar;
#pragma unroll 1
    for (;; ++from) {
        const float reached = key_float(from);
        for (int j = 0; j < turns; ++j) {
            const uint32_t those = __ballot_sync(0xffffffffu, groups[j * NT + tid] >= reached);
            if (those == 0) continue;
            int at = 0;
            if (lane == 0) at = atomicAdd(&S.n_hits, __popc(those));
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(those & ((1u << lane) - 1));
            if ((those >> lane & 1) && at < kLHits) S.hits[at] = uint16_t(j * NT + tid);
        }
        __syncthreads();
        const int n_hits = S.n_hits;
        n = INT_MAX;
        if (n_hits <= kLHits) {
            for (int i = tid; i < kLGroup * n_hits; i += NT) {
                const int group = S.hits[i / kLGroup], j = group / NT;
                const int32_t v = v0 + (j * kLGroup + i % kLGroup) * NT + (group - j * NT);
                if (v >= v1) continue;
                float x[E];
                row.values(row.load(v), x);
                uint32_t bits = 0, ties = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) bits |= uint32_t(float_key(x[e]) >= from) << e, ties |= uint32_t(float_key(x[e]) == from) << e;
                if (bits == 0) continue;
                int at = atomicAdd(&S.n_cand, __popc(bits));
                if (ties != 0) atomicAdd(&S.n_ties, __popc(ties));
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (bits >> e & 1) {
                        if (at < LogSmem<NT>::kCands) S.cand[at] = ranked(x[e], v * E - row.head + e);
                        ++at;
                    }
            }
            __syncthreads();
            n = S.n_cand;
        }
        if (from > bar || n <= (2 * S.n_ties > n ? 2 * kLTop : LogSmem<NT>::kCands)) break;
        __syncthreads();
        if (tid == 0) S.n_hits = S.n_cand = 0;
        __syncthreads();
    }
    if (n < k && from > bar) {  // the first ones at the bar, in the row's order
        const float reached = key_float(bar);
        for (int j = 0; j < turns && n < k; ++j) {
            const bool near = groups[j * NT + tid] >= reached;
            for (int g = 0; g < kLGroup && n < k; ++g) {
                const int32_t v = v0 + (j * kLGroup + g) * NT + tid;
                uint32_t bits = 0;  // of the vector's values at the bar
                if (near && v < v1) {
                    float x[E];
                    row.values(row.load(v), x);
#pragma unroll
                    for (int e = 0; e < E; ++e) bits |= uint32_t(float_key(x[e]) == bar) << e;
                }
                int all, at = n + block_before(S, __popc(bits), all);
                for (; bits != 0 && at < k; bits &= bits - 1, ++at)
                    S.cand[at] = ranked(key_float(bar), v * E - row.head + __ffs(bits) - 1);
                n = n + all < k ? n + all : k;
            }
        }
        __syncthreads();
    } else if (n > LogSmem<NT>::kCands) {
        // Many different ones, in the places of few threads: the k-th largest pair of value and index, bit by bit.
        auto visit = [&](uint32_t from, auto f) {  // the values of the groups whose maximum's key is `from` or more
            for (int j = 0; j < turns; ++j) {
                if (float_key(groups[j * NT + tid]) < from) continue;
#pragma unroll
                for (int g = 0; g < kLGroup; ++g) {
                    const int32_t v = v0 + (j * kLGroup + g) * NT + tid;
                    if (v >= v1) continue;
                    float x[E];
                    row.values(row.load(v), x);
#pragma unroll
                    for (int e = 0; e < E; ++e) f(x[e], v * E - row.head + e);
                }
            }
        };
        unsigned long long edge = 0;
#pragma unroll 1
        for (int b = 63; b >= 0; --b) {
            const unsigned long long up = edge | (1ull << b);
            int some = 0, all;
            visit(uint32_t(up >> 32) > low ? uint32_t(up >> 32) : low, [&](float x, int32_t i) { some += ranked(x, i) >= up; });
            block_before(S, some, all);
            if (all >= k) edge = up;
        }
        if (tid == 0) S.n_cand = 0;
        __syncthreads();
        visit(uint32_t(edge >> 32), [&](float x, int32_t i) {
            if (ranked(x, i) >= edge) S.cand[atomicAdd(&S.n_cand, 1)] = ranked(x, i);  // (k of them)
        });
        __syncthreads();
        n = S.n_cand;
    }
    for (int i = tid; i < n; i += NT) {
        const unsigned long long c = S.cand[i];
        int at = 0;
        for (int j = 0; j < n; ++j) at += S.cand[j] > c;
        if (at < k) S.list[at] = c;
    }
    if (tid == 0) S.listed = n < k ? n : k;
    __syncthreads();
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) token_logprobs_kernel(const LogArgs a, int cluster) {
    constexpr int E = RowView<T>::E;
    extern __shared__ __align__(16) float groups[];  // maxima of the groups, [turn][thread]
    __shared__ LogSmem<NT> S;
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
    const int64_t step = gridDim.x / uint32_t(cluster);
    int64_t r = blockIdx.x / uint32_t(cluster);
    const int rank = int(blockIdx.x) - int(r) * cluster;
    const float c = a.scale * 1.4426950408889634f;
    uint4 next[kLGroup];
    auto fetch = [&](const RowView<T>& row, int32_t v1, int32_t at) {  // vectors at .. of a slice that ends at v1
        const int32_t behind = at + kLGroup * NT;
        if ((at > 0 || row.head == 0) && behind <= v1 && behind * E <= row.head + row.vocab) {  // every one lies within the row
            const uint4* p = reinterpret_cast<const uint4*>(row.base) + at + tid;
#pragma unroll
            for (int g = 0; g < kLGroup; ++g) next[g] = __ldg(p + g * NT);
        } else {
#pragma unroll
            for (int g = 0; g < kLGroup; ++g) {
                const int32_t v = at + g * NT + tid;
                next[g] = v < v1 ? row.load(v) : (sizeof(T) == 4 ? make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u)
                                                                 : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u));
            }
        }
    };
    auto first = [&](const RowView<T>& row) { const int32_t nv = row.vectors(); return rank * a.slice < nv ? rank * a.slice : nv; };
    auto end = [&](const RowView<T>& row) { const int32_t nv = row.vectors(); return (rank + 1) * a.slice < nv ? (rank + 1) * a.slice : nv; };
    {
        const RowView<T> row(a, r);
        fetch(row, end(row), first(row));
    }
    for (; r < a.n; r += step) {
        const RowView<T> row(a, r);
        const int32_t v0 = first(row), v1 = end(row);
        const int turns = (v1 - v0 + NT * kLGroup - 1) / (NT * kLGroup);
        // the given tokens' logits, while the row comes in
        float x_given = -INFINITY;
        if (rank == 0 && tid < a.given) {
            const int64_t id = a.tokens[r * a.given + tid];
            if (id >= 0 && id < a.vocab)
                x_given = sizeof(T) == 4 ? reinterpret_cast<const float*>(a.x)[r * a.stride + id]
                                         : __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(a.x)[r * a.stride + id]) << 16);
            else if (id != -1)
                record(a.st, CSA2_ERR_DEVICE_BOUNDS, CHK_TOKEN, int32_t(r), int32_t(id));
        }
        // ---- one pass: base, sum and tilt of a thread, its maximum, its groups' maxima
        LogPart part;
        float top = -INFINITY;
        bool bad = false;
        for (int j = 0; j < turns; ++j) {
            uint32_t w[4 * kLGroup];
#pragma unroll
            for (int g = 0; g < kLGroup; ++g)
                w[4 * g] = next[g].x, w[4 * g + 1] = next[g].y, w[4 * g + 2] = next[g].z, w[4 * g + 3] = next[g].w;
            if (j + 1 < turns) fetch(row, v1, v0 + (j + 1) * kLGroup * NT);
            const float m = RowView<T>::most(w);
            groups[j * NT + tid] = m;
            if (!(part.over(m, c) <= kLReach)) {  // the first group, one far above the base, NaN
                if (!(m < INFINITY)) bad = true;
                part.move(m, c);
            }
            top = fmaxf(top, m);
            if (part.plain) {
                RowView<T>::at_least(w, part.floor);
                uint64_t gs[2] = {0, 0}, gt[2] = {0, 0};
                const uint64_t minus = both(-part.base, -part.base), cc = both(c, c);
#pragma unroll
                for (int e = 0; e < 2 * E; ++e) {
                    float y0, y1;
                    each(fma_both(RowView<T>::pair(w, e), cc, minus), y0, y1);
                    const float p0 = exp2_of(y0), p1 = exp2_of(y1);
                    gs[e & 1] = add_both(gs[e & 1], both(p0, p1));
                    gt[e & 1] = fma_both(both(p0, p1), both(y0, y1), gt[e & 1]);
                }
                float s0, s1, t0, t1;
                each(add_both(gs[0], gs[1]), s0, s1);
                each(add_both(gt[0], gt[1]), t0, t1);
                add_kept(part.sum, part.sum_rest, s0 + s1);
                add_kept(part.tilt, part.tilt_rest, t0 + t1);
            } else if (m > -INFINITY) {
                float s0 = 0.f, t0 = 0.f;
#pragma unroll
                for (int e = 0; e < 2 * E; ++e) {
                    float x[2];
                    each(RowView<T>::pair(w, e), x[0], x[1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float y = fmaxf((x[i] - part.raw) * c, kLFloor), p = exp2_of(y);
                        s0 += p;
                        t0 = fmaf(p, y, t0);
                    }
                }
                add_kept(part.sum, part.sum_rest, s0);
                add_kept(part.tilt, part.tilt_rest, t0);
            }
        }
        if (r + step < a.n) {
            const RowView<T> ahead(a, r + step);
            fetch(ahead, end(ahead), first(ahead));
        }
        float sum = part.sum + part.sum_rest, tilt = part.tilt + part.tilt_rest;
        // ---- the slice's: everything against its maximum
        float m = top;
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) S.red[0][warp] = m;
        const bool any_bad = __syncthreads_or(bad);
        m = S.red[0][lane & (NT / 32 - 1)];
#pragma unroll
        for (int o = NT / 64; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        {
            const float d = sum == 0.f ? 0.f : -part.over(m, c), f = sum == 0.f ? 0.f : exp2_of(d);
            tilt = f == 0.f ? 0.f : f * fmaf(sum, d, tilt);
            sum = f * sum;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            tilt += __shfl_xor_sync(0xffffffffu, tilt, o);
        }
        if (lane == 0) S.red[1][warp] = sum, S.red[2][warp] = tilt;
        if (a.top > 0 && !any_bad) top_of_slice<NT, T>(S, groups, row, v0, v1, turns, top, a.top);
        else if (tid == 0) S.listed = 0;
        __syncthreads();
        if (tid == 0) {
            float s = 0.f, t = 0.f;
            for (int w = 0; w < NT / 32; ++w) s += S.red[1][w], t += S.red[2][w];
            S.max = m, S.sum = s, S.tilt = t, S.bad = any_bad;
        }
        // ---- the row's
        if (cluster > 1) {
            cluster_arrive();
            cluster_wait();
            if (rank == 0) {
                if (tid < cluster) {
                    S.all_f[tid][0] = __uint_as_float(peer_u32(peer(&S.max, tid)));
                    S.all_f[tid][1] = __uint_as_float(peer_u32(peer(&S.sum, tid)));
                    S.all_f[tid][2] = __uint_as_float(peer_u32(peer(&S.tilt, tid)));
                    S.all_n[tid] = int(peer_u32(peer(&S.listed, tid)));
                }
                int b = tid < cluster ? int(peer_u32(peer(&S.bad, tid))) : 0;
                for (int i = tid; i < cluster * a.top; i += NT) {
                    const int q = i / a.top, e = i - q * a.top;
                    S.all[q][e] = peer_u64(peer(&S.list[e], q));  // (behind its last one: whatever is there)
                }
                b = __syncthreads_or(b);
                if (tid == 0) S.all_bad = b;
            }
            cluster_arrive();  // the others' parts are read
            if (rank != 0) {
                cluster_wait();
                continue;
            }
        } else {
            __syncthreads();
            if (tid == 0) {
                S.all_f[0][0] = S.max, S.all_f[0][1] = S.sum, S.all_f[0][2] = S.tilt;
                S.all_n[0] = S.listed;
                S.all_bad = S.bad;
            }
            for (int i = tid; i < a.top; i += NT) S.all[0][i] = S.list[i];
            __syncthreads();
        }
        float big = -INFINITY;
        for (int q = 0; q < cluster; ++q) big = fmaxf(big, S.all_f[q][0]);
        float s = 0.f, t = 0.f;
        int total = 0;
        for (int q = 0; q < cluster; ++q) {
            const float sq = S.all_f[q][1], d = sq == 0.f ? 0.f : (S.all_f[q][0] - big) * c, f = sq == 0.f ? 0.f : exp2_of(d);
            s = fmaf(f, sq, s);
            t = f == 0.f ? t : fmaf(f, fmaf(sq, d, S.all_f[q][2]), t);
            total += S.all_n[q];
        }
        const bool none = s == 0.f, nan = S.all_bad != 0;  // nothing above -inf; NaN or infinity among them
        const float log_s = logf(s), not_a = __uint_as_float(0x7FC00000u);
        if (tid == 0) {
            if (a.lse) a.lse[r] = nan ? not_a : none ? -INFINITY : fmaf(big, a.scale, log_s);
            if (a.entropy) a.entropy[r] = nan ? not_a : none ? 0.f : log_s - t / s * 0.6931471805599453f;
        }
        if (tid < a.given)
            a.logprobs[r * a.given + tid] = nan ? not_a : none || x_given == -INFINITY ? -INFINITY : (x_given - big) * a.scale - log_s;
        // alternatives: a value's place is how many of all lists are larger (none where a slice has NaN, whatever the others list)
        if (tid >= (nan ? 0 : total) && tid < a.top) {
            a.ids[r * a.top + tid] = -1;
            a.best[r * a.top + tid] = nan ? not_a : -INFINITY;
        }
        for (int i = tid; i < cluster * a.top && !nan; i += NT) {
            const int q = i / a.top, e = i - q * a.top;
            if (e >= S.all_n[q]) continue;
            const unsigned long long v = S.all[q][e];
            int at = e;
            if (cluster > 1) {
                int larger[LogSmem<NT>::NC] = {};  // of every list, its own among them: searched side by side
                for (int half = 1 << (31 - __clz(a.top)); half > 0; half >>= 1)
#pragma unroll
                    for (int o = 0; o < LogSmem<NT>::NC; ++o)
                        if (o < cluster && larger[o] + half <= S.all_n[o] && S.all[o][larger[o] + half - 1] > v) larger[o] += half;
                at = 0;
#pragma unroll
                for (int o = 0; o < LogSmem<NT>::NC; ++o) at += larger[o];
            }
            if (at < a.top) {
                a.ids[r * a.top + at] = int32_t(~uint32_t(v));
                a.best[r * a.top + at] = (key_float(uint32_t(v >> 32)) - big) * a.scale - log_s;
            }
        }
        __syncthreads();  // the next row writes where this one's parts were read
        if (cluster > 1) cluster_wait();
    }
}

}  // namespace csa2

using namespace csa2;

template <typename T, int NT>
static csa2_status logprobs_launch(const LogArgs& a, int cluster, cudaStream_t s) {
    const int64_t turns = ceil_div<int64_t>(a.slice, NT * kLGroup);
    if (turns > kLMaxTurns || a.n * cluster > INT32_MAX) return CSA2_ERR_UNSUPPORTED;
    static std::atomic<bool> done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CSA2_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(token_logprobs_kernel<T, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kLMaxTurns * NT * int(sizeof(float))) != cudaSuccess)
            return CSA2_ERR_CUDA;
        done[dev].store(true, std::memory_order_release);
    }
    timer_begin(K_LOGPROBS, s);
    // blocks that are resident at once walk over the rows (a cluster is made for few rows, one each)
    const int64_t most = 1024 / NT * int64_t(sm_count());
    launch(token_logprobs_kernel<T, NT>, dim3(unsigned(cluster > 1 || a.n < most ? a.n * cluster : most)), NT,
           size_t(turns) * NT * sizeof(float), s, unsigned(cluster), a, cluster);
    timer_end(K_LOGPROBS, s);
    return launch_status();
}

extern "C" csa2_status csa2_token_logprobs(const void* logits, int dtype, int64_t stride, int64_t n, int64_t vocab, float scale,
                                           const int64_t* tokens, int given, float* logprobs, float* lse, float* entropy, int top,
                                           int32_t* ids, float* best, void* ws, size_t ws_bytes, csa2_stream_t stream) {
    if (n < 0 || vocab < 1 || given < 0 || top < 0 || !(scale > 0.f) || !(scale <= FLT_MAX)) return CSA2_ERR_INVALID_ARG;
    if (dtype != CSA2_OUT_BF16 && dtype != CSA2_OUT_F32) return CSA2_ERR_UNSUPPORTED;
    if (n > (1 << 24) || vocab > (1 << 21) || given > kLTop || top > kLTop || !(scale >= 0x1p-20f) || !(scale <= 0x1p20f))
        return CSA2_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < CSA2_STATUS_BYTES || !aligned16(ws)) return CSA2_ERR_WORKSPACE;
    if (!logits || stride < vocab || stride > (int64_t(1) << 36)) return CSA2_ERR_INVALID_ARG;
    if (given > 0 && (!tokens || !logprobs)) return CSA2_ERR_INVALID_ARG;
    if (top > 0 && (!ids || !best)) return CSA2_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(logprobs), static_cast<const void*>(lse), static_cast<const void*>(entropy),
                          static_cast<const void*>(ids), static_cast<const void*>(best)})
        if (!aligned16(p)) return CSA2_ERR_INVALID_ARG;
    const int64_t size = dtype == CSA2_OUT_BF16 ? 2 : 4, in = ((n - 1) * stride + vocab) * size;
    if (reinterpret_cast<uintptr_t>(logits) % uint64_t(size) || reinterpret_cast<uintptr_t>(tokens) % 8) return CSA2_ERR_INVALID_ARG;
    if (n == 0) return CSA2_OK;
    const Span outs[] = {{logprobs, n * given * 4}, {lse, n * 4}, {entropy, n * 4}, {ids, n * top * 4}, {best, n * top * 4}};
    const Span ins[] = {{logits, in}, {tokens, n * given * 8}};
    if (!apart(outs, ins)) return CSA2_ERR_INVALID_ARG;
    LogArgs a{};
    a.x = static_cast<const uint8_t*>(logits);
    a.tokens = tokens;
    a.logprobs = logprobs;
    a.lse = lse;
    a.entropy = entropy;
    a.ids = ids;
    a.best = best;
    a.st = static_cast<Status*>(ws);
    a.stride = stride;
    a.n = n;
    a.vocab = int32_t(vocab);
    a.given = given;
    a.top = top;
    a.scale = scale;
    // A row in slices, so that all multiprocessors have a block of at least a vector per thread, or two blocks of 16 vectors
    // per thread; and so many that the groups' maxima find room.  (us, with 1 / 2 / 4 / 8 slices and 20 alternatives: 30 rows
    // of 32000 fp32 8.2 / 8.2 / 7.9 / 8.8, 61 rows 8.2 / 8.4 / 8.4 / 11; 61 of 100003 14 / 13 / 11 / 14, 152 of them
    // 24 / 19 / 26 / 26; 76 of 131072 bf16 13 / 11.5 / 15 / 19: clusters of four and more are not placed evenly.)
    const int64_t nv = vocab * size / 16 + 2;  // vectors of a row, wherever it begins
    auto fits = [&](int64_t c) {
        const int64_t sms = sm_count(), per_thread = nv / (c * kLThreads);
        return (n * c <= sms && per_thread >= 1) || (n * c <= (c == 2 ? 2 * sms : sms * 13 / 8) && per_thread >= 16);
    };
    int cluster = 1;
    while (cluster < kLMaxCluster &&
           (fits(2 * cluster) || ceil_div<int64_t>(ceil_div<int64_t>(nv, cluster), kLThreads * kLGroup) > kLMaxTurns))
        cluster *= 2;
    a.slice = int32_t(ceil_div<int64_t>(nv, cluster));
    cudaStream_t st = cudaStream_t(stream);
    // More rows than 256-thread blocks at once: smaller blocks, whose rows' starts and ends, and last rounds, go side by side.
    // (us with 256 / 128 / 64 threads, 20 alternatives: 2048 rows of 1000 fp32 22 / 13 / 9, of 5003 27 / 19 / 15, of 16000
    // 39 / 33 / 30, of 50021 86 / 77 / -; 1200 rows of 16000 22 / 19 / 21, of 65536 39 / 34 / - in
    // bf16 and 57 / 54 / - in fp32; but 620 rows of 32000 bf16 18 / 20 / 19, of 50021 24 / 27 / -, fp32 36 / 31 / -, whose
    // rows wait for memory rather than for instructions.  Longer rows' maxima leave little L1 beside eight blocks: 2048 of
    // 131072 bf16 104 / 110, 1200 of 100003 fp32 81 / 141.  64 threads are few for 64 alternatives: 2048 of 5003
    // 53 / 37 / 191.)
    const int64_t sms = sm_count();
    int threads = kLThreads;
    if (cluster == 1 && n > 4 * sms) {
        if (top <= kLFew && nv <= (n >= 12 * sms ? 4096 : 2560)) threads = 64;
        else if (size == 4 ? nv - 2 <= 16384 : nv - 2 <= 12800 && n >= 6 * sms) threads = 128;
    }
    auto go = [&](auto type) {
        using T = decltype(type);
        return threads == 64 ? logprobs_launch<T, 64>(a, 1, st) : threads == 128 ? logprobs_launch<T, 128>(a, 1, st) : logprobs_launch<T, kLThreads>(a, cluster, st);
    };
    return dtype == CSA2_OUT_BF16 ? go(__nv_bfloat16()) : go(float());
}
