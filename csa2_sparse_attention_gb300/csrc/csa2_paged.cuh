// Shared by the kernels of the paged attention call: arguments, the requests'
// work items, small wrappers of instructions, number formats.
#pragma once

#include "csa2_common.cuh"
#include "csa2_layout.cuh"
#include "csa2_tc.cuh"

namespace csa2 {

constexpr int kPD = CSA2_LATENT_DIM;
constexpr int kPHalf = kPD / 2;       // channels of one half
constexpr int kPN = 128;              // keys of a tile
constexpr int kPSoftWarps = 4;
// Decoded tiles (paged_decode_kernel): blocks of 128 channels, [16 key groups]
// [16 chunks of 8 channels][8 keys][16 bytes] in f16 each, as shared memory holds
// them; and per tile 128 bits of keys without a page, 128 bits of keys with a NaN
// latent.
constexpr int64_t kPTileBytes = int64_t(kPN) * kPD * 2;
constexpr int kPFlagBytes = 32;
// Probabilities enter the products in f16 as 2^(l - b), with b lowered by this
// much below the row's maximum when it is set, and set again once a logit lies
// kPGrow above it: P reaches 2^15 at most and the largest one 2^7 at least, so
// that what f16 rounds below its normal range (2^-25 each) is 2^-32 of the sum.
// (With b at the maximum it was 2^-25: half a million keys of probability just
// under that, 1.3 % of the output together, all rounded to zero.)
constexpr float kPBase = 7.f, kPGrow = 15.f;

// n / d for 0 <= n < 2^31 by a multiplication: with mul = floor(2^(31 + s) / d) + 1
// and 2^s >= d, mul d = 2^(31 + s) + e, 0 < e <= d, so n mul / 2^(31 + s) lies
// above n / d by n e / (d 2^(31 + s)) < 1 / d: the floor is that of n / d.  (The
// set-up of a CTA runs once through code that the instruction cache does not
// hold: a division by an unknown number is 25 instructions, this is three.)
struct FastDiv {
    uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f{d, 0, 31};
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    f.mul = uint32_t((uint64_t(1) << (31 + s)) / d + 1);
    f.shift = 31 + s;
    return f;
}
__device__ __forceinline__ int32_t operator/(int32_t n, const FastDiv& f) {
    return int32_t((uint64_t(uint32_t(n)) * f.mul) >> f.shift);
}

struct PagedArgs {
    const uint8_t* q;
    const int32_t* q_start;
    const int32_t* kv_len;
    const uint8_t* codes;
    const uint8_t* scales;
    const int32_t* table;
    uint8_t* out;
    float* lse;
    float* part_o;    // [splits][part_rows][512], each split's normalized output
    float* part_lse;  // [splits][part_rows], log2 domain
    uint8_t* tiles;   // decoded tiles [n_req][span][128 KB], or null
    uint8_t* flags;   // [n_req][span][32]
    Status* st;
    uint64_t wlim;
    int64_t n_rows_pages;  // pages of the cache
    int64_t max_pages;
    int64_t rows;          // n_tokens * heads
    int64_t part_rows;     // rows; behind the tile kernel n_req * few_rows, a request's from r * few_rows on
    int64_t n_req;
    int32_t n_tokens, heads, max_q, max_kv, page, window;
    // Key tiles per split; with `slots` the kernel lowers it, not below chunk_min,
    // to what spreads the requests' real lengths over that many items, and leaves
    // it at *chunk_out for the merge.
    int32_t chunk, chunk_min, slots;
    int32_t* chunk_out;
    FastDiv by_heads, by_page, by_few;
    int32_t span;          // decoded tiles per request
    int32_t item;          // rows of a work item: 64, or the 256 of two row tiles (decoded tiles); 2^item_log2
    int32_t item_log2, item_tokens;
    int32_t rows_over, rows_to;  // requests of rows_over < rows <= rows_to are this kernel's
    int32_t few_rows;      // the most rows of such a request
    int32_t tail;          // one request whose last items are split (paged_tail)
    int32_t behind;        // the few-row kernel: launched behind the tile kernel, which it does not depend on
    float sm_scale;
};

// A request's tokens and entries; false when it is to be skipped.  Problems
// go to `st` when it is not null.
struct PagedReq {
    int32_t q0, nq, len;
};
__device__ __forceinline__ bool paged_request(const PagedArgs& a, int64_t r, PagedReq& o, Status* st) {
    o.q0 = a.q_start[r];
    const int32_t q1 = a.q_start[r + 1];
    o.len = a.kv_len[r];
    if (o.q0 < 0 || q1 < o.q0 || q1 > a.n_tokens || q1 - o.q0 > a.max_q) {
        if (st) record(st, CSA2_ERR_DEVICE_BOUNDS, CHK_LENGTH, int32_t(r), q1);
        return false;
    }
    o.nq = q1 - o.q0;
    if (o.len < 0 || o.len > a.max_kv || o.len > a.max_pages * a.page) {
        if (st) record(st, CSA2_ERR_DEVICE_BOUNDS, CHK_LENGTH, int32_t(r), o.len);
        o.len = 0;
    }
    return o.nq > 0;
}
__device__ __forceinline__ bool paged_mine(const PagedArgs& a, const PagedReq& rq) {
    const int32_t rows = rq.nq * a.heads;
    return rows > a.rows_over && rows <= a.rows_to;
}
// Work items of a request; key tiles that one can span at most; its splits.
__host__ __device__ inline int32_t paged_items(int32_t nq, int32_t heads, int32_t item) {
    return (nq * heads + item - 1) / item;
}
__host__ __device__ inline int32_t paged_key_tiles(int32_t nq, int32_t len, int32_t window, int32_t item_tokens) {
    int32_t n = (len + kPN - 1) / kPN;
    if (window > 0) {
        const int32_t span = window + (nq < item_tokens ? nq : item_tokens) + 7;
        const int32_t w = (span + kPN - 1) / kPN + 1;  // and one where the first tile begins early
        n = n < w ? n : w;
    }
    return n;
}
// Tokens that an item's rows can belong to at most.
inline int32_t paged_item_tokens(int32_t heads, int32_t item) { return (item - 1) / heads + 2; }
__device__ __forceinline__ int32_t paged_splits(int32_t tiles, int32_t chunk) {
    if (tiles <= chunk) return 1;
    int32_t n = int32_t(__fdividef(float(tiles), float(chunk)));  // 32 at most, so off by one at most
    n += n * chunk < tiles;
    return n + (n * chunk < tiles);
}
// With I items of T key tiles in all, splits of c tiles make at most T / c + I of
// them: the least c with no more than `slots`.
__device__ __forceinline__ int32_t paged_chunk(const PagedArgs& a, uint32_t items, uint32_t tiles) {
    const uint32_t slots = uint32_t(a.slots);
    if (items >= slots || tiles >= uint32_t(a.chunk) * (slots - items)) return a.chunk;
    int32_t c = int32_t(__fdividef(float(tiles), float(slots - items)));
    while (uint32_t(c) * (slots - items) < tiles) ++c;
    return c > a.chunk_min ? c : a.chunk_min;
}

// One long request is rarely a whole number of waves: its last items (those
// with the fewest keys), what is left of whole waves of kPTailSlots, are split
// where two or more fit into the place of one.  `items`: how many are split,
// `splits`: into how many.
constexpr int32_t kPTailSlots = 38, kPTailTiles = 12;  // items of 4 CTAs at a time; key tiles that are worth it
__host__ __device__ inline void paged_tail(int32_t n, int32_t tiles, int32_t& items, int32_t& splits) {
    items = n % kPTailSlots;
    splits = items > 0 ? kPTailSlots / items : 1;
    if (splits > 8) splits = 8;
    if (splits < 2 || tiles < kPTailTiles) items = 0, splits = 1;
}

// First key that any token of the request sees, a multiple of 8: where the
// request's decoded tiles begin.
__device__ __forceinline__ int32_t paged_base(const PagedArgs& a, const PagedReq& rq) {
    const int32_t lo = a.window > 0 ? rq.len - rq.nq + 1 - a.window : 0;
    return lo > 0 ? lo & ~7 : 0;
}
// First key (a multiple of 8; with decoded tiles, where one begins), end and
// key tiles of a work item.
__device__ __forceinline__ void paged_item_keys(const PagedArgs& a, const PagedReq& rq, int32_t ti, int32_t& begin,
                                                int32_t& end, int32_t& tiles) {
    const int32_t rows = rq.nq * a.heads, r0 = ti * a.item, r1 = (r0 + a.item < rows ? r0 + a.item : rows) - 1;
    end = rq.len - rq.nq + r1 / a.by_heads + 1;
    int32_t lo = a.window > 0 ? rq.len - rq.nq + r0 / a.by_heads + 1 - a.window : 0;
    if (lo < 0) lo = 0;
    begin = lo & ~7;
    if (a.tiles != nullptr) {
        const int32_t base = paged_base(a, rq);
        begin = base + (begin - base) / kPN * kPN;
    }
    tiles = end > begin ? (end - begin + kPN - 1) / kPN : 0;
}

// The bits of a tile's keys as the softmax reads them.
struct alignas(32) PagedFlags {
    uint16_t hidden[8];  // keys without a page, a bit each
    uint16_t nan[8];     // keys with a NaN latent
};

// A CTA's part of the work: request, item of it, split, key tiles.
struct PagedWork {
    PagedReq rq;
    int32_t req;                 // -1: none
    int32_t item, split, splits;
    int32_t nt, key0;            // key tiles (0: nothing to see) and the first key
    int64_t out0, part0;         // the item's first row of the outputs and of the partial ones
};
// Finds it for the grid's `place`, by a scan of the requests' items, into shared
// memory; all WARPS warps of the block call it and synchronize behind it.  Up to
// 32 requests are the first warp's alone, more go to all warps 32 each (`sums`
// [2][WARPS] in shared memory): by one warp, 1024 requests took 0.5 us for every
// 32, 9 of a CTA's 32 us.  `all`: look at every request, so that each one's
// problems are recorded.  (`slots`: at most 32 requests, or 32 per warp.)
template <int WARPS>
__device__ __forceinline__ void paged_find(const PagedArgs& a, int64_t place, bool all, PagedWork& w, int64_t* sums) {
    const int lane = lane_id(), warp = threadIdx.x >> 5;
    const bool wide = a.n_req > 32;
    if (threadIdx.x == 0) w.req = -1;
    __syncwarp();
    if (!wide && warp != 0) return;
    int64_t base = 0;
#pragma unroll 1
    for (int64_t r0 = 0; r0 < a.n_req; r0 += 32 * WARPS) {
        const int64_t r = r0 + 32 * warp + lane;
        int32_t n = 0, tiles = 0, chunk = a.chunk;
        PagedReq rq;
        if (r < a.n_req && paged_request(a, r, rq, all ? a.st : nullptr) && paged_mine(a, rq)) {
            tiles = paged_key_tiles(rq.nq, rq.len, a.window, a.item_tokens);
            n = (rq.nq * a.heads + a.item - 1) >> a.item_log2;
        }
        if (a.slots) {
            // each bounded so that 256 of them are below 2^32 (the host sees to it that chunk * slots is below 2^24)
            const int64_t all_tiles = int64_t(n) * tiles;
            uint32_t si = __reduce_add_sync(0xffffffffu, n < (1 << 24) - 1 ? uint32_t(n) : (1u << 24) - 1);
            uint32_t st = __reduce_add_sync(0xffffffffu, all_tiles < (1 << 24) - 1 ? uint32_t(all_tiles) : (1u << 24) - 1);
            if (wide) {
                if (lane == 0) sums[warp] = si, sums[WARPS + warp] = st;
                __syncthreads();
                si = st = 0;
#pragma unroll 1
                for (int v = 0; v < WARPS; ++v) si += uint32_t(sums[v]), st += uint32_t(sums[WARPS + v]);
                __syncthreads();
            }
            chunk = paged_chunk(a, si, st);
            if (all && threadIdx.x == 0) *a.chunk_out = chunk;
        }
        const int32_t ns = paged_splits(tiles, chunk);
        int32_t tail = 0, tail_splits = 1;
        if (a.tail) paged_tail(n, tiles, tail, tail_splits);
        const int64_t mine = int64_t(n) * ns + tail * (tail_splits - 1);
        int64_t inc = mine, before = base;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (wide) {
            int64_t* at = sums + ((r0 / (32 * WARPS)) & 1) * WARPS;  // two halves in turn: one barrier a round is enough
            if (lane == 31) at[warp] = inc;
            __syncthreads();
#pragma unroll 1
            for (int v = 0; v < WARPS; ++v) {
                if (v < warp) before += at[v];
                base += at[v];
            }
        }
        const int64_t local = place - before - (inc - mine);
        if (local >= 0 && local < mine) {
            const uint32_t back = uint32_t(local) / uint32_t(ns);
            int32_t item = n - 1 - int32_t(back), split = int32_t(uint32_t(local) - back * ns);  // the most keys first
            if (local >= n - tail && tail > 0) {
                const int32_t k = int32_t(local) - (n - tail);
                item = tail - 1 - k / tail_splits;
                split = k % tail_splits;
            }
            int32_t begin, end, seen;
            paged_item_keys(a, rq, item, begin, end, seen);
            if (item < tail) chunk = (seen + tail_splits - 1) / tail_splits;
            const int32_t splits = paged_splits(seen, chunk), j0 = split * chunk;
            if (split < splits) {
                w.rq = rq;
                w.req = int32_t(r);
                w.item = item;
                w.split = split;
                w.splits = splits;
                w.nt = seen - j0 < chunk ? seen - j0 : chunk;
                w.key0 = begin + j0 * kPN;
                w.out0 = int64_t(rq.q0) * a.heads + item * a.item;
                w.part0 = item < tail ? (int64_t(split) * tail + item) * a.item
                                      : split * a.part_rows + (a.behind ? r * a.few_rows + item * a.item : w.out0);
            }
        }
        if (!wide || (base > place && !all)) break;
    }
}

__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
                 ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(uint32_t(acc)));
}
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// One bulk copy shared memory -> global (addresses and size multiples of 16
// bytes), and the wait until this thread's copies have read shared memory (what
// they write is there when the kernel is done).
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\ncp.async.bulk.commit_group;" ::"l"(dst),
                 "r"(smem_u32(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_s2g_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f32x2_out(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t* o) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t* o) {
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n"
        " cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
        : "=r"(o[0]), "=r"(o[1]) : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// 32 bytes from a 16-byte aligned address: one load where it is 32-byte aligned
// (all rows of an operand are, or none), two otherwise.
struct U32x8 {
    uint32_t w[8];
};
__device__ __forceinline__ U32x8 ldg_32b(const uint8_t* p) {
    U32x8 v;
    asm volatile(
        "{\n .reg .pred one;\n .reg .b64 t;\n and.b64 t, %8, 16;\n setp.eq.u64 one, t, 0;\n"
        " @one ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
        " @!one ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%8];\n"
        " @!one ld.global.nc.v4.b32 {%4,%5,%6,%7}, [%8+16];\n}\n"
        : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
          "=r"(v.w[7])
        : "l"(p));
    return v;
}
// nonzero when one of the four E4M3 bytes is NaN (0x7F or 0xFF)
__device__ __forceinline__ uint32_t e4m3_nan4(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Q's conversion to f16: 8 rows per warp, four lanes per row, lane / 8 with 32
// bytes of every 128.  The power of two of a row from its maximum, max |q| 2^-qs
// in [2^14, 2^15): exact for elements above 2^-28 of it.
__device__ __forceinline__ void paged_q_load(const PagedArgs& a, int64_t flat, bool on, U32x8 (&v)[8]) {
    const uint8_t* src = a.q + (on ? flat : 0) * (kPD * 2) + 32 * (lane_id() >> 3);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (on) {
            v[i] = ldg_32b(src + 128 * i);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i].w[e] = 0;
        }
    }
}
__device__ __forceinline__ int paged_q_exponent(const U32x8 (&v)[8]) {
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) am = __vmaxu2(am, v[i].w[e] & 0x7FFF7FFFu);
    am = max(am & 0xFFFFu, am >> 16);
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 8));
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 16));
    const int qs = am != 0 ? int(am >> 7) - 127 - 14 : 0;
    return qs < -100 ? -100 : qs;
}
// Channels 64 i + 16 (lane / 8) .. + 15 of a row into two chunks, 128 bytes
// apart.
__device__ __forceinline__ void paged_q_store(uint8_t* dst, const U32x8& v, int qs) {
    const float qf = __uint_as_float(uint32_t(127 - qs) << 23);
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = f16x2(bf16_lo(v.w[e]) * qf, bf16_hi(v.w[e]) * qf);
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(dst + 128) = make_uint4(o[4], o[5], o[6], o[7]);
}
// The factor of a row's raw logits, log2 domain (never 0: -inf stays -inf).
__device__ __forceinline__ float paged_q_scale(const PagedArgs& a, int qs) {
    return fmaxf(a.sm_scale * 1.4426950408889634f * __uint_as_float(uint32_t(127 + qs) << 23), 1.1754944e-38f);
}

constexpr float kLn2 = 0.6931471805599453f;

// The kernels of csa2_paged_rows.cu and csa2_paged_tiles.cu, launched on `s`.
csa2_status paged_rows_launch(const PagedArgs& a, bool fp8, unsigned grid, cudaStream_t s);
csa2_status paged_tiles_launch(const PagedArgs& a, bool fp8, unsigned grid, cudaStream_t s);

}  // namespace csa2
