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
    // Trees (null otherwise): a token sees the positions before its request's
    // tokens (within the window behind its own position) and those of its
    // request's tokens whose bit is set in its row of the mask.
    const uint32_t* mask;  // [n_tokens][words]
    const int64_t* pos;    // [n_tokens]; below 0: sees nothing
    int32_t words;
    int32_t groups;        // of a tree: CTAs that walk over the items (walk_first), 0: a CTA a split (paged_find)
    struct WalkCut* cuts;  // [groups]
};
// An item whose second piece is the first item of group g: paged_walk_merge_kernel
// joins its pieces, from group g - 1's on.
struct WalkCut {
    int64_t out0;          // its first row of the outputs
    int32_t rows, pieces;  // its rows; 0 pieces: none
    int32_t slot, pad[3];  // of the first piece (the others are their groups' first)
};

// Bits off .. off + 31 of a mask row (0 outside of it).
__device__ __forceinline__ uint32_t tree_bits(const uint32_t* row, int32_t words, int32_t off) {
    if (off <= -32 || off >= 32 * words) return 0;
    if (off < 0) return __ldg(row) << -off;
    const int32_t w = off >> 5;
    const uint32_t lo = __ldg(row + w), hi = w + 1 < words ? __ldg(row + w + 1) : 0;
    return __funnelshift_r(lo, hi, off & 31);
}
// The position of a node for its window: within [first, place], the request's first
// node's and the one that it would have in a chain.  Key tiles begin at the first
// node's window, so a position of the caller's below it has nothing more to see.
__device__ __forceinline__ int32_t tree_position(int64_t pos, int32_t first, int32_t place) {
    return pos <= first ? first : pos < place ? int32_t(pos) : place;
}
// Bits of the keys k .. k + 31 that lie in [lo, hi).
__device__ __forceinline__ uint32_t range_bits(int32_t k, int32_t lo, int32_t hi) {
    const int32_t l = lo - k, h = hi - k;
    if (l >= 32 || h <= 0) return 0;
    uint32_t v = 0xFFFFFFFFu;
    if (l > 0) v &= 0xFFFFFFFFu << l;
    if (h < 32) v &= 0xFFFFFFFFu >> (32 - h);
    return v;
}

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
// Tokens that an item's rows can belong to at most; of a tree, whose window begins
// at its request's first token for all of them, as many as the request has.
inline int32_t paged_item_tokens(int32_t heads, int32_t item, bool tree) { return tree ? INT32_MAX : (item - 1) / heads + 2; }
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
    // (a tree's later tokens may lie as far up as its first one)
    int32_t lo = a.window > 0 ? rq.len - rq.nq + (a.mask != nullptr ? 0 : r0 / a.by_heads) + 1 - a.window : 0;
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
    // Trees: the request's items and the key tiles of each, and what is left of the group's share from the item's start
    // on; of the group's first item, whether others hold pieces of it.
    int32_t items, tiles;
    int64_t left;
    WalkCut cut;
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

// Trees of several requests: the grid is one wave, and the requests' items are laid
// out over it by their real key tiles, in one of two ways:
//   pieces  every item is cut into pieces of at most c tiles, the least c with no
//           more pieces than groups of CTAs; a group takes one.
//   shares  every group walks over an equal share of all items' tiles in order, an
//           item's start counted as kWalkStart more; shares begin and end anywhere
//           in an item, so a group starts on two items or more.
// (walk_cut has the border.)  A group is one CTA of the few-row kernel, or the four
// of a pair of row tiles; it leaves two pieces at most that are no whole items: its
// first item's and a later one's.  64 heads, FP4, us so and with one split length
// for all requests: 16 requests of up to 8 nodes over 2K to 8K 109 and 188, 32 of 8
// over 4K to 16K 331 and 441 (few-row kernel); 4 of up to 32 over 2K to 8K 108 and
// 157, 8 of up to 64 over 4K to 16K 564 and 600 (row tiles).
// Key tiles' time of an item's start and end: as 2, 3, 4 or 6, 11 requests of up to 32 nodes x 32 heads over 2K take 48,
// 45, 48, 50 us, 14 of 38 x 16 over 6K 93, 91, 94, 97, 16 of 8 x 64 over 8K 110, 109, 109, 113.
constexpr int32_t kWalkStart = 3;
constexpr int32_t kWalkLeast = 2;  // tiles of a piece, and weight of a share
struct WalkSums {
    int64_t items, tiles;  // of all requests: items, and their tiles
};
// By pieces a CTA has c tiles and a start, by shares an even part of all tiles and
// two starts.
__device__ __forceinline__ int64_t walk_cut(const PagedArgs& a, const WalkSums& all) {  // c, or 0: by shares
    if (all.items >= a.groups) return 0;
    const int64_t n = a.groups - all.items;
    int64_t c = int64_t(__fdividef(float(all.tiles), float(n)));  // below 2^24 within one of the quotient, and enough above
    while (c * n < all.tiles) c += 1 + (all.tiles - c * n) / n;
    if (c < kWalkLeast) c = kWalkLeast;
    return c * a.groups <= all.tiles + kWalkStart * int64_t(a.groups) || c == kWalkLeast ? c : 0;
}
// Weight of a group's share, all but the last ones' equal.  (By a float's division,
// a little above the quotient: a whole number's takes a hundred instructions, and
// every block asks.)
__device__ __forceinline__ int64_t walk_share(const PagedArgs& a, int64_t total) {
    const int64_t n = int64_t(__fdividef(float(total), float(a.groups)) * (1.0f + 0x1p-19f)) + 1;
    return n > kWalkLeast ? n : kWalkLeast;
}
// A request's items, all with the key tiles of the whole request; pieces of an item
// of `cut` tiles each at most, evened out.
__device__ __forceinline__ void walk_items(const PagedArgs& a, int64_t r, PagedReq& rq, int32_t& items, int32_t& tiles, Status* st) {
    items = tiles = 0;
    if (r >= a.n_req || !paged_request(a, r, rq, st) || !paged_mine(a, rq)) return;
    const int32_t base = paged_base(a, rq);
    items = (rq.nq * a.heads + a.item - 1) >> a.item_log2;
    tiles = rq.len > base ? (rq.len - base + kPN - 1) / kPN : 0;
}
__device__ __forceinline__ int32_t walk_pieces(int32_t tiles, int64_t cut, int32_t& per) {
    per = tiles;
    if (tiles <= cut) return 1;
    const int32_t n = (tiles + int32_t(cut) - 1) / int32_t(cut);
    per = (tiles + n - 1) / n;
    return (tiles + per - 1) / per;
}
// Tiles [j0, j1) of w's item into the rest of w.
__device__ __forceinline__ void walk_piece(const PagedArgs& a, PagedWork& w, int64_t j0, int64_t j1, int64_t slot) {
    const int32_t rows = w.rq.nq * a.heads, r0 = w.item * a.item, r1 = (r0 + a.item < rows ? r0 + a.item : rows) - 1;
    const int32_t base = paged_base(a, w.rq), end = w.rq.len - w.rq.nq + r1 / a.by_heads + 1;
    const int32_t seen = end > base ? (end - base + kPN - 1) / kPN : 0;  // behind them no row of the item sees a key
    const int32_t last = int32_t(j1) < seen ? int32_t(j1) : seen;
    w.split = 0;
    w.splits = j0 == 0 && j1 == w.tiles ? 1 : 2;
    w.nt = last > j0 ? last - int32_t(j0) : 0;
    w.key0 = base + int32_t(j0) * kPN;
    w.out0 = int64_t(w.rq.q0) * a.heads + r0;
    w.part0 = slot * a.item;
}
// By shares, the group's part of w's item, `off` into it, to the end of the share
// (w.left from the item's start); w.nt is -1 where it has none.  An item without
// tiles is whole, and its zeros are of the group whose share has its start, also
// where the share ends within the start's weight.
__device__ __forceinline__ void walk_part(const PagedArgs& a, PagedWork& w, int64_t off, int64_t slot) {
    const int64_t j0 = off > kWalkStart ? off - kWalkStart : 0;
    const int64_t j1 = w.tiles > 0 && w.left - kWalkStart < w.tiles ? w.left - kWalkStart : w.tiles;
    if (w.tiles > 0 ? j1 <= j0 : off != 0) w.nt = -1;
    else walk_piece(a, w, j0, j1, slot);
}
// The item behind w's into `to` (which may be w), by one warp.
__device__ __forceinline__ void walk_next(const PagedArgs& a, const PagedWork& w, PagedWork& to, int64_t group) {
    const int lane = lane_id();
    const int64_t left = w.left - (w.tiles + kWalkStart);
    int64_t req = left > 0 ? w.req : -1;
    PagedReq rq = w.rq;
    int32_t item = w.item + 1, items = w.items, tiles = w.tiles;
    if (left > 0 && item >= items) {
        item = 0;
        req = -1;
        for (int64_t r0 = w.req + 1; r0 < a.n_req; r0 += 32) {
            walk_items(a, r0 + lane, rq, items, tiles, nullptr);
            const uint32_t some = __ballot_sync(0xffffffffu, items > 0);
            if (some == 0) continue;
            const int from = __ffs(some) - 1;
            req = r0 + from;
            rq.q0 = __shfl_sync(0xffffffffu, rq.q0, from), rq.nq = __shfl_sync(0xffffffffu, rq.nq, from);
            rq.len = __shfl_sync(0xffffffffu, rq.len, from);
            items = __shfl_sync(0xffffffffu, items, from), tiles = __shfl_sync(0xffffffffu, tiles, from);
            break;
        }
    }
    __syncwarp();  // (`to` may be w)
    if (lane == 0) {
        to.req = int32_t(req);
        if (req >= 0) {
            to.rq = rq;
            to.item = item;
            to.items = items;
            to.tiles = tiles;
            to.left = left;
            walk_part(a, to, 0, 2 * group + 1);
            if (to.nt < 0) to.req = -1;  // the share ends before the item's first tile
        }
    }
}
// The group's first item into w, by all WARPS warps of the block, which synchronize
// behind it.  (`sums` as in paged_find.)
template <int WARPS>
__device__ __forceinline__ void walk_first(const PagedArgs& a, int64_t group, bool all, PagedWork& w, int64_t* sums) {
    const int lane = lane_id(), warp = threadIdx.x >> 5;
    const bool wide = a.n_req > 32;
    if (threadIdx.x == 0) w.req = -1, w.cut.pieces = 0;
    __syncwarp();
    if (!wide && warp != 0) return;
    PagedReq rq;
    int32_t items = 0, tiles = 0;
    WalkSums total{0, 0};
    for (int64_t r0 = 0; r0 < a.n_req; r0 += 32 * WARPS) {
        walk_items(a, r0 + 32 * warp + lane, rq, items, tiles, all ? a.st : nullptr);
        total.items += items;
        total.tiles += int64_t(items) * tiles;
        if (!wide) break;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        total.items += __shfl_xor_sync(0xffffffffu, total.items, o);
        total.tiles += __shfl_xor_sync(0xffffffffu, total.tiles, o);
    }
    if (wide) {
        if (lane == 0) sums[warp] = total.items, sums[WARPS + warp] = total.tiles;
        __syncthreads();
        total.items = total.tiles = 0;
#pragma unroll 1
        for (int v = 0; v < WARPS; ++v) total.items += sums[v], total.tiles += sums[WARPS + v];
        __syncthreads();
    }
    const int64_t cut = walk_cut(a, total), weight = total.tiles + total.items * kWalkStart;
    const int64_t share = cut > 0 ? 1 : walk_share(a, weight), from = group * share;
    int64_t base = 0;
#pragma unroll 1
    for (int64_t r0 = 0; r0 < a.n_req; r0 += 32 * WARPS) {
        const int64_t r = r0 + 32 * warp + lane;
        if (wide) walk_items(a, r, rq, items, tiles, nullptr);
        int32_t per = 0;
        const int64_t each = cut > 0 ? walk_pieces(tiles, cut, per) : tiles + kWalkStart, mine = items * each;
        int64_t inc = mine, before = base;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (wide) {
            int64_t* at = sums + ((r0 / (32 * WARPS)) & 1) * WARPS;
            if (lane == 31) at[warp] = inc;
            __syncthreads();
#pragma unroll 1
            for (int v = 0; v < WARPS; ++v) {
                if (v < warp) before += at[v];
                base += at[v];
            }
        }
        const int64_t local = from - before - (inc - mine);
        const bool here = local >= 0 && local < mine;
        if (here) {
            const int64_t item = mine < (int64_t(1) << 32) ? int64_t(uint32_t(local) / uint32_t(each)) : local / each;
            const int64_t off = local - item * each;
            w.rq = rq;
            w.req = int32_t(r);
            w.item = int32_t(item);
            w.items = items;
            w.tiles = tiles;
            int32_t pieces = 0, slot = 0;
            if (cut > 0) {
                w.left = 0;
                walk_piece(a, w, off * per, (off + 1) * per < tiles ? (off + 1) * per : tiles, 2 * group);
                if (off == 1) pieces = int32_t(each);
            } else {
                w.left = off + (from + share < weight ? share : weight - from);
                walk_part(a, w, off, 2 * group);
                const int64_t back = off - share;  // where the share before this one begins
                if (group > 0 && off > kWalkStart && back <= kWalkStart) {
                    for (pieces = 2; off + (pieces - 1) * share < each; ++pieces) {}
                    slot = back < 0;
                }
            }
            if (pieces > 0) {
                const int32_t rows = rq.nq * a.heads - w.item * a.item;
                w.cut.out0 = w.out0;
                w.cut.rows = rows < a.item ? rows : a.item;
                w.cut.pieces = pieces;
                w.cut.slot = slot;
            }
        }
        if (__any_sync(0xffffffffu, here)) {
            __syncwarp();
            if (w.nt < 0) walk_next(a, w, w, group);  // an item without keys that an earlier share has
        }
        if (!wide || base > from) break;
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
