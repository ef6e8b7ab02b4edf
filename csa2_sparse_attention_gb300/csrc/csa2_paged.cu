// Causal attention over paged latents: the call's plan, its entry points and
// the join of its splits (the kernels: csa2_paged_rows.cu for requests of up to
// 256 (token, head) rows or four key tiles, csa2_paged_tiles.cu for more).
#include "csa2_paged.cuh"
#include "csa2_timer.cuh"

#include <cfloat>

namespace csa2 {

constexpr int kPSms = 152;  // multiprocessors the split is planned for
constexpr int kPSlotReqs = 256;  // a request per thread of the tile kernel's block

// Joins the splits of a kernel's rows: weights 2^(lse_s - max lse) over the
// normalized partial outputs.  128 threads per row, 4 channels each; rows whose
// tile had one split were written by the attention kernel.
// Two rows per CTA, or eight where most of them may not be there.
inline __host__ __device__ int paged_merge_rows(const PagedArgs& a) { return a.behind || a.tail ? 8 : 2; }
__global__ void __launch_bounds__(256) paged_merge_kernel(const PagedArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const int t = threadIdx.x & 127, lane = lane_id();
    const int32_t chunk = a.slots ? *a.chunk_out : a.chunk;
#pragma unroll 1
    for (int i = threadIdx.x >> 7; i < paged_merge_rows(a); i += 2) {
        const int64_t prow = int64_t(blockIdx.x) * paged_merge_rows(a) + i;  // of the partial outputs
        if (prow >= a.part_rows) return;
        int64_t req = 0;
        if (a.behind) {
            req = int32_t(prow) / a.by_few;
        } else if (!a.tail) {  // the last request that starts at or before the token
            const int32_t tok = int32_t(prow) / a.by_heads;
            int64_t hi = a.n_req;
            while (hi - req > 1) {
                const int64_t mid = (req + hi) / 2;
                if (a.q_start[mid] <= tok) req = mid;
                else hi = mid;
            }
        }
        PagedReq rq;
        bool found = paged_request(a, req, rq, nullptr);
        if (!a.behind && !a.tail) {
            // A token behind the last request, or q_start is out of order, where the search above leads anywhere: the
            // attention kernel took every request with good bounds all the same, so look at all of them.
            const int32_t tok = int32_t(prow) / a.by_heads;
            auto owns = [&](const PagedReq& o) { return tok >= o.q0 && tok - o.q0 < o.nq; };
            found = found && owns(rq);
            if (!found) {
                int32_t own = INT32_MAX;
                for (int64_t r = lane; r < a.n_req && own == INT32_MAX; r += 32)
                    if (paged_request(a, r, rq, nullptr) && owns(rq)) own = int32_t(r);
                own = __reduce_min_sync(0xffffffffu, own);
                found = own != INT32_MAX && paged_request(a, own, rq, nullptr);
            }
        }
        if (!found || !paged_mine(a, rq)) continue;
        const int64_t at = prow - (a.behind ? req * a.few_rows : a.tail ? 0 : int64_t(rq.q0) * a.heads);  // of the request's rows
        if (at < 0 || at >= int64_t(rq.nq) * a.heads) continue;
        int32_t begin, end, tiles;
        paged_item_keys(a, rq, int32_t(at) >> a.item_log2, begin, end, tiles);
        int32_t splits;
        int64_t stride = a.part_rows;
        if (a.tail) {
            int32_t tail, tail_splits;
            paged_tail((rq.nq * a.heads + a.item - 1) >> a.item_log2, paged_key_tiles(rq.nq, rq.len, a.window, a.item_tokens), tail,
                       tail_splits);
            stride = tail * a.item;
            splits = at < stride ? paged_splits(tiles, (tiles + tail_splits - 1) / tail_splits) : 1;
        } else {
            splits = paged_splits(tiles, chunk);
        }
        if (splits == 1) continue;
        const int64_t row = int64_t(rq.q0) * a.heads + at;
        // a lane per split (there are at most 32), and eight splits' loads under way
        float m = lane < splits ? a.part_lse[lane * stride + prow] : -INFINITY, f = m;
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        f = f == -INFINITY ? 0.f : ex2(f - m);
        float w = f;
#pragma unroll
        for (int d = 16; d; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
        const float4* src = reinterpret_cast<const float4*>(a.part_o + prow * kPD) + t;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int32_t s0 = 0; s0 < splits; s0 += 8) {
            float4 v[8];
#pragma unroll
            for (int s = 0; s < 8; ++s)
                v[s] = s0 + s < splits ? src[(s0 + s) * stride * (kPD / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const float fs = __shfl_sync(0xffffffffu, f, s0 + s);
                o.x = fmaf(fs, v[s].x, o.x);
                o.y = fmaf(fs, v[s].y, o.y);
                o.z = fmaf(fs, v[s].z, o.z);
                o.w = fmaf(fs, v[s].w, o.w);
            }
        }
        const float inv = w == 0.f ? 0.f : 1.0f / w;
        const __nv_bfloat162 h0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), h1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        reinterpret_cast<uint2*>(a.out + row * kPD * 2)[t] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
        if (a.lse && t == 0) a.lse[row] = w == 0.f ? -INFINITY : (m + log2f(w)) * kLn2;
    }
}

// How a call runs, from the host's bounds alone.  Requests of up to 256 rows
// go in items of 64 rows (csa2_paged_rows.cu), longer ones in pairs of 128
// rows over decoded tiles (csa2_paged_tiles.cu) where those need no more than
// 4 GB.  Decoding a key once pays from a few items on: 1024 tokens x 64 heads
// over 16K entries take 1.79 ms from tiles and 2.69 ms in items of 64 rows.  The
// border, 64 heads over 8K entries: 16 requests of 4 tokens (4 items each) 135 us
// from tiles and 125 us without, of 8 tokens 191 and 209 us; single tokens would
// write and read 1 KB per key for nothing (125 and 43 us).  About where an item
// sees four tiles it stops paying as well (64 heads, 1024 tokens with a window of
// 128, 3 tiles: 115 us from tiles, 120 without; 100 tokens + 31 single ones over
// 500, 5 tiles: 32 and 26; 4 x 512 with 512, 6 tiles: 310 and 354).  Tiles run
// requests of any length; beside them the few-row kernel takes the short ones
// where the call's tokens say that there are enough of those, by a sixth of the
// longest request per request, or three quarters from 16 key tiles on.  64 heads,
// us with both kernels and with tiles alone:
//   512 tokens + 63 single ones, 8K   727   865     + 15 single ones   630  638
//   256 tokens + 31 single ones, 32K 1345  2008
//   100 tokens + 31 single ones, 500   32    39     16 x 100, 1K       340  324
//   8 x 64 + 24 single ones, 1K       158   130     8 x 64 + 8, 1K     142  123
//   8 x 64 + 24 single ones, 8K       658   687     8 x 64 + 8, 8K     647  646
// 16 heads, 8 x 64 + 24 single ones: 8K 238 and 375, 2K 84 and 112.  With few
// single tokens over less than 8K the tiles alone would be the faster (8 x 64 + 8,
// 16 heads: 8K 258 and 238, 4K 120 and 102, 2K 78 and 56): a row tile behind a
// request's rows leaves at once.  The border stands where it was when it did not.
// One request's last wave is filled by splitting its last items (paged_tail): 512
// tokens x 64 heads over 8K, 128 items in 3.4 waves, 567 us without and 523 with.
// The split count of each is the one with the least time by: waves of 152 CTAs,
// each a start and end of 8 us and a time per key tile, plus the merge's pass
// over the partial outputs.  That is for requests as long as max_kv; with up to
// kPSlotReqs requests the kernels then shorten the splits by the real lengths
// (paged_chunk), down to half: 16 single tokens x 64 heads over 2K to 8K entries
// took 42.0 us without that and 34.6 us with it.
struct PagedShare {  // of one of the kernels
    int32_t chunk = 1, splits = 1;         // as the partial outputs are sized
    int32_t chunk_min = 1, slots = 0;      // see PagedArgs
    int64_t grid = 0;                      // 0: not launched
};
static PagedShare paged_share(int64_t planned, int64_t most, int ctas, int64_t n_req, int32_t nt, double tile_us,
                              double merge_rows) {
    PagedShare p;
    p.chunk = nt > 0 ? nt : 1;
    double best = 1e30;
    for (int s = 1; s <= 32 && s <= (nt > 0 ? nt : 1); ++s) {
        const int32_t chunk = (nt + s - 1) / s;
        if (s > 1 && (nt + chunk - 1) / chunk != s) continue;
        const double waves = double((planned * ctas * s + kPSms - 1) / kPSms);
        double us = waves * (8.0 + tile_us * chunk);
        if (s > 1) us += 4.0 + merge_rows * s * kPD * 4 * 2 / 4e6;
        if (us < best) {
            best = us;
            p.chunk = chunk > 0 ? chunk : 1;
        }
    }
    p.splits = nt > p.chunk ? (nt + p.chunk - 1) / p.chunk : 1;
    p.grid = most * p.splits;
    if (p.splits > 1 && n_req <= kPSlotReqs && p.chunk < (1 << 16)) {
        const int cap = p.splits < 16 ? 2 * p.splits : 32;
        p.chunk_min = (nt + cap - 1) / cap;
        p.splits = (nt + p.chunk_min - 1) / p.chunk_min;
        p.slots = kPSms / ctas;
        const int64_t full = most * p.splits < p.slots ? most * p.splits : p.slots;
        p.grid = p.grid > full ? p.grid : full;
    }
    p.grid *= ctas;
    return p;
}
struct PagedPlan {
    PagedShare tiles, few;
    int32_t span, few_rows, tail;
    size_t tile_lse, tile_o, few_lse, few_o, tile_at, flags, total;
};
constexpr size_t kPMaxTileBytes = size_t(4) << 30;
constexpr int32_t kPFewRows = 256, kPFewTiles = 4;
static PagedPlan paged_plan(int64_t n_tokens, int n_heads, int64_t n_req, int32_t max_q, int32_t max_kv, int window) {
    PagedPlan p{};
    if (window >= max_kv) window = 0;
    if (max_q > n_tokens) max_q = int32_t(n_tokens);
    const int64_t rows = n_tokens * n_heads;
    const int32_t tile_keys = paged_key_tiles(max_q, max_kv, window, paged_item_tokens(n_heads, 256));
    if (int64_t(max_q) * n_heads > kPFewRows && tile_keys > kPFewTiles) {
        int64_t span = (max_kv + kPN - 1) / kPN;
        if (window > 0) {  // from the first token's window to the last token
            const int64_t w = (int64_t(window) + max_q + 7 + kPN - 1) / kPN;
            span = span < w ? span : w;
        }
        if (n_req <= 65535 && size_t(n_req) * size_t(span) * kPTileBytes <= kPMaxTileBytes) p.span = int32_t(span);
    }
    auto items = [&](int32_t q, int32_t item) {  // each request rounds up
        const int64_t all = rows / item + n_req, each = n_req * paged_items(q, n_heads, item);
        return all < each ? all : each;
    };
    if (p.span > 0) {
        const int64_t n = items(max_q, 256);
        p.tiles = paged_share(n, n, 4, n_req, tile_keys, 1.9, double(rows));
    }
    const bool beside = p.span > 0;
    const int64_t tile_items = p.tiles.grid / 4;
    int32_t tail = 0, tail_splits = 1;
    if (n_req == 1 && beside && p.tiles.splits == 1) paged_tail(int32_t(tile_items), tile_keys, tail, tail_splits);
    if (tail > 0) {  // by the bounds: the kernel goes by the request, which may have fewer items
        p.tail = 1;
        p.tiles.grid = (tile_items + kPTailSlots - 1) / kPTailSlots * kPTailSlots * 4;
    }
    const int64_t padded = n_req * max_q;
    if (!beside || n_tokens <= padded / 6 || (tile_keys >= 16 && n_tokens <= padded / 4 * 3)) {
        const int32_t q = beside ? kPFewRows / n_heads : max_q;
        p.few_rows = beside ? q * n_heads : 0;
        const int64_t most = items(q, 64), planned = beside ? n_req * paged_items(1, n_heads, 64) : most;  // single tokens
        p.few = paged_share(planned, most, 1, n_req, paged_key_tiles(q, max_kv, window, paged_item_tokens(n_heads, 64)), 2.9,
                            beside ? double(n_req) * n_heads : double(rows));
    }
    size_t at = CSA2_STATUS_BYTES;
    auto partials = [&](const PagedShare& h, int64_t n, size_t& lse, size_t& o) {
        lse = at;
        if (h.splits > 1) at = align256(at + size_t(h.splits) * size_t(n) * 4);
        o = at;
        if (h.splits > 1) at = align256(at + size_t(h.splits) * size_t(n) * kPD * 4);
    };
    if (p.tail) {  // no more than kPTailSlots pieces of an item
        PagedShare whole = p.tiles;
        whole.splits = 2;
        partials(whole, kPTailSlots / 2 * 256, p.tile_lse, p.tile_o);
    } else {
        partials(p.tiles, rows, p.tile_lse, p.tile_o);
    }
    partials(p.few, beside ? n_req * p.few_rows : rows, p.few_lse, p.few_o);
    p.flags = at;
    at = align256(at + size_t(n_req) * p.span * kPFlagBytes);
    p.tile_at = at;
    at += size_t(n_req) * p.span * kPTileBytes;
    p.total = at;
    return p;
}

static bool paged_sizes(int64_t n_tokens, int n_heads, int64_t n_req, int32_t max_q, int32_t max_kv, int window) {
    return n_tokens >= 0 && n_tokens <= (int64_t(1) << 22) && n_heads >= 1 && n_heads <= 128 && n_req >= 0 &&
           n_req <= (1 << 20) && max_q >= 0 && max_kv >= 0 && max_kv <= (1 << 30) && window >= 0;
}

}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_paged_attn_workspace_bytes(int64_t n_tokens, int n_heads, int64_t n_req, int32_t max_q,
                                                  int32_t max_kv, int window) {
    return paged_sizes(n_tokens, n_heads, n_req, max_q, max_kv, window)
               ? paged_plan(n_tokens, n_heads, n_req, max_q, max_kv, window).total
               : 0;
}

extern "C" csa2_status csa2_paged_attn(const void* q_bf16, int64_t n_tokens, int n_heads, const int32_t* q_start,
                                       const int32_t* kv_len, int64_t n_req, int32_t max_q, int32_t max_kv, int fmt,
                                       const uint8_t* codes, const uint8_t* scales, int64_t n_rows, const int32_t* table,
                                       int64_t max_pages, int page_size, int window, float sm_scale, void* out,
                                       float* out_lse, void* ws, size_t ws_bytes, csa2_stream_t stream) {
    if (n_tokens < 0 || n_req < 0 || max_q < 0 || max_kv < 0 || window < 0 || n_rows < 0 || max_pages < 0 ||
        max_pages > INT32_MAX)
        return CSA2_ERR_INVALID_ARG;
    if (!(sm_scale > 0.f) || !(sm_scale < FLT_MAX)) return CSA2_ERR_INVALID_ARG;
    if (!paged_sizes(n_tokens, n_heads, n_req, max_q, max_kv, window)) return CSA2_ERR_UNSUPPORTED;
    if (page_size < 8 || page_size > 65536 || page_size % 8) return CSA2_ERR_UNSUPPORTED;
    if (fmt != CSA2_FMT_FP4 && fmt != CSA2_FMT_FP8) return CSA2_ERR_UNSUPPORTED;
    if ((fmt == CSA2_FMT_FP4) != (scales != nullptr)) return CSA2_ERR_INVALID_ARG;
    if (!q_bf16 || !q_start || !kv_len || !codes || !table || !out) return CSA2_ERR_INVALID_ARG;
    for (const void* p : {q_bf16, static_cast<const void*>(q_start), static_cast<const void*>(kv_len),
                          static_cast<const void*>(codes), static_cast<const void*>(scales),
                          static_cast<const void*>(table), static_cast<const void*>(out),
                          static_cast<const void*>(out_lse)})
        if (!aligned16(p)) return CSA2_ERR_INVALID_ARG;
    const PagedPlan plan = paged_plan(n_tokens, n_heads, n_req, max_q, max_kv, window);
    if (!ws || !aligned16(ws) || ws_bytes < plan.total) return CSA2_ERR_WORKSPACE;
    if (n_tokens == 0 || n_req == 0 || max_q == 0) return CSA2_OK;
    const size_t bytes = size_t(n_tokens) * n_heads * kPD * 2;  // of the queries and of the outputs
    const char *q0 = static_cast<const char*>(q_bf16), *o0 = static_cast<const char*>(out);
    if (o0 < q0 + bytes && q0 < o0 + bytes) return CSA2_ERR_INVALID_ARG;
    cudaStream_t s = cudaStream_t(stream);
    if (plan.tiles.grid > INT32_MAX || plan.few.grid > INT32_MAX) return CSA2_ERR_UNSUPPORTED;
    PagedArgs a{};
    a.q = static_cast<const uint8_t*>(q_bf16);
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.codes = codes;
    a.scales = scales;
    a.table = table;
    a.out = static_cast<uint8_t*>(out);
    a.lse = out_lse;
    a.st = static_cast<Status*>(ws);
    a.wlim = wait_limit_ns();
    a.n_rows_pages = n_rows / page_size;
    a.max_pages = max_pages;
    a.rows = n_tokens * n_heads;
    a.n_req = n_req;
    a.n_tokens = int32_t(n_tokens);
    a.heads = n_heads;
    a.max_q = max_q;
    a.max_kv = max_kv;
    a.page = page_size;
    a.window = window >= max_kv ? 0 : window;
    a.by_heads = fast_div(uint32_t(n_heads));
    a.by_page = fast_div(uint32_t(page_size));
    a.sm_scale = sm_scale;
    char* w = static_cast<char*>(ws);
    auto share = [&](PagedArgs& b, const PagedShare& p, int32_t item, int32_t item_log2, size_t lse, size_t o) {
        b.chunk = p.chunk;
        b.chunk_min = p.chunk_min;
        b.slots = p.slots;
        b.chunk_out = reinterpret_cast<int32_t*>(w + CSA2_STATUS_BYTES / 2) + (item == 64);
        b.item = item;
        b.item_log2 = item_log2;
        b.item_tokens = paged_item_tokens(n_heads, item);
        b.part_lse = reinterpret_cast<float*>(w + lse);
        b.part_o = reinterpret_cast<float*>(w + o);
        b.part_rows = a.rows;
    };
    PagedArgs few = a;
    const bool both = plan.tiles.grid > 0 && plan.few.grid > 0;
    share(few, plan.few, 64, 6, plan.few_lse, plan.few_o);
    few.rows_to = both ? kPFewRows : INT32_MAX;
    if (both) {
        few.behind = 1;
        few.few_rows = plan.few_rows;
        few.by_few = fast_div(uint32_t(plan.few_rows));
        few.part_rows = n_req * plan.few_rows;
    }
    share(a, plan.tiles, 256, 8, plan.tile_lse, plan.tile_o);
    a.tiles = reinterpret_cast<uint8_t*>(w + plan.tile_at);
    a.flags = reinterpret_cast<uint8_t*>(w + plan.flags);
    a.span = plan.span;
    a.rows_over = both ? kPFewRows : 0;
    a.tail = plan.tail;
    if (plan.tail) a.part_rows = kPTailSlots / 2 * 256;  // rows that may have been split
    a.rows_to = plan.tiles.grid > 0 ? INT32_MAX : 0;
    const bool fp8 = fmt == CSA2_FMT_FP8;
    csa2_status e = CSA2_OK;
    if (plan.tiles.grid > 0) e = paged_tiles_launch(a, fp8, unsigned(plan.tiles.grid), s);
    if (e == CSA2_OK && plan.few.grid > 0) e = paged_rows_launch(few, fp8, unsigned(plan.few.grid), s);
    if (e != CSA2_OK) {
        cudaGetLastError();
        return e;
    }
    for (const PagedArgs* b : {&a, &few}) {
        if ((b == &a ? plan.tiles : plan.few).splits == 1 && !b->tail) continue;
        timer_begin(K_PAGED_MERGE, s);
        launch(paged_merge_kernel, dim3(unsigned(ceil_div<int64_t>(b->part_rows, paged_merge_rows(*b)))), 256, 0, s, 1, *b);
        timer_end(K_PAGED_MERGE, s);
    }
    return launch_status();
}
