// Block tables, slot maps and positions of a step over a paged cache, from
// the requests' lengths on the device.
//
// One launch.  Every CTA adds up the lengths itself (8 bytes per request,
// from L2) and so needs no exchange with the others: a first pass gives the
// totals that decide whether the step can be served, a second one walks the
// requests 256 at a time with a block scan of (new tokens, new pages) and
// writes the CTA's share of the tokens, 16 bytes each.  The token that opens
// a page also writes the page's table entry.
#include "csa2_common.cuh"
#include "csa2_timer.cuh"

namespace csa2 {

constexpr int kPlanThreads = 256;

// Pages that hold `n` entries.
__device__ __forceinline__ int64_t pages_of(int64_t n, int page) { return (n + page - 1) / page; }

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(
    const int32_t* __restrict__ cached, const int32_t* __restrict__ added, int64_t n_req, int page, int32_t* table,
    int64_t max_pages, const int32_t* __restrict__ free_pages, int64_t n_pages, const int32_t* n_free,
    int32_t* n_free_out, int32_t* __restrict__ q_start, int32_t* __restrict__ kv_len, int64_t* __restrict__ slots,
    int64_t* __restrict__ pos, int64_t max_new, int64_t per_cta, Status* st, unsigned* ticket) {
    __shared__ long long red[3][kPlanThreads / 32];
    __shared__ int32_t s_end[kPlanThreads];    // tokens up to and with request i of the chunk, from the chunk's first
    __shared__ int32_t s_cached[kPlanThreads];
    __shared__ int64_t s_first[kPlanThreads];  // new pages of every earlier request
    __shared__ bool last;
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
    const int64_t have = *n_free;

    // totals and the first bad request
    long long tok = 0, pg = 0, bad = n_req;
    for (int64_t r = tid; r < n_req; r += kPlanThreads) {
        const int64_t c = cached[r], a = added[r];
        if (c < 0 || a < 0 || c + a > max_pages * page || c + a > INT32_MAX) {
            bad = bad < r ? bad : r;
        } else {
            tok += a;
            pg += pages_of(c + a, page) - pages_of(c, page);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        tok += __shfl_xor_sync(0xffffffffu, tok, o);
        pg += __shfl_xor_sync(0xffffffffu, pg, o);
        const long long b = __shfl_xor_sync(0xffffffffu, bad, o);
        bad = b < bad ? b : bad;
    }
    if (lane == 0) red[0][warp] = tok, red[1][warp] = pg, red[2][warp] = bad;
    __syncthreads();
    tok = pg = 0;
    bad = n_req;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        tok += red[0][w];
        pg += red[1][w];
        bad = red[2][w] < bad ? red[2][w] : bad;
    }
    const bool fits = bad == n_req && tok <= max_new && have >= 0 && have <= n_pages && pg <= have;
    if (!fits && blockIdx.x == 0 && tid == 0) {
        if (bad < n_req)
            record(st, CSA2_ERR_DEVICE_BOUNDS, CHK_LENGTH, int32_t(bad), cached[bad] < 0 ? cached[bad] : added[bad]);
        else if (tok > max_new)
            record(st, CSA2_ERR_DEVICE_BOUNDS, CHK_CAPACITY, 0, int32_t(tok > INT32_MAX ? INT32_MAX : tok));
        else
            record(st, CSA2_ERR_DEVICE_BOUNDS, CHK_CAPACITY, 1, int32_t(have));
    }
    if (!fits) tok = pg = 0;

    // the CTA's tokens, and its share of the requests' sums
    const int64_t t0 = int64_t(blockIdx.x) * per_cta;
    const int64_t t1 = t0 + per_cta < max_new ? t0 + per_cta : max_new;
    int64_t tok0 = 0, pg0 = 0;  // sums before the chunk
    for (int64_t r0 = 0, chunk = 0; r0 < n_req; r0 += kPlanThreads, ++chunk) {
        const int64_t r = r0 + tid;
        int64_t c = 0, a = 0, need = 0;
        if (fits && r < n_req) {
            c = cached[r];
            a = added[r];
            need = pages_of(c + a, page) - pages_of(c, page);
        }
        // inclusive block scan of (a, need)
        int64_t sa = a, sn = need;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t ua = __shfl_up_sync(0xffffffffu, sa, o), un = __shfl_up_sync(0xffffffffu, sn, o);
            if (lane >= o) sa += ua, sn += un;
        }
        __syncthreads();  // the previous chunk's reads of the shared arrays
        if (lane == 31) red[0][warp] = sa, red[1][warp] = sn;
        __syncthreads();
        int64_t ta = 0, tn = 0;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) sa += red[0][w], sn += red[1][w];
            ta += red[0][w];
            tn += red[1][w];
        }
        if (chunk % gridDim.x == blockIdx.x && r < n_req) {
            q_start[r + 1] = int32_t(tok0 + sa);
            kv_len[r] = int32_t(c + a);
            if (r == 0) q_start[0] = 0;
        }
        const int64_t lo = t0 > tok0 ? t0 : tok0, hi = t1 < tok0 + ta ? t1 : tok0 + ta;
        if (lo < hi) {  // uniform: tokens of this chunk in the CTA's range
            s_end[tid] = int32_t(sa);
            s_cached[tid] = int32_t(c);
            s_first[tid] = pg0 + sn - need;
            __syncthreads();
            for (int64_t i = lo + tid; i < hi; i += kPlanThreads) {
                const int32_t at = int32_t(i - tok0);
                int b = 0;  // the first request of the chunk that ends behind the token
#pragma unroll
                for (int step = kPlanThreads / 2; step; step >>= 1)
                    if (s_end[b + step - 1] <= at) b += step;
                const int32_t start = b ? s_end[b - 1] : 0, had = s_cached[b];
                const int32_t p = had + (at - start);
                const int32_t idx = p / page, off = p - idx * page, held = int32_t(pages_of(had, page));
                int32_t* entry = table + (r0 + b) * max_pages + idx;
                int32_t id;
                if (idx < held) {
                    id = *entry;
                } else {
                    id = free_pages[have - 1 - (s_first[b] + idx - held)];
                    if (off == 0) *entry = id >= 0 && id < n_pages ? id : -1;
                }
                const bool ok = id >= 0 && id < n_pages;
                if (!ok) record(st, CSA2_ERR_DEVICE_BOUNDS, CHK_PAGE, int32_t(r0 + b), id);
                slots[i] = ok ? int64_t(id) * page + off : -1;
                pos[i] = p;
            }
        }
        tok0 += ta;
        pg0 += tn;
    }
    if (n_req == 0 && blockIdx.x == 0 && tid == 0) q_start[0] = 0;
    for (int64_t i = (t0 > tok ? t0 : int64_t(tok)) + tid; i < t1; i += kPlanThreads) slots[i] = pos[i] = -1;

    // n_free_out may be n_free: the last CTA writes it, when all have read
    if (gridDim.x > 1) {
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            last = atomicAdd(ticket, 1u) == gridDim.x - 1;
            if (last) *ticket = 0;
        }
        __syncthreads();
    }
    if (tid == 0 && (gridDim.x == 1 || last)) *n_free_out = int32_t(have - pg);
}

}  // namespace csa2

using namespace csa2;

extern "C" csa2_status csa2_page_plan(const int32_t* cached, const int32_t* added, int64_t n_req, int page_size,
                                      int32_t* table, int64_t max_pages, const int32_t* free_pages, int64_t n_pages,
                                      const int32_t* n_free, int32_t* n_free_out, int32_t* q_start, int32_t* kv_len,
                                      int64_t* slots, int64_t* pos, int64_t max_new, void* ws, size_t ws_bytes,
                                      csa2_stream_t stream) {
    if (n_req < 0 || n_req > INT32_MAX || max_pages < 0 || max_pages > INT32_MAX || n_pages < 0 ||
        n_pages > INT32_MAX || max_new < 0 || max_new > INT32_MAX)
        return CSA2_ERR_INVALID_ARG;
    if (page_size < 8 || page_size > 65536 || page_size % 8) return CSA2_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < CSA2_STATUS_BYTES || !aligned16(ws)) return CSA2_ERR_WORKSPACE;
    if (!n_free || !n_free_out || !q_start) return CSA2_ERR_INVALID_ARG;
    if (n_req > 0 && (!cached || !added || !kv_len || cached == kv_len || added == kv_len)) return CSA2_ERR_INVALID_ARG;
    if (n_req > 0 && max_pages > 0 && !table) return CSA2_ERR_INVALID_ARG;
    if (n_pages > 0 && !free_pages) return CSA2_ERR_INVALID_ARG;
    if (max_new > 0 && (!slots || !pos)) return CSA2_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(cached), static_cast<const void*>(added),
                          static_cast<const void*>(table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(slots), static_cast<const void*>(pos)})
        if (!aligned16(p)) return CSA2_ERR_INVALID_ARG;
    for (const int32_t* p : {n_free, static_cast<const int32_t*>(n_free_out), static_cast<const int32_t*>(q_start),
                             static_cast<const int32_t*>(kv_len)})
        if (reinterpret_cast<uintptr_t>(p) % sizeof(int32_t)) return CSA2_ERR_INVALID_ARG;
    cudaStream_t s = cudaStream_t(stream);
    // 1024 tokens per CTA (four per thread), at most two CTAs per SM
    int64_t grid = ceil_div<int64_t>(max_new, 1024);
    const int64_t cap = 2 * int64_t(sm_count());
    grid = grid < 1 ? 1 : (grid > cap ? cap : grid);
    const int64_t per_cta = ceil_div<int64_t>(max_new, grid);
    timer_begin(K_PAGE_PLAN, s);
    launch(page_plan_kernel, dim3(unsigned(grid)), kPlanThreads, 0, s, 1, cached, added, n_req, page_size, table, max_pages,
           free_pages, n_pages, n_free, n_free_out, q_start, kv_len, slots, pos, max_new, per_cta, static_cast<Status*>(ws),
           reinterpret_cast<unsigned*>(static_cast<char*>(ws) + 64));
    timer_end(K_PAGE_PLAN, s);
    return launch_status();
}
