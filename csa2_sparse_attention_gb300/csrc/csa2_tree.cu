// Trees of drafted tokens: positions and ancestor masks before a step, and the
// commit of the accepted path after it.
#include "csa2_common.cuh"
#include "csa2_timer.cuh"

namespace csa2 {

constexpr int kTreeMost = CSA2_TREE_NODES;  // nodes of a request
constexpr int kTreeThreads = 128;

// A request's nodes [q0, q0 + nq) and the position of the first one; nq is 0
// where it has none, or a token bound does not hold.  Without `good`, which such
// a bound and a length that does not hold take (recorded), `first` is anything.
struct TreeReq {
    int32_t q0, nq, first, len;
    bool good;
};
__device__ __forceinline__ TreeReq tree_request(const int32_t* q_start, const int32_t* kv_len, int64_t r, int64_t n_tokens,
                                                int32_t max_q, int64_t max_len, Status* st) {
    TreeReq o;
    o.q0 = q_start[r];
    const int32_t q1 = q_start[r + 1];
    o.len = kv_len[r];
    o.nq = int32_t(uint32_t(q1) - uint32_t(o.q0));  // (bounds may be anything, and the differences wrap around)
    o.first = int32_t(uint32_t(o.len) - uint32_t(o.nq));
    o.good = o.q0 >= 0 && q1 >= o.q0 && q1 <= n_tokens && o.nq <= max_q;
    if (!o.good) o.nq = 0;
    if (o.good && (o.len < o.nq || o.len > max_len)) o.good = false;
    if (!o.good && threadIdx.x == 0) record(st, CSA2_ERR_DEVICE_BOUNDS, CHK_LENGTH, int32_t(r), o.nq == 0 ? q1 : o.len);
    return o;
}

// Positions and masks: a block per request, a thread per node.  A warp has the
// nodes of one word of a mask: five rounds of pointer jumping by shuffles give each
// its ancestors within the word and the nearest one before it.  A row is then a walk
// from word to word, at most 32 dependent loads from shared memory however deep
// the tree is (from node to node it was one for each, on lanes that part ways: a
// chain of 1024 took 217 us).
//
// Bound by the launch: 16 x 8 and 8 x 64 nodes 1.6 us, 192 x 61 1.8, a chain of
// 1024 18 (its rows' words, a node's behind one another, go out one by one).
__global__ void __launch_bounds__(kTreeMost) tree_plan_kernel(const int32_t* __restrict__ parent,
                                                              const int32_t* __restrict__ q_start,
                                                              const int32_t* __restrict__ kv_len, int64_t n_tokens,
                                                              int32_t max_q, int32_t window, int64_t* __restrict__ pos,
                                                              uint32_t* __restrict__ mask, int32_t words, Status* st) {
    __shared__ uint32_t within[kTreeMost];  // a node and its ancestors of the same word
    __shared__ int16_t before[kTreeMost];   // the nearest ancestor of an earlier word; -1: none; -2: lost, a parent was bad
    grid_dep_wait();
    grid_dep_launch();
    const int64_t r = blockIdx.x;
    const TreeReq t = tree_request(q_start, kv_len, r, n_tokens, max_q, INT32_MAX, st);
    const int i = threadIdx.x;  // (a block has a thread for each of max_q nodes)
    int up = -1;
    if (i < t.nq) {
        up = parent[t.q0 + i];
        const bool ok = up >= -1 && up < i;
        if (!ok) record(st, CSA2_ERR_DEVICE_BOUNDS, CHK_PARENT, t.q0 + i, up);
        if (!ok || !t.good) up = -2;
    }
    uint32_t bits = 1u << (i & 31);
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        const uint32_t its = __shfl_sync(0xffffffffu, bits, up & 31);
        const int next = __shfl_sync(0xffffffffu, up, up & 31);
        if (up >= 0 && (up ^ i) < 32) bits |= its, up = next;
    }
    within[i] = bits;
    before[i] = int16_t(up);
    __syncthreads();
    if (i >= t.nq) return;
    uint32_t* row = mask + int64_t(t.q0 + i) * words;
    int depth = 0, at = i, left = window > 0 ? window : kTreeMost;  // nodes that a window leaves, the nearest ones
    for (int w = words - 1; w >= 0; --w) {
        uint32_t b = 0;
        if (at >> 5 == w) {
            b = within[at];
            at = before[at];
            const int n = __popc(b);
            depth += n;
            for (int k = left; k < n; ++k) b &= b - 1;
            left = left > n ? left - n : 0;
        }
        row[w] = b;
    }
    if (at == -2)  // sees nothing
        for (int w = 0; w < words; ++w) row[w] = 0;
    pos[t.q0 + i] = at == -2 ? -1 : int64_t(t.first) + depth - 1;
}

struct CommitArgs {
    const int32_t* parent;
    const int64_t* token;
    const int64_t* choice;
    const int32_t* q_start;
    const int32_t* kv_len;
    uint8_t* codes;
    uint8_t* scales;
    const int32_t* table;
    int32_t* free_pages;
    const int32_t* n_free;
    int32_t* n_free_out;
    int32_t* cached;
    int32_t* path;
    int32_t* accepted;
    int64_t* next;
    Status* st;
    unsigned long long* ticket;  // blocks that came by << 32 | pages that they give back
    int64_t n_req, n_tokens, row_pages, max_pages, n_pages;
    int32_t max_q, page, code_chunks, chunks;  // 16-byte chunks of a row's codes, and of codes and scales
};

constexpr int kCommitRows = 32, kCommitHeld = 8;  // rows moved at a time; chunks that a thread holds of them

__device__ __forceinline__ int64_t commit_pages(int64_t n, int page) { return (n + page - 1) / page; }

// A block per request.  Every node looks whether it continues its parent: the
// lowest one that does is kept in shared memory, so the path is a walk of a few
// dependent shared loads.  Its rows move down by batches, all of a batch loaded
// before any is stored: node path[j] >= j, so what a batch stores no later batch
// loads.  The last block to come by gives the pages back, in the order that undoes
// the plan's taking: the ticket carries the number of pages beside the blocks', and
// the place of a request's pages is a scan.
//
// Bound by a chain of dependent accesses: bounds, then nodes and table together,
// walk, rows; in the last block lengths, table, free list.  16 x 8 nodes 6.6 us, 192 x
// 61 9.9 (tables read twice over and counted by the last block: 7.4 and 13).
__global__ void __launch_bounds__(kTreeThreads) tree_commit_kernel(const CommitArgs a) {
    __shared__ int64_t choice[kTreeMost];
    __shared__ int32_t best[kTreeMost];
    __shared__ int16_t path[kTreeMost];
    __shared__ int32_t pages[kTreeMost / 8 + 1];  // of the step's entries
    __shared__ int64_t src[kCommitRows], dst[kCommitRows];
    __shared__ int32_t sums[kTreeThreads / 32];
    __shared__ int s_len;
    __shared__ unsigned s_total;
    __shared__ bool last;
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
    const int64_t r = blockIdx.x;
    const TreeReq t = tree_request(a.q_start, a.kv_len, r, a.n_tokens, a.max_q, a.max_pages * a.page, a.st);
    const bool some = t.good && t.nq > 0;
    const int page0 = some ? t.first / a.page : 0, n_pages = some ? (t.len - 1) / a.page - page0 + 1 : 0;
    for (int j = tid; j < n_pages; j += kTreeThreads) {
        const int32_t id = a.table[r * a.max_pages + page0 + j];
        if (id < 0 || id >= a.n_pages || (a.codes != nullptr && id >= a.row_pages))
            record(a.st, CSA2_ERR_DEVICE_BOUNDS, CHK_PAGE, int32_t(r), id);
        pages[j] = id;
    }
    if (some) {
        int32_t p[kTreeMost / kTreeThreads];
        int64_t tok[kTreeMost / kTreeThreads];
#pragma unroll
        for (int k = 0; k < kTreeMost / kTreeThreads; ++k) {
            const int i = tid + k * kTreeThreads;
            if (i < t.nq) p[k] = a.parent[t.q0 + i], tok[k] = a.token[t.q0 + i], choice[i] = a.choice[t.q0 + i], best[i] = INT32_MAX;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTreeMost / kTreeThreads; ++k) {
            const int i = tid + k * kTreeThreads;
            if (i >= t.nq) break;
            if (p[k] < -1 || p[k] >= i) record(a.st, CSA2_ERR_DEVICE_BOUNDS, CHK_PARENT, t.q0 + i, p[k]);
            else if (p[k] >= 0 && tok[k] == choice[p[k]]) atomicMin(&best[p[k]], i);
        }
        if (tid == 0) s_len = p[0];  // (0's parent)
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0;
        if (lane == 0) {
            if (some && s_len == -1)
                for (int32_t at = 0; at != INT32_MAX; at = best[at]) path[n++] = int16_t(at);
            a.accepted[r] = n;
            a.next[r] = n > 0 ? choice[path[n - 1]] : -1;
            if (some) a.cached[r] = t.first + n;
            __threadfence();
        }
        n = __shfl_sync(0xffffffffu, n, 0);
        unsigned back = 0;  // pages that hold no kept entry
        // (none of a request whose bounds do not hold: `first` may be anything then, and `pages` holds nothing)
        const int back0 = some ? int(commit_pages(t.first + n, a.page)) - page0 : 0;
        for (int j = back0 + lane; j < n_pages; j += 32) back += pages[j] >= 0 && pages[j] < a.n_pages;
        back = __reduce_add_sync(0xffffffffu, back);
        if (lane == 0) {
            s_len = n;
            const unsigned long long was = atomicAdd(a.ticket, (1ull << 32) + back);
            last = unsigned(was >> 32) == gridDim.x - 1;
            s_total = unsigned(was) + back;
            if (last) *a.ticket = 0;
        }
    }
    __syncthreads();
    const int len = s_len;
    for (int i = tid; i < t.nq; i += kTreeThreads) a.path[t.q0 + i] = i < len ? path[i] : -1;
    // ---- rows, from the first one that moves
    if (a.codes != nullptr) {
        int j0 = 0;
        while (j0 < len && path[j0] == j0) ++j0;
        for (; j0 < len; j0 += kCommitRows) {
            const int n = len - j0 < kCommitRows ? len - j0 : kCommitRows;
            if (tid < 2 * n) {  // rows of the cache, -1 where a page is none
                const int j = j0 + (tid >> 1);
                const int32_t p = t.first + (tid & 1 ? path[j] : j), page = p / a.page, id = pages[page - page0];
                (tid & 1 ? src : dst)[tid >> 1] = id >= 0 && id < a.row_pages ? int64_t(id) * a.page + (p - page * a.page) : -1;
            }
            __syncthreads();
            uint4 v[kCommitHeld];
            auto place = [&](int i, const int64_t* rows) -> uint4* {
                const int j = i / a.chunks, c = i - j * a.chunks;
                return c < a.code_chunks ? reinterpret_cast<uint4*>(a.codes) + rows[j] * a.code_chunks + c
                                         : reinterpret_cast<uint4*>(a.scales) + rows[j] * (a.chunks - a.code_chunks) + c - a.code_chunks;
            };
            auto moved = [&](int i) { return i < n * a.chunks && src[i / a.chunks] >= 0 && dst[i / a.chunks] >= 0; };
#pragma unroll
            for (int k = 0; k < kCommitHeld; ++k) {
                const int i = tid + k * kTreeThreads;
                if (moved(i)) v[k] = *place(i, src);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kCommitHeld; ++k) {
                const int i = tid + k * kTreeThreads;
                if (moved(i)) *place(i, dst) = v[k];
            }
            __syncthreads();
        }
    }
    // ---- pages, by the last block
    if (!last) return;
    __threadfence();
    const int64_t have = *a.n_free, total = s_total;
    if (have < 0 || have + total > a.n_pages) {  // a free list that has no room for them: nothing goes back
        if (tid == 0) {
            record(a.st, CSA2_ERR_DEVICE_BOUNDS, CHK_CAPACITY, 2, int32_t(have));
            *a.n_free_out = int32_t(have);
        }
        return;
    }
    int64_t base = have + total;  // a request's pages end there
    for (int64_t r0 = 0; r0 < a.n_req; r0 += kTreeThreads) {
        const int64_t q = r0 + tid;
        const int32_t* ids = a.table + q * a.max_pages;
        int64_t from = 0, to = 0;
        int32_t mine = 0;
        if (q < a.n_req) {
            const int32_t q0 = a.q_start[q], q1 = a.q_start[q + 1], kv = a.kv_len[q], kept = __ldcg(a.accepted + q);
            const bool good = q0 >= 0 && q1 > q0 && q1 <= a.n_tokens && q1 - q0 <= a.max_q && kv >= q1 - q0 && kv <= a.max_pages * a.page;
            if (good) from = commit_pages(kv - (q1 - q0) + kept, a.page), to = commit_pages(kv, a.page);
            for (int64_t j = from; j < to; ++j) mine += ids[j] >= 0 && ids[j] < a.n_pages;
        }
        int32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) sums[warp] = inc;
        __syncthreads();
        int32_t before = 0, all = 0;
        for (int w = 0; w < kTreeThreads / 32; ++w) {
            if (w < warp) before += sums[w];
            all += sums[w];
        }
        __syncthreads();
        int64_t at = base - (before + inc - mine);
        for (int64_t j = from; j < to; ++j)
            if (ids[j] >= 0 && ids[j] < a.n_pages) a.free_pages[--at] = ids[j];
        base -= all;
    }
    if (tid == 0) *a.n_free_out = int32_t(have + total);
}

}  // namespace csa2

using namespace csa2;

extern "C" csa2_status csa2_tree_plan(const int32_t* parent, const int32_t* q_start, const int32_t* kv_len, int64_t n_req,
                                      int64_t n_tokens, int32_t max_q, int window, int64_t* pos, uint32_t* mask, int mask_words,
                                      void* ws, size_t ws_bytes, csa2_stream_t stream) {
    if (n_req < 0 || n_tokens < 0 || max_q < 0 || window < 0) return CSA2_ERR_INVALID_ARG;
    if (n_req > (1 << 20) || n_tokens > (1 << 22) || max_q > kTreeMost) return CSA2_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < CSA2_STATUS_BYTES || !aligned16(ws)) return CSA2_ERR_WORKSPACE;
    if (!parent || !q_start || !kv_len || !pos || !mask || mask_words != ceil_div(max_q, 32)) return CSA2_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(parent), static_cast<const void*>(q_start), static_cast<const void*>(kv_len),
                          static_cast<const void*>(pos), static_cast<const void*>(mask)})
        if (!aligned16(p)) return CSA2_ERR_INVALID_ARG;
    if (n_req == 0 || n_tokens == 0 || max_q == 0) return CSA2_OK;
    // what is written lies apart from what is read and from each other
    const Span out[] = {{pos, 8 * n_tokens}, {mask, n_tokens * mask_words * 4}};
    const Span in[] = {{parent, 4 * n_tokens}, {q_start, 4 * (n_req + 1)}, {kv_len, 4 * n_req}};
    if (!apart(out, in)) return CSA2_ERR_INVALID_ARG;
    cudaStream_t s = cudaStream_t(stream);
    timer_begin(K_TREE_PLAN, s);
    launch(tree_plan_kernel, dim3(unsigned(n_req)), ceil_div(max_q, 32) * 32, 0, s, 1, parent, q_start, kv_len, n_tokens, max_q, window, pos, mask,
           mask_words, static_cast<Status*>(ws));
    timer_end(K_TREE_PLAN, s);
    return launch_status();
}

extern "C" csa2_status csa2_tree_commit(const int32_t* parent, const int64_t* token, const int64_t* choice, const int32_t* q_start,
                                        const int32_t* kv_len, int64_t n_req, int64_t n_tokens, int32_t max_q, int fmt,
                                        uint8_t* codes, uint8_t* scales, int64_t n_rows, const int32_t* table, int64_t max_pages,
                                        int page_size, int32_t* free_pages, int64_t n_pages, const int32_t* n_free,
                                        int32_t* n_free_out, int32_t* cached, int32_t* path, int32_t* accepted, int64_t* next,
                                        void* ws, size_t ws_bytes, csa2_stream_t stream) {
    if (n_req < 0 || n_tokens < 0 || max_q < 0 || n_rows < 0 || max_pages < 0 || max_pages > INT32_MAX || n_pages < 0 ||
        n_pages > INT32_MAX)
        return CSA2_ERR_INVALID_ARG;
    if (n_req > (1 << 20) || n_tokens > (1 << 22) || max_q > kTreeMost) return CSA2_ERR_UNSUPPORTED;
    if (page_size < 8 || page_size > 65536 || page_size % 8) return CSA2_ERR_UNSUPPORTED;
    if (codes && fmt != CSA2_FMT_FP4 && fmt != CSA2_FMT_FP8) return CSA2_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < CSA2_STATUS_BYTES || !aligned16(ws)) return CSA2_ERR_WORKSPACE;
    if (codes ? (fmt == CSA2_FMT_FP4) != (scales != nullptr) : scales != nullptr) return CSA2_ERR_INVALID_ARG;
    if (!q_start || !kv_len || !table || !free_pages || !n_free || !n_free_out || !cached || !accepted || !next) return CSA2_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!parent || !token || !choice || !path)) return CSA2_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(parent), static_cast<const void*>(token), static_cast<const void*>(choice),
                          static_cast<const void*>(q_start), static_cast<const void*>(kv_len), static_cast<const void*>(codes),
                          static_cast<const void*>(scales), static_cast<const void*>(table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(cached), static_cast<const void*>(path), static_cast<const void*>(accepted),
                          static_cast<const void*>(next)})
        if (!aligned16(p)) return CSA2_ERR_INVALID_ARG;
    for (const int32_t* p : {n_free, static_cast<const int32_t*>(n_free_out)})  // (one number, which may lie among others)
        if (reinterpret_cast<uintptr_t>(p) % sizeof(int32_t)) return CSA2_ERR_INVALID_ARG;
    if (n_req == 0) return CSA2_OK;
    // what is written lies apart from what is read and from each other (blocks read what others are done with)
    const int64_t row_codes = fmt == CSA2_FMT_FP4 ? 256 : 512;
    const Span out[] = {{codes, codes ? n_rows * row_codes : 0}, {scales, scales ? n_rows * 32 : 0}, {free_pages, 4 * n_pages},
                            {n_free_out, 4}, {cached, 4 * n_req}, {path, 4 * n_tokens}, {accepted, 4 * n_req}, {next, 8 * n_req}};
    const Span in[] = {{parent, 4 * n_tokens}, {token, 8 * n_tokens}, {choice, 8 * n_tokens}, {q_start, 4 * (n_req + 1)},
                           {kv_len, 4 * n_req}, {table, 4 * n_req * max_pages}, {n_free, n_free == n_free_out ? 0 : 4}};
    if (!apart(out, in)) return CSA2_ERR_INVALID_ARG;
    CommitArgs a{};
    a.parent = parent;
    a.token = token;
    a.choice = choice;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.codes = codes;
    a.scales = scales;
    a.table = table;
    a.free_pages = free_pages;
    a.n_free = n_free;
    a.n_free_out = n_free_out;
    a.cached = cached;
    a.path = path;
    a.accepted = accepted;
    a.next = next;
    a.st = static_cast<Status*>(ws);
    a.ticket = reinterpret_cast<unsigned long long*>(static_cast<char*>(ws) + 64);
    a.n_req = n_req;
    a.n_tokens = n_tokens;
    a.row_pages = n_rows / page_size;
    a.max_pages = max_pages;
    a.n_pages = n_pages;
    a.max_q = max_q;
    a.page = page_size;
    a.code_chunks = fmt == CSA2_FMT_FP4 ? 16 : 32;
    a.chunks = fmt == CSA2_FMT_FP4 ? 18 : 32;
    cudaStream_t s = cudaStream_t(stream);
    timer_begin(K_TREE_COMMIT, s);
    launch(tree_commit_kernel, dim3(unsigned(n_req)), kTreeThreads, 0, s, 1, a);
    timer_end(K_TREE_COMMIT, s);
    return launch_status();
}
