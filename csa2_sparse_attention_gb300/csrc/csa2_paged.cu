// Causal attention of each request's new tokens over its paged latents.
//
//   l_p = sm_scale q . c_p,  o = sum_p softmax(l)_p c_p,  c_p a 512-wide
//   latent in FP4 (E2M1, one E4M3 scale per 16 channels) or E4M3
//
// Rows are (token, head) pairs: 128 consecutive rows of a request make a tile
// of the tensor cores' M, whatever the number of heads.  All heads share the
// latents, so a key costs 2048 FLOPs a row against 288 bytes: the tensor cores
// bound the kernel even for single tokens.
//
// The fp32 accumulator of 128 rows x 512 channels would fill TMEM (512
// columns) and leave no room for the logits, so a CTA takes 128 rows and one
// half of the output channels ("own", Y) and computes the logits over both
// halves: 3 products of 256 channels where 2 would do.  (Sharing the logits
// between two CTAs would move 64 KB of fp32 partial logits per 128 keys over
// distributed shared memory at 16-24 B/clk per SM: 2700 clocks or more, against
// the 1060 clocks of tensor time that the third product costs.)
//
//   TMEM  [0, 256) O   [256, 384) S   [384, 512) own half of Q, f16
//   smem  other half of Q (64 KB), two 64 KB groups of latents, P (32 KB)
//
// Keys go in tiles of 128: an M = 128 MMA of K = 16 takes 64 clocks for any
// N up to 128 (measured 64-69) and 128 for N = 256, so S wants 128 keys and O
// 256 channels at once.  Three roles:
//   producers (8 warps)  read the rows through the page table and decode them
//       to f16 (exact) into shared memory, the other half's channels X first,
//       then, as the logits' MMAs release them, the own half's Y in the same
//       group.  One copy of Y serves S (K-major) and O (MN-major).
//   MMA warp, per tile:  S += Q_X X^T, then O += P Y of the previous tile,
//       then S += Q_Y Y^T: the softmax of a tile runs under the next tile's
//       S_X, and the decoding of Y under the previous tile's O.
//   softmax (4 warps, a thread per row)  takes S out of TMEM, keeps the
//       running maximum and sum in fp32, writes P as f16 to shared memory.  O
//       is rescaled only when a row's maximum grew by more than 2^8: P stays
//       below 2^8 and the sums in fp32, so nothing is lost by waiting.
// P is rounded to f16 (2^-11 relative, an eighth of the step of the bf16
// output); Q goes to f16 times a power of two per row (exact down to 2^-28 of
// the row's maximum).
//
// Long axes with few rows are split over CTAs in chunks of key tiles that the
// host sizes; the partial outputs are joined by paged_merge_kernel.
#include "csa2_common.cuh"
#include "csa2_timer.cuh"
#include "csa2_layout.cuh"
#include "csa2_tc.cuh"

#include <atomic>
#include <cfloat>

namespace csa2 {

constexpr int kPD = CSA2_LATENT_DIM;
constexpr int kPHalf = kPD / 2;       // channels of one half
constexpr int kPM = 128;              // rows of a tile
constexpr int kPN = 128;              // keys of a tile
constexpr int kPSoftWarps = 4, kPProdWarps = 8;
constexpr int kPThreads = 32 * (kPSoftWarps + kPProdWarps + 4);  // and a warpgroup for the MMA thread
constexpr int kPTileThreads = 32 * (kPSoftWarps + 4);            // the same without producers (decoded tiles)
// Where the latents come from: rows in pages, or tiles that paged_decode_kernel
// laid out as shared memory holds them: per half [16 key groups][32 chunks of 8
// channels][8 keys][16 bytes], f16.
enum { kSrcFp4 = 0, kSrcFp8 = 1, kSrcTiles = 2 };
constexpr int64_t kPTileBytes = int64_t(kPN) * kPD * 2;
constexpr int kPFlagBytes = 32;       // per tile: 128 bits of keys without a page, 128 bits of keys with NaN
// Registers per thread: the launch gives 128 x 512; the warpgroups pass them
// on as 208 + 2 x 120 + 64 = 512 = 4 x 128.  No role spills: the latents
// stream through what L1 the shared memory leaves (27 KB), so a spilled value
// came back from L2 (the MMA thread issued one MMA per 300 clocks with its
// descriptors spilled, against 64).
constexpr int kPLaunchRegs = 128, kPSoftRegs = 208, kPProdRegs = 120, kPMmaRegs = 64;
static_assert(kPSoftRegs + 2 * kPProdRegs + kPMmaRegs <= 4 * kPLaunchRegs, "registers");
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 384;
constexpr int kPSms = 152;            // multiprocessors the split is planned for

struct PagedArgs {
    const uint8_t* q;
    const int32_t* q_start;
    const int32_t* kv_len;
    const uint8_t* codes;
    const uint8_t* scales;
    const int32_t* table;
    uint8_t* out;
    float* lse;
    float* part_o;    // [splits][rows][512], each split's normalized output
    float* part_lse;  // [splits][rows], log2 domain
    uint8_t* tiles;   // decoded tiles [n_req][span][128 KB], or null
    uint8_t* flags;   // [n_req][span][32]
    Status* st;
    uint64_t wlim;
    int64_t n_rows_pages;  // pages of the cache
    int64_t max_pages;
    int64_t rows;          // n_tokens * heads
    int64_t n_req;
    int32_t n_tokens, heads, max_q, max_kv, page, window;
    int32_t chunk;         // key tiles per split
    int32_t span;          // decoded tiles per request
    int32_t item;          // rows of a work item: a row tile, or the two of a cluster (decoded tiles)
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
__host__ __device__ inline int32_t paged_items(int32_t nq, int32_t heads, int32_t item) { return (nq * heads + item - 1) / item; }
// Key tiles that a work item of a request can span at most, and its splits.
__host__ __device__ inline int32_t paged_key_tiles(int32_t nq, int32_t len, int32_t heads, int32_t window, int32_t item) {
    int32_t n = (len + kPN - 1) / kPN;
    if (window > 0) {
        const int32_t tok = (item - 1) / heads + 2, span = window + (nq < tok ? nq : tok) + 7;
        const int32_t w = (span + kPN - 1) / kPN + 1;  // and one where the first tile begins early
        n = n < w ? n : w;
    }
    return n;
}
__host__ __device__ inline int32_t paged_splits(int32_t tiles, int32_t chunk) {
    return tiles > chunk ? (tiles + chunk - 1) / chunk : 1;
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
    end = rq.len - rq.nq + r1 / a.heads + 1;
    int32_t lo = a.window > 0 ? rq.len - rq.nq + r0 / a.heads + 1 - a.window : 0;
    if (lo < 0) lo = 0;
    begin = lo & ~7;
    if (a.tiles != nullptr) {
        const int32_t base = paged_base(a, rq);
        begin = base + (begin - base) / kPN * kPN;
    }
    tiles = end > begin ? (end - begin + kPN - 1) / kPN : 0;
}

struct PagedSmem {
    uint8_t qx[kPM * kPHalf * 2];      // other half of Q, K-major: 8-row groups of 4096 B, 8-channel chunks of 128 B
    uint8_t c[2][kPN * kPHalf * 2];    // latents: 8-key groups of 4096 B, 8-channel chunks of 128 B
    uint8_t p[kPM * kPN * 2];          // P: 8-row groups of 2048 B, 8-key chunks of 128 B
    struct alignas(32) {
        uint16_t hidden[8];            // keys of a tile without a page, a bit each
        uint16_t nan[8];               // keys with a NaN latent
    } flags[2];
    float q_scale[kPM];                // logits' scale of each row (log2 domain)
    uint64_t full_x[2][2], full_y[2][2], empty_x[2][2], empty_o[2];
    uint64_t s_full, s_free, p_full, o_done, q_done, drain;
    uint32_t tmem;
    int32_t req, local;
    PagedReq rq;
};
static_assert(sizeof(PagedSmem) + 1024 <= 227 * 1024, "shared memory of the paged attention");
static_assert(kPM * (kPHalf * 4 + 16) <= 2 * kPN * kPHalf * 2 + kPM * kPN * 2, "the epilogue's rows in the latents' and P's place");

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
// Clusters of two CTAs: a barrier of all their threads; an arrival at the other
// CTA's mbarrier; a commit and a bulk copy that reach both (same offsets).
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_peer(uint64_t* bar, uint32_t cta) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(bar)), "r"(cta));
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(at) : "memory");
}
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"(uint16_t(3))
                 : "memory");
}
__device__ __forceinline__ void bulk_g2s_pair(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.multicast::cluster [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "h"(uint16_t(3))
        : "memory");
}
// One bulk copy shared memory -> global (addresses and size multiples of 16
// bytes), and the wait for this thread's copies: written, not only read.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\ncp.async.bulk.commit_group;" ::"l"(dst),
                 "r"(smem_u32(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_s2g_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
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
// nonzero when one of the four E4M3 bytes is NaN (0x7F or 0xFF)
__device__ __forceinline__ uint32_t e4m3_nan4(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// grid: 2 CTAs (output halves) per (row tile, split), row tiles with the most
// keys first; CTAs beyond the last one leave at once.
template <int SRC>
__global__ void __launch_bounds__(SRC == kSrcTiles ? kPTileThreads : kPThreads, 1) paged_attn_kernel(const PagedArgs a) {
    constexpr bool FP8 = SRC == kSrcFp8, TILES = SRC == kSrcTiles;
    constexpr int kMmaWarp = TILES ? kPSoftWarps : kPSoftWarps + kPProdWarps;
    constexpr int kFullCount = TILES ? 1 : kPProdWarps;  // arrivals that fill a block
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    PagedSmem& S = *reinterpret_cast<PagedSmem*>(smem_raw);
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
    // grid.x: work items, halves, and with decoded tiles the two row tiles of a cluster
    const int half = TILES ? (blockIdx.x >> 1) & 1 : blockIdx.x & 1;
    const int rank = TILES ? blockIdx.x & 1 : 0;
    grid_dep_wait();
    grid_dep_launch();

    // ---- the CTA's request: a warp scan of the requests' work items
    if (warp == 0) {
        const int64_t item = blockIdx.x >> (TILES ? 2 : 1);
        int64_t base = 0;
        int32_t req = -1;
        for (int64_t r0 = 0; r0 < a.n_req; r0 += 32) {
            const int64_t r = r0 + lane;
            int64_t items = 0;
            PagedReq rq;
            if (r < a.n_req && paged_request(a, r, rq, blockIdx.x == 0 ? a.st : nullptr))
                items = int64_t(paged_items(rq.nq, a.heads, a.item)) *
                        paged_splits(paged_key_tiles(rq.nq, rq.len, a.heads, a.window, a.item), a.chunk);
            int64_t inc = items;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += u;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, base + inc > item);
            if (hit != 0 && req < 0) {
                const int src = __ffs(hit) - 1;
                req = int32_t(r0) + src;
                if (lane == src) {
                    S.local = int32_t(item - base - (inc - items));
                    S.rq = rq;
                }
                if (blockIdx.x != 0) break;  // the first CTA looks at every request
            }
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) S.req = req;
    }
    __syncthreads();
    if (S.req < 0) return;
    const int64_t req = S.req;
    const PagedReq rq = S.rq;
    const int32_t items_r = paged_items(rq.nq, a.heads, a.item);
    const int32_t ns_r = paged_splits(paged_key_tiles(rq.nq, rq.len, a.heads, a.window, a.item), a.chunk);
    const int32_t it = items_r - 1 - S.local / ns_r, split = S.local % ns_r;
    int32_t k_begin, k_end, k_tiles;
    paged_item_keys(a, rq, it, k_begin, k_end, k_tiles);
    const int32_t splits = paged_splits(k_tiles, a.chunk);
    if (split >= splits) return;
    const int32_t j0 = split * a.chunk;
    const int32_t nt = k_tiles - j0 < a.chunk ? k_tiles - j0 : a.chunk;  // this CTA's key tiles (0: nothing to see)
    const int32_t key0 = k_begin + j0 * kPN;
    // the CTA's row tile (a cluster's second one may be behind the request's rows: it then only helps to copy)
    const int32_t ti = TILES ? 2 * it + rank : it;
    const int32_t n_row = rq.nq * a.heads - ti * kPM < kPM ? rq.nq * a.heads - ti * kPM : kPM;
    const int64_t flat0 = int64_t(rq.q0) * a.heads + (n_row > 0 ? int64_t(ti) * kPM : 0);
    const int x_dim = kPHalf * (1 - half), y_dim = kPHalf * half;

    // ---- Q: 8 rows per warp, four lanes per row (64 contiguous bytes an
    // instruction); the first loads are under way while the CTA sets up
    constexpr int kQWarps = 8;  // all with decoded tiles, else all but the producers
    const int q_warp = TILES || warp < kPSoftWarps ? warp : warp - kPProdWarps;
    const bool q_on = TILES || warp < kPSoftWarps || warp >= kMmaWarp;
    const int q_groups = (n_row + 7) / 8;  // rows behind the last one stay what they are: they reach no other row
    constexpr int QN = TILES ? 2 : 1;      // groups whose loads fit into the registers
    uint4 qv[QN][16];
    auto q_load = [&](int rg, uint4 (&v)[16]) {
        const int row = 8 * rg + (lane & 7);
        const bool on = row < n_row;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (flat0 + (on ? row : 0)) * (kPD * 2)) + (lane >> 3);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = on ? __ldg(src + 4 * i) : make_uint4(0, 0, 0, 0);
    };
    if (q_on) {
#pragma unroll
        for (int n = 0; n < QN; ++n)
            if (q_warp + kQWarps * n < q_groups) q_load(q_warp + kQWarps * n, qv[n]);
    }
    if (tid == 0) {
        for (int g = 0; g < 2; ++g) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(&S.full_x[g][b], kFullCount);
                mbar_init(&S.full_y[g][b], kFullCount);
                mbar_init(&S.empty_x[g][b], TILES ? 2 : 1);  // with clusters: both CTAs' MMAs
            }
            mbar_init(&S.empty_o[g], TILES ? 2 : 1);
        }
        mbar_init(&S.s_full, 1);
        mbar_init(&S.s_free, kPSoftWarps);
        mbar_init(&S.p_full, kPSoftWarps);
        mbar_init(&S.o_done, 1);
        mbar_init(&S.q_done, (TILES ? 2 : 1) * kPSoftWarps);
        mbar_init(&S.drain, TILES ? 2 : 1);
        mbar_init_fence();
    }
    if (warp == kMmaWarp) tmem_alloc(&S.tmem, 512);
    tc_fence_before();
    if (TILES) cluster_sync();  // the other CTA's barriers are initialized as well
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;

    // ---- decoded tiles: a block of 128 channels is 2 KB of each of 16 key
    // groups.  Each CTA of the cluster copies half of them into both: without
    // sharing, 128 KB per key tile and CTA took 7.8 TB/s from L2 and bounded the
    // kernel.
    const int64_t tile0 = TILES ? req * a.span + (key0 - paged_base(a, rq)) / kPN : 0;
    auto copy_block = [&](uint64_t* bar, int g, int b, const uint8_t* src, const uint8_t* fl) {
        if (lane == 0) mbar_arrive_expect_tx(bar, kPN * 128 * 2 + (fl ? kPFlagBytes : 0));
        __syncwarp();
        const int kg = rank * (kPN / 16) + lane;
        if (lane < kPN / 16)
            bulk_g2s_pair(S.c[g] + kg * 4096 + b * 2048, src + kg * 4096 + b * 2048, 2048, bar);
        else if (lane == kPN / 16 && fl && rank == 0)
            bulk_g2s_pair(&S.flags[g], fl, kPFlagBytes, bar);
        __syncwarp();
    };
    const uint8_t* x_src = a.tiles + tile0 * kPTileBytes + (1 - half) * (kPTileBytes / 2);
    if (TILES && warp == kMmaWarp + 1 && nt > 0)
        for (int b = 0; b < 2; ++b) copy_block(&S.full_x[0][b], 0, b, x_src, nullptr);

    // ---- Q to f16 times a power of two per row: the other half to its place, the
    // own half by way of the second group of latents into TMEM
    if (q_on) {
        auto q_store = [&](int rg, const uint4 (&v)[16]) {
            const int row = 8 * rg + (lane & 7), piece = lane >> 3;
            uint32_t am = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                am = __vmaxu2(am, __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu));
                am = __vmaxu2(am, __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
            }
            am = max(am & 0xFFFFu, am >> 16);
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 8));
            am = max(am, __shfl_xor_sync(0xffffffffu, am, 16));
            int qs = am != 0 ? int(am >> 7) - 127 - 14 : 0;  // max |q| 2^-qs in [2^14, 2^15)
            qs = qs < -100 ? -100 : qs;
            const float qf = __uint_as_float(uint32_t(127 - qs) << 23);
            if (piece == 0)
                S.q_scale[row] = fmaxf(a.sm_scale * 1.4426950408889634f * __uint_as_float(uint32_t(127 + qs) << 23), FLT_MIN);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = f16x2(bf16_lo(w[e]) * qf, bf16_hi(w[e]) * qf);
                uint8_t* dst = (i >= 8) == (half == 1) ? S.c[1] : S.qx;  // channels 256 .. 511 are the own half of half 1
                *reinterpret_cast<uint4*>(dst + (row >> 3) * 4096 + (4 * (i & 7) + piece) * 128 + (row & 7) * 16) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
        };
#pragma unroll
        for (int n = 0; n < QN; ++n)
            if (q_warp + kQWarps * n < q_groups) q_store(q_warp + kQWarps * n, qv[n]);
        if (!TILES && q_warp + kQWarps < q_groups) {
            q_load(q_warp + kQWarps, qv[0]);
            q_store(q_warp + kQWarps, qv[0]);
        }
        fence_async_smem();
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kQWarps) : "memory");
    }

    if (warp < kPSoftWarps) {
        if (!TILES) regs_up<kPSoftRegs>();
        // ================= softmax: row = TMEM lane = thread
        const int row = tid;
        const uint32_t tm = tmem + (uint32_t(32 * warp) << 16);
        const bool row_on = row < n_row;
        const float sm_eff = S.q_scale[row];
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {  // the own half of Q into TMEM, 64 channels at a time
            uint32_t o[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(S.c[1] + (row >> 3) * 4096 + (8 * b + i) * 128 + (row & 7) * 16);
                o[4 * i] = v.x, o[4 * i + 1] = v.y, o[4 * i + 2] = v.z, o[4 * i + 3] = v.w;
            }
            tmem_st32(tm + kColQ + 32 * b, o);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&S.q_done);  // the second group of latents may be filled
            if (TILES) mbar_arrive_peer(&S.q_done, rank ^ 1);
            mbar_arrive(&S.s_free);  // phase 0: Q is in place
        }

        // ---- key tiles
        int32_t lo_r = 0, hi_r = INT32_MAX;  // the row's keys
        if (row_on) {
            hi_r = rq.len - rq.nq + (ti * kPM + row) / a.heads + 1;
            lo_r = a.window > 0 ? hi_r - a.window : 0;
        }
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        if (32 * warp >= n_row) {  // no rows: P stays zero
            uint8_t* pd = S.p + (row >> 3) * 2048 + (row & 7) * 16;
#pragma unroll
            for (int i = 0; i < 16; ++i) *reinterpret_cast<uint4*>(pd + i * 128) = make_uint4(0, 0, 0, 0);
            fence_async_smem();
            for (int32_t j = 0; j < nt; ++j) {
                ok = __all_sync(0xffffffffu, mbar_wait(&S.s_full, j & 1, a.wlim));
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive(&S.s_free);
                    mbar_arrive(&S.p_full);
                }
            }
        }
        for (int32_t j = 0; j < nt && 32 * warp < n_row; ++j) {
            ok = __all_sync(0xffffffffu, mbar_wait(&S.s_full, j & 1, a.wlim));
            if (!ok) break;
            tc_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int b = 0; b < 4; ++b) tmem_ld32(tm + kColS + 32 * b, s[b]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.s_free);  // phase j + 1: S may be overwritten
            const int32_t c0 = key0 + j * kPN;
            const int g = j & 1;
            const uint4 hid = *reinterpret_cast<const uint4*>(S.flags[g].hidden);
            const uint4 n4 = *reinterpret_cast<const uint4*>(S.flags[g].nan);
            const uint32_t hidden[4] = {hid.x, hid.y, hid.z, hid.w}, nan[4] = {n4.x, n4.y, n4.z, n4.w};
            if (__any_sync(0xffffffffu, c0 < lo_r || c0 + kPN > hi_r) ||
                (hidden[0] | hidden[1] | hidden[2] | hidden[3] | nan[0] | nan[1] | nan[2] | nan[3]) != 0) {
                const int32_t lo = lo_r - c0, hi = hi_r - c0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    // bits of the block's columns in [lo, hi) that have a page
                    const int32_t l0 = lo - 32 * b, h0 = hi - 32 * b;
                    uint32_t see = l0 >= 32 || h0 <= 0 ? 0u : ~hidden[b];
                    if (l0 > 0 && l0 < 32) see &= 0xFFFFFFFFu << l0;
                    if (h0 > 0 && h0 < 32) see &= 0xFFFFFFFFu >> (32 - h0);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if ((nan[b] >> i) & 1u) s[b][i] = 0x7FC00000u;
                        if (!((see >> i) & 1u)) s[b][i] = 0xFF800000u;
                    }
                }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; i += 2)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    mx[b] = fmaxf(mx[b], fmaxf(__uint_as_float(s[b][i]), __uint_as_float(s[b][i + 1])));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sm_eff;
            const bool grew = top > m + 8.f;
            if (__any_sync(0xffffffffu, grew)) {
                const float mn = grew ? top : m;
                const float alpha = !grew ? 1.f : m == -INFINITY ? 0.f : ex2(m - mn);
                if (j > 0) {  // every MMA before S_Y of this tile is done, the previous O among them
#pragma unroll 1
                    for (int b = 0; b < kPHalf / 32; ++b) {
                        uint32_t o[32];
                        tmem_ld32(tm + kColO + 32 * b, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(tm + kColO + 32 * b, o);
                    }
                    tmem_st_wait();
                }
                l *= alpha;
                m = mn;
            }
            const float mu = m == -INFINITY ? 0.f : m;
            const uint64_t sm2 = f32x2(sm_eff, sm_eff), mu2 = f32x2(-mu, -mu);
            uint64_t acc[4] = {0, 0, 0, 0};
            uint8_t* pd = S.p + (row >> 3) * 2048 + (row & 7) * 16;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x, y;
                        f32x2_out(fma2(f32x2(__uint_as_float(s[b][8 * i + 2 * e]), __uint_as_float(s[b][8 * i + 2 * e + 1])), sm2, mu2), x, y);
                        x = ex2(x);
                        y = ex2(y);
                        acc[e] = add2(acc[e], f32x2(x, y));
                        w[e] = f16x2(x, y);
                    }
                    *reinterpret_cast<uint4*>(pd + (4 * b + i) * 128) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            {
                float x, y;
                f32x2_out(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), x, y);
                l += x + y;
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.p_full);
        }
        if (ok && nt > 0) ok = __all_sync(0xffffffffu, mbar_wait(&S.o_done, 0, a.wlim));
        if (!ok && lane == 0) record(a.st, CSA2_ERR_TIMEOUT, 6, int32_t(req), ti);
        // ---- epilogue: O / l, the row's 256 channels of the own half.  The row
        // is put together in shared memory (the latents' and P's, which the MMAs
        // are done with) and leaves in one bulk copy: 16-byte stores of a row per
        // lane took 5400 clocks.
        if (ok && 32 * warp < n_row) {
            tc_fence_after();
            const float inv = l == 0.f ? 0.f : 1.0f / l;
            const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
            const int64_t flat = flat0 + row;
            const bool whole = splits == 1;
            uint8_t* stage = S.c[0] + row * (whole ? kPHalf * 2 + 16 : kPHalf * 4 + 16);
#pragma unroll 1
            for (int b = 0; b < kPHalf / 32; ++b) {
                uint32_t o[32];
                if (nt > 0) {
                    tmem_ld32(tm + kColO + 32 * b, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0;
                }
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(o[8 * i + 2 * e]) * inv,
                                                                           __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
                            w[e] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                        *reinterpret_cast<uint4*>(stage + b * 64 + i * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4*>(stage + b * 128 + i * 16) =
                            make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                        __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
                }
            }
            fence_async_smem();
            if (row_on) {
                if (whole)
                    bulk_s2g(a.out + (flat * kPD + y_dim) * 2, stage, kPHalf * 2);
                else
                    bulk_s2g(a.part_o + (int64_t(split) * a.rows + flat) * kPD + y_dim, stage, kPHalf * 4);
                if (half == 0) {
                    if (!whole)
                        a.part_lse[int64_t(split) * a.rows + flat] = lse2;
                    else if (a.lse)
                        a.lse[flat] = lse2 * 0.6931471805599453f;
                }
                bulk_s2g_wait();
            }
        }
    } else if (!TILES && warp < kPSoftWarps + kPProdWarps) {
        regs_down<kPProdRegs>();
        // ================= producers: keys 16 pw + (lane % 8) and + 8, piece lane / 8
        // Four lanes read 64 contiguous bytes of a row, eight rows an
        // instruction: a row per lane took 32 passes through the L1 data path
        // for 512 bytes, which the MMAs' operand reads need (3072 passes a tile
        // doubled the MMAs' time).  A quarter-warp stores 8 keys of one chunk:
        // no bank conflicts.  Keys in eights share a page.
        const int pw = warp - kPSoftWarps, k8 = lane & 7, piece = lane >> 3;
        constexpr int NV = FP8 ? 2 : 1;  // 16-byte pieces per key and 128 channels
        uint4 v[4][2][NV];               // the four 128-channel blocks of a tile (X, X, Y, Y) of two keys
        uint2 sc[2];                     // FP4: the scales of block `piece` in channel order
        const int32_t* trow = a.table + req * a.max_pages;
        const uint8_t* src[2];           // the tile being loaded: its keys' codes (from `piece` on), null without a row
        const uint8_t* ssrc[2];          //   and scales
        const int64_t last_page = a.n_rows_pages;
        const int32_t k_last = key0 + nt * kPN < k_end ? key0 + nt * kPN : k_end;  // end of this CTA's keys
        // page ids of the warp's two key groups in 16 tiles, one per lane: a tile's are shuffled out
        int32_t ids = -1;
        // place within its page of the first key of the tile that is located next; a tile on is 128 keys on
        const int32_t step_off = kPN % a.page;
        int32_t off_t = (key0 + 16 * pw) % a.page + k8;  // groups of 8 keys share a page, so this is below it
        auto locate = [&](int32_t j) {
            if ((j & 15) == 0) {
                const int32_t p = key0 + (j + (lane >> 1)) * kPN + 16 * pw + 8 * (lane & 1);
                ids = p < k_last ? trow[p / a.page] : -1;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int32_t id = __shfl_sync(0xffffffffu, ids, 2 * (j & 15) + i);
                const int32_t off = off_t + 8 * i >= a.page ? off_t + 8 * i - a.page : off_t + 8 * i;
                const bool in = key0 + j * kPN + 16 * pw + 8 * i + k8 < k_last;
                src[i] = ssrc[i] = nullptr;
                if (in && id >= 0 && id < last_page) {
                    const int64_t row = int64_t(id) * a.page + off;
                    src[i] = a.codes + row * (FP8 ? kPD : kPD / 2) + 16 * piece;
                    ssrc[i] = a.scales + row * (kPD / 16) + 8 * piece;
                } else if (in && piece == 0 && half == 0) {
                    record(a.st, CSA2_ERR_DEVICE_BOUNDS, CHK_PAGE, int32_t(req), id);
                }
            }
            off_t += step_off;
            if (off_t >= a.page) off_t -= a.page;
        };
        auto load_scales = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                sc[i] = !FP8 && src[i] ? __ldg(reinterpret_cast<const uint2*>(ssrc[i])) : make_uint2(0, 0);
        };
        auto load = [&](int b) {
            const int dim = (b < 2 ? x_dim : y_dim) + 128 * (b & 1);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < NV; ++e)
                    v[b][i][e] = src[i] ? __ldg(reinterpret_cast<const uint4*>(src[i] + (FP8 ? dim : dim / 2)) + 4 * e)
                                        : make_uint4(0, 0, 0, 0);
        };
        locate(0);
        load_scales();
#pragma unroll
        for (int b = 0; b < 4; ++b) load(b);
        uint32_t gone = (src[0] ? 0u : 1u) | (src[1] ? 0u : 2u);
        locate(1);  // always the tile behind the one that is decoded
        bool ok = true;
        for (int32_t j = 0; j < nt && ok; ++j) {
            const int g = j & 1;
            const uint32_t ph = (j >> 1) & 1;
            uint32_t bad[2] = {0, 0};
            const uint2 sc0 = sc[0], sc1 = sc[1];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                // the block's place: X after the O MMAs of the tile before last (in the second group: after Q's
                // own half has left it), Y after this tile's S_X MMAs
                if (b == 0 && j >= 1)
                    ok = __all_sync(0xffffffffu, j == 1 ? mbar_wait(&S.q_done, 0, a.wlim) : mbar_wait(&S.empty_o[g], ph ^ 1, a.wlim));
                if (b >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&S.empty_x[g][b & 1], ph, a.wlim));
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint8_t* dst = S.c[g] + (2 * pw + i) * 4096 + (16 * (b & 1)) * 128 + k8 * 16;
                    if (FP8) {
                        uint32_t n4 = 0;
#pragma unroll
                        for (int e = 0; e < NV; ++e)
                            n4 |= e4m3_nan4(v[b][i][e].x) | e4m3_nan4(v[b][i][e].y) | e4m3_nan4(v[b][i][e].z) |
                                  e4m3_nan4(v[b][i][e].w);
                        bad[i] |= n4;
                        const uint32_t keep = n4 ? 0u : 0xFFFFFFFFu;
#pragma unroll
                        for (int e = 0; e < NV; ++e) {
                            const uint32_t w[4] = {v[b][i][e].x & keep, v[b][i][e].y & keep, v[b][i][e].z & keep, v[b][i][e].w & keep};
                            uint32_t o[8];
#pragma unroll
                            for (int t = 0; t < 4; ++t) e4m3x4_f16(w[t], o + 2 * t);
                            *reinterpret_cast<uint4*>(dst + (8 * e + 2 * piece) * 128) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4*>(dst + (8 * e + 2 * piece + 1) * 128) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                    } else {
                        // scales of channels 32 piece .. + 31 of block b: 16 bits of the word that lane b of the row holds
                        const int d = b < 2 ? (x_dim / 128) + b : (y_dim / 128) + (b - 2);
                        const uint2 mine = i ? sc1 : sc0;
                        const uint32_t lo = __shfl_sync(0xffffffffu, mine.x, k8 + 8 * d), hi = __shfl_sync(0xffffffffu, mine.y, k8 + 8 * d);
                        uint32_t s2 = ((piece & 2 ? hi : lo) >> (16 * (piece & 1))) & 0xFFFFu;
                        const uint32_t n2 = e4m3_nan4(s2);
                        bad[i] |= n2;
                        uint32_t ss[2];
                        e4m3x4_f16(n2 ? 0u : s2, ss);
                        const uint32_t w[4] = {v[b][i][0].x, v[b][i][0].y, v[b][i][0].z, v[b][i][0].w};
#pragma unroll
                        for (int e = 0; e < 2; ++e) {  // one group of 16 channels
                            const uint32_t s = __byte_perm(ss[0], 0, e ? 0x3232 : 0x1010);
                            uint32_t o[8];
                            e2m1x8_f16(w[2 * e], o);
                            e2m1x8_f16(w[2 * e + 1], o + 4);
#pragma unroll
                            for (int t = 0; t < 8; ++t) o[t] = mul_f16x2(o[t], s);
                            *reinterpret_cast<uint4*>(dst + (4 * piece + 2 * e) * 128) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4*>(dst + (4 * piece + 2 * e + 1) * 128) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                    }
                }
                if (b == 3) {
                    // per key of each eight: a bit of any of its four lanes
                    uint32_t n0 = __ballot_sync(0xffffffffu, bad[0] != 0), n1 = __ballot_sync(0xffffffffu, bad[1] != 0);
                    n0 |= n0 >> 16;
                    n1 |= n1 >> 16;
                    const uint32_t h0 = __ballot_sync(0xffffffffu, gone & 1u), h1 = __ballot_sync(0xffffffffu, gone & 2u);
                    if (lane == 0) {
                        S.flags[g].nan[pw] = uint16_t(((n0 | n0 >> 8) & 0xFFu) | ((n1 | n1 >> 8) & 0xFFu) << 8);
                        S.flags[g].hidden[pw] = uint16_t((h0 & 0xFFu) | (h1 & 0xFFu) << 8);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(b < 2 ? &S.full_x[g][b] : &S.full_y[g][b - 2]);
                load(b);  // the next tile's block, a tile's time ahead
                if (b == 2) load_scales();
            }
            gone = (src[0] ? 0u : 1u) | (src[1] ? 0u : 2u);
            locate(j + 2);
        }
        if (!ok && lane == 0) record(a.st, CSA2_ERR_TIMEOUT, 7, int32_t(req), ti);
    } else {
        if (!TILES) regs_down<kPMmaRegs>();
        if (tid == 32 * kMmaWarp) {
        // ================= MMA issue
        constexpr uint32_t id_s = idesc_f16(kPM, kPN, 0, false, false), id_o = idesc_f16(kPM, kPHalf, 0, false, true);
        // descriptors; a step of 16 along K is 256 bytes (K-major) or two 8-key groups (MN-major)
        const uint64_t dq0 = umma_desc(smem_u32(S.qx), 128, 4096), dp0 = umma_desc(smem_u32(S.p), 128, 2048);
        const uint64_t dk[2] = {umma_desc(smem_u32(S.c[0]), 128, 4096), umma_desc(smem_u32(S.c[1]), 128, 4096)};
        const uint64_t dv[2] = {umma_desc(smem_u32(S.c[0]), 4096, 128), umma_desc(smem_u32(S.c[1]), 4096, 128)};
        // (a value the compiler cannot know: it would keep every step's descriptor of the loop in registers, and spill)
        auto fresh = [](uint64_t v) {
            asm volatile("" : "+l"(v));
            return v;
        };
        bool ok = true;
        auto o_mma = [&](int32_t j) {  // O += P Y of tile j
            ok = ok && mbar_wait(&S.p_full, j & 1, a.wlim);
            if (!ok) return;
            tc_fence_after();
            const uint64_t d = fresh(j & 1 ? dv[1] : dv[0]), dp = fresh(dp0);
#pragma unroll
            for (int k = 0; k < kPN / 16; ++k)
                mma_f16_ss(tmem + kColO, dp + k * (256 >> 4), d + k * (8192 >> 4), id_o, k > 0 || j > 0);
        };
        for (int32_t j = 0; j < nt && ok; ++j) {
            const int g = j & 1;
            const uint32_t ph = (j >> 1) & 1;
            uint64_t d = fresh(g ? dk[1] : dk[0]), dq = fresh(dq0);
            ok = mbar_wait(&S.s_free, j & 1, a.wlim);  // phase 0: Q; phase j: S of the tile before has been read
            tc_fence_after();
    #pragma unroll
            for (int b = 0; b < 2; ++b) {
                ok = ok && mbar_wait(&S.full_x[g][b], ph, a.wlim);
                if (!ok) break;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_f16_ss(tmem + kColS, dq + (8 * b + k) * (256 >> 4), d + (8 * b + k) * (256 >> 4), id_s, k > 0 || b > 0);
                if (TILES) tc_commit_pair(&S.empty_x[g][b]);
                else tc_commit(&S.empty_x[g][b]);
            }
            if (ok && j > 0) {
                o_mma(j - 1);
                // (only what a producer waits for: an arrival at the other CTA must not outlive it)
                if (ok && TILES && j + 1 < nt) tc_commit_pair(&S.empty_o[g ^ 1]);
                if (ok && !TILES) tc_commit(&S.empty_o[g ^ 1]);
            }
    #pragma unroll
            for (int b = 0; b < 2; ++b) {
                ok = ok && mbar_wait(&S.full_y[g][b], ph, a.wlim);
                if (!ok) break;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_f16_ts(tmem + kColS, tmem + kColQ + 8 * (8 * b + k), d + (8 * b + k) * (256 >> 4), id_s, true);
            }
            if (ok) tc_commit(&S.s_full);
        }
        if (nt > 0) {
            if (ok) o_mma(nt - 1);
            if (ok) tc_commit(&S.o_done);
            if (!ok) record(a.st, CSA2_ERR_TIMEOUT, 8, int32_t(req), ti);
            // after a give-up anywhere, TMEM and shared memory stay until the MMAs in flight are done (in a cluster:
            // until both CTAs' commits have arrived here)
            if (TILES) tc_commit_pair(&S.drain);
            else tc_commit(&S.drain);
            mbar_wait(&S.drain, 0, kDrainNs);
        }
        } else if (TILES && warp == kMmaWarp + 1) {
            // ================= tile copies (the first X blocks are under way)
            const uint8_t* y_src = a.tiles + tile0 * kPTileBytes + half * (kPTileBytes / 2);
            const uint8_t* flags = a.flags + tile0 * kPFlagBytes;
            bool ok = true;
            int32_t last_x[2][2] = {{-1, -1}, {-1, -1}}, last_y[2][2] = {{-1, -1}, {-1, -1}};  // tiles copied last
            for (int32_t j = 0; j < nt && ok; ++j) {
                const int g = j & 1;
                const uint32_t ph = (j >> 1) & 1;
                if (j >= 1)
                    ok = __all_sync(0xffffffffu, j == 1 ? mbar_wait(&S.q_done, 0, a.wlim) : mbar_wait(&S.empty_o[g], ph ^ 1, a.wlim));
                for (int b = 0; b < 2 && ok; ++b) {
                    if (j > 0) copy_block(&S.full_x[g][b], g, b, x_src + j * kPTileBytes, nullptr);
                    last_x[g][b] = j;
                }
                for (int b = 0; b < 2 && ok; ++b) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&S.empty_x[g][b], ph, a.wlim));
                    if (!ok) break;
                    copy_block(&S.full_y[g][b], g, b, y_src + j * kPTileBytes, b ? flags + j * kPFlagBytes : nullptr);
                    last_y[g][b] = j;
                }
            }
            if (!ok && lane == 0) record(a.st, CSA2_ERR_TIMEOUT, 9, int32_t(req), ti);
            // every copy lands before the CTA leaves its shared memory, also after a give-up
            for (int g = 0; g < 2; ++g)
                for (int b = 0; b < 2; ++b) {
                    if (last_x[g][b] >= 0) mbar_wait(&S.full_x[g][b], (last_x[g][b] >> 1) & 1, kDrainNs);
                    if (last_y[g][b] >= 0) mbar_wait(&S.full_y[g][b], (last_y[g][b] >> 1) & 1, kDrainNs);
                }
        }
    }
    tc_fence_before();
    if (TILES) cluster_sync();  // neither CTA leaves while the other may copy or arrive here
    else __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Decodes the pages of every request once into tiles of 128 keys (see
// kSrcTiles), for calls whose requests have several row tiles: each of them
// would decode every key again, and the decoding, not the MMAs, bounds the
// kernel then (12,600 warp instructions a key tile).  grid (tiles, requests).
template <bool FP8>
__global__ void __launch_bounds__(256) paged_decode_kernel(const PagedArgs a) {
    __shared__ uint32_t s_nan[4], s_hidden[4];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t req = blockIdx.y;
    PagedReq rq;
    if (!paged_request(a, req, rq, nullptr)) return;
    const int32_t base = paged_base(a, rq) + int32_t(blockIdx.x) * kPN;
    if (base >= rq.len) return;
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5, k8 = lane & 7, piece = lane >> 3;
    uint8_t* tile = a.tiles + (req * a.span + blockIdx.x) * kPTileBytes;
    if (tid < 4) s_nan[tid] = s_hidden[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // key groups of 8: 2 warp + i; a lane has 16 bytes of every 64
        const int kg = 2 * warp + i, key = 8 * kg + k8;
        const int32_t p = base + key;
        int64_t row = -1;
        if (p < rq.len) {
            const int32_t id = a.table[req * a.max_pages + p / a.page];
            if (id >= 0 && id < a.n_rows_pages)
                row = int64_t(id) * a.page + p % a.page;
            else if (piece == 0)
                record(a.st, CSA2_ERR_DEVICE_BOUNDS, CHK_PAGE, int32_t(req), id);
        }
        uint32_t bad = 0;
        constexpr int NP = FP8 ? 8 : 4;  // 64-byte parts of a row
        uint4 v[NP];
        uint4 sc[2];
#pragma unroll
        for (int e = 0; e < NP; ++e)
            v[e] = row >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.codes + row * (FP8 ? kPD : kPD / 2) + 64 * e) + piece)
                            : make_uint4(0, 0, 0, 0);
        sc[0] = sc[1] = make_uint4(0, 0, 0, 0);
        if (!FP8 && row >= 0) {
            sc[0] = __ldg(reinterpret_cast<const uint4*>(a.scales + row * (kPD / 16)));
            sc[1] = __ldg(reinterpret_cast<const uint4*>(a.scales + row * (kPD / 16)) + 1);
        }
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            const uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
            // channels: FP4 128 e + 32 piece .. + 31, FP8 64 e + 16 piece .. + 15
            constexpr int NC = FP8 ? 2 : 4;
            const int chunk = FP8 ? 8 * e + 2 * piece : 16 * e + 4 * piece;
            uint8_t* dst = tile + (chunk >> 5) * (kPTileBytes / 2) + kg * 4096 + (chunk & 31) * 128 + k8 * 16;
            uint32_t o[4 * NC];
            if (FP8) {
                const uint32_t n4 = e4m3_nan4(w[0]) | e4m3_nan4(w[1]) | e4m3_nan4(w[2]) | e4m3_nan4(w[3]);
                bad |= n4;
#pragma unroll
                for (int m = 0; m < 4; ++m) e4m3x4_f16(n4 ? 0u : w[m], o + 2 * m);
            } else {
                const uint32_t* s8 = &sc[0].x + 2 * e;  // the 8 scales of 128 channels
                const uint32_t s2 = ((piece & 2 ? s8[1] : s8[0]) >> (16 * (piece & 1))) & 0xFFFFu;
                const uint32_t n2 = e4m3_nan4(s2);
                bad |= n2;
                uint32_t ss[2];
                e4m3x4_f16(n2 ? 0u : s2, ss);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint32_t s = __byte_perm(ss[0], 0, m >= 2 ? 0x3232 : 0x1010);
                    e2m1x8_f16(w[m], o + (4 * m) % (4 * NC));
#pragma unroll
                    for (int q = 0; q < 4; ++q) o[(4 * m + q) % (4 * NC)] = mul_f16x2(o[(4 * m + q) % (4 * NC)], s);
                }
            }
#pragma unroll
            for (int c = 0; c < NC; ++c)
                *reinterpret_cast<uint4*>(dst + c * 128) = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
        if (bad) atomicOr(&s_nan[key >> 5], 1u << (key & 31));
        if (row < 0) atomicOr(&s_hidden[key >> 5], 1u << (key & 31));
    }
    __syncthreads();
    uint32_t* fl = reinterpret_cast<uint32_t*>(a.flags + (req * a.span + blockIdx.x) * kPFlagBytes);
    if (tid < 4) fl[tid] = s_hidden[tid], fl[4 + tid] = s_nan[tid];
}

// Joins the splits of a row: weights 2^(lse_s - max lse) over the normalized
// partial outputs.  128 threads per row, 4 channels each; rows whose tile had
// one split were written by the attention kernel.
__global__ void __launch_bounds__(256) paged_merge_kernel(const PagedArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row = int64_t(blockIdx.x) * 2 + (threadIdx.x >> 7);
    const int t = threadIdx.x & 127;
    if (row >= a.rows) return;
    const int32_t tok = int32_t(row / a.heads);
    int64_t lo = 0, hi = a.n_req;  // the last request that starts at or before the token
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (a.q_start[mid] <= tok) lo = mid;
        else hi = mid;
    }
    PagedReq rq;
    if (!paged_request(a, lo, rq, nullptr) || tok < rq.q0 || tok >= rq.q0 + rq.nq) return;
    int32_t begin, end, tiles;
    paged_item_keys(a, rq, int32_t((row - int64_t(rq.q0) * a.heads) / a.item), begin, end, tiles);
    const int32_t splits = paged_splits(tiles, a.chunk);
    if (splits == 1) return;
    float m = -INFINITY;
    for (int32_t s = 0; s < splits; ++s) m = fmaxf(m, a.part_lse[s * a.rows + row]);
    float w = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int32_t s = 0; s < splits; ++s) {
        const float ls = a.part_lse[s * a.rows + row];
        const float f = ls == -INFINITY ? 0.f : ex2(ls - m);
        const float4 v = reinterpret_cast<const float4*>(a.part_o + (s * a.rows + row) * kPD)[t];
        w += f;
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
    }
    const float inv = w == 0.f ? 0.f : 1.0f / w;
    const __nv_bfloat162 h0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), h1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    reinterpret_cast<uint2*>(a.out + row * kPD * 2)[t] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
    if (a.lse && t == 0) a.lse[row] = w == 0.f ? -INFINITY : (m + log2f(w)) * 0.6931471805599453f;
}

// How a call runs, from the host's bounds alone.  A CTA takes one (row tile,
// half, split); the split count is the one with the least time by: waves of
// 152 CTAs, each a start of 5 us and a time per key tile, plus the merge's pass
// over the partial outputs.
// Requests of more than two row tiles take the latents from decoded tiles where
// those need no more than 1 GB: 1024 tokens x 64 heads over 16K entries take
// DECODED_MS against 3.00 ms; at one row tile a key would be decoded once
// either way, and written and read besides.
struct PagedPlan {
    int32_t chunk, splits, span, item;
    int64_t grid;
    size_t part_lse, part_o, tiles, flags, total;
};
constexpr size_t kPMaxTileBytes = size_t(1) << 30;
static PagedPlan paged_plan(int64_t n_tokens, int n_heads, int64_t n_req, int32_t max_q, int32_t max_kv, int window) {
    PagedPlan p{};
    if (window >= max_kv) window = 0;
    const int64_t rows = n_tokens * n_heads;
    p.item = kPM;
    if (paged_items(max_q, n_heads, kPM) > 2) {
        int64_t span = (max_kv + kPN - 1) / kPN;
        if (window > 0) {  // from the first token's window to the last token
            const int64_t w = (int64_t(window) + max_q + 7 + kPN - 1) / kPN;
            span = span < w ? span : w;
        }
        if (n_req <= 65535 && size_t(n_req) * size_t(span) * kPTileBytes <= kPMaxTileBytes) {
            p.span = int32_t(span);
            p.item = 2 * kPM;
        }
    }
    int64_t items = rows / p.item + n_req;  // each request rounds up
    const int64_t each = n_req * paged_items(max_q, n_heads, p.item);
    items = items < each ? items : each;
    const int64_t ctas = 2 * items * (p.item / kPM);
    const int32_t nt = paged_key_tiles(max_q, max_kv, n_heads, window, p.item);
    const double tile_us = p.span ? 1.9 : 3.4;
    p.chunk = nt > 0 ? nt : 1;
    double best = 1e30;
    for (int s = 1; s <= 32 && s <= (nt > 0 ? nt : 1); ++s) {
        const int32_t chunk = (nt + s - 1) / s;
        if (s > 1 && paged_splits(nt, chunk) != s) continue;
        const double waves = double((ctas * s + kPSms - 1) / kPSms);
        double us = waves * (5.0 + tile_us * chunk);
        if (s > 1) us += 4.0 + double(rows) * s * kPD * 4 * 2 / 4e6;
        if (us < best) {
            best = us;
            p.chunk = chunk > 0 ? chunk : 1;
        }
    }
    p.splits = paged_splits(nt, p.chunk);
    p.grid = ctas * p.splits;
    size_t at = CSA2_STATUS_BYTES;
    p.part_lse = at;
    if (p.splits > 1) at = align256(at + size_t(p.splits) * size_t(rows) * 4);
    p.part_o = at;
    if (p.splits > 1) at = align256(at + size_t(p.splits) * size_t(rows) * kPD * 4);
    p.flags = at;
    at = align256(at + size_t(n_req) * p.span * kPFlagBytes);
    p.tiles = at;
    at += size_t(n_req) * p.span * kPTileBytes;
    p.total = at;
    return p;
}

// Once per device and format: the shared memory opt-in, and the register
// count that the kernel's split of them is made for.
template <int SRC>
static csa2_status prepare_paged() {
    static std::atomic<bool> done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CSA2_ERR_CUDA;
    if (done[dev].load(std::memory_order_acquire)) return CSA2_OK;
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, paged_attn_kernel<SRC>) != cudaSuccess ||
        (SRC != kSrcTiles && at.numRegs != kPLaunchRegs) ||
        cudaFuncSetAttribute(paged_attn_kernel<SRC>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(PagedSmem))) !=
            cudaSuccess) {
        cudaGetLastError();
        return CSA2_ERR_CUDA;
    }
    done[dev].store(true, std::memory_order_release);
    return CSA2_OK;
}

static bool paged_sizes(int64_t n_tokens, int n_heads, int64_t n_req, int32_t max_q, int32_t max_kv, int window) {
    return n_tokens >= 0 && n_tokens <= (int64_t(1) << 22) && n_heads >= 1 && n_heads <= 128 && n_req >= 0 &&
           n_req <= (1 << 20) && max_q >= 0 && max_kv >= 0 && window >= 0;
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
    if (!ws || !aligned16(ws) ||
        ws_bytes < csa2_paged_attn_workspace_bytes(n_tokens, n_heads, n_req, max_q, max_kv, window))
        return CSA2_ERR_WORKSPACE;
    if (n_tokens == 0 || n_req == 0 || max_q == 0) return CSA2_OK;
    cudaStream_t s = cudaStream_t(stream);
    const PagedPlan plan = paged_plan(n_tokens, n_heads, n_req, max_q, max_kv, window);
    if (plan.grid > INT32_MAX) return CSA2_ERR_UNSUPPORTED;
    const bool fp8 = fmt == CSA2_FMT_FP8;
    auto kernel = plan.span ? paged_attn_kernel<kSrcTiles> : fp8 ? paged_attn_kernel<kSrcFp8> : paged_attn_kernel<kSrcFp4>;
    const csa2_status prep = plan.span ? prepare_paged<kSrcTiles>() : fp8 ? prepare_paged<kSrcFp8>() : prepare_paged<kSrcFp4>();
    if (prep != CSA2_OK) return prep;
    PagedArgs a{};
    a.q = static_cast<const uint8_t*>(q_bf16);
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.codes = codes;
    a.scales = scales;
    a.table = table;
    a.out = static_cast<uint8_t*>(out);
    a.lse = out_lse;
    a.part_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.part_lse);
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.part_o);
    if (plan.span) {
        a.tiles = reinterpret_cast<uint8_t*>(static_cast<char*>(ws) + plan.tiles);
        a.flags = reinterpret_cast<uint8_t*>(static_cast<char*>(ws) + plan.flags);
        a.span = plan.span;
    }
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
    a.chunk = plan.chunk;
    a.item = plan.item;
    a.sm_scale = sm_scale;
    if (plan.span) {
        timer_begin(K_PAGED_DECODE, s);
        launch(fp8 ? paged_decode_kernel<true> : paged_decode_kernel<false>, dim3(unsigned(plan.span), unsigned(n_req)), 256, 0,
               s, 1, a);
        timer_end(K_PAGED_DECODE, s);
    }
    timer_begin(K_PAGED_ATTN, s);
    const cudaError_t e = launch(kernel, dim3(unsigned(plan.grid)), plan.span ? kPTileThreads : kPThreads, sizeof(PagedSmem), s,
                                 plan.span ? 2 : 1, a);
    timer_end(K_PAGED_ATTN, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return CSA2_ERR_CUDA;
    }
    if (plan.splits > 1) {
        timer_begin(K_PAGED_MERGE, s);
        launch(paged_merge_kernel, dim3(unsigned(ceil_div<int64_t>(a.rows, 2))), 256, 0, s, 1, a);
        timer_end(K_PAGED_MERGE, s);
    }
    return launch_status();
}
