// Causal attention over paged latents for requests of few rows (single tokens
// and short chunks) and for chunks that see few keys: 64 (token, head) rows per
// CTA, all 512 channels.
//
// With few rows every key is decoded for one or a few CTAs only, and the
// decoding costs as much as the MMAs.  A CTA of 128 rows and half of the output
// channels (csa2_paged_tiles.cu) would need each key decoded for both halves,
// and at 64 heads half of its rows stay empty.  Transposed, the products need
// one copy of a decoded tile and 64 columns of TMEM per 128 channels:
//
//   S^T [128 keys x 64 rows]     = C Q^T     32 MMAs, M = keys, K = channels
//   O^T [4 x 128 channels x 64]  += C^T P^T  4 x 8 MMAs, M = channels, K = keys
//
// (an M = 128 MMA of K = 16 takes 64 clocks for any N up to 128: 4100 clocks a
// tile).  C [128 keys][512] in f16 fills 128 KB, so the next tile is decoded in
// halves of the channels as O^T is done with this one's: the first half under
// the second half's O^T, the second under the first half's S^T.
//
//   smem  Q 64 KB, C 128 KB (four blocks of 128 channels), P^T 16 KB      TMEM  O^T 256, S^T 64
//
// Softmax: a thread per key, the 64 rows in its registers.  The rows' bases
// stand in shared memory; a tile whose logits all stay below kPGrow (log2) above
// needs no reduction at all, since each thread sums its own key's
// probabilities row by row over all tiles and the 128 threads' sums are joined
// once at the end.  A logit above that (and the first tile) takes the
// reduction over the keys and rescales O^T and the sums.
#include "csa2_paged.cuh"
#include "csa2_timer.cuh"

#include <atomic>
#include <cfloat>

namespace csa2 {

constexpr int kRRows = 64;
constexpr int kRProdWarps = 8;
constexpr int kRThreads = 32 * (kPSoftWarps + kRProdWarps + 4);  // and a warpgroup for the MMA thread
constexpr int kRMmaWarp = kPSoftWarps + kRProdWarps;
constexpr int kRBlock = kPN * 128 * 2;  // bytes of 128 channels of a tile: 8-key groups of 2048 B, 8-channel chunks of 128 B
constexpr uint32_t kRColO = 0, kRColS = 256;
// Registers per thread: the launch gives 128 x 512; the warpgroups pass them
// on as 208 + 2 x 112 + 80 = 512 = 4 x 128.  No role spills: the latents stream
// through what L1 the shared memory leaves, so a spilled value comes back from
// L2 (the MMA thread issued one MMA per 300 clocks with spilled descriptors).
constexpr int kRLaunchRegs = 128, kRSoftRegs = 208, kRProdRegs = 112, kRMmaRegs = 80;
static_assert(kRSoftRegs + 2 * kRProdRegs + kRMmaRegs <= 4 * kRLaunchRegs, "registers");

struct PagedRowsSmem {
    uint8_t q[kRRows * kPD * 2];  // 8-row groups of 8192 B, 8-channel chunks of 128 B
    uint8_t c[4][kRBlock];        // a tile's channels in blocks of 128
    uint8_t p[kPN * kRRows * 2];  // P^T: 8-key groups of 1024 B, 8-row chunks of 128 B
    float2 row[kRRows];           // a row's factor of the raw logits and its base (log2 domain; 0 before any key)
    int2 keys[kRRows];            // keys [x, y) that a row sees
    float alpha[kRRows], delta[kRRows];
    float red[4][kRRows];
    int fresh;                    // rows that have seen no key yet
    PagedFlags flags[2][2];       // of a tile, by each team of producers
    uint64_t full[2], empty[4], s_full, p_full, o_done, drain;  // full: of each half of the channels
    uint32_t tmem;
    PagedWork work;
    int64_t sums[2 * kRThreads / 32];
};
static_assert(sizeof(PagedRowsSmem) + 1024 <= 227 * 1024, "shared memory of the few-row paged attention");

// Barriers of the four softmax warps, and the OR / AND of their threads' flags.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 2, 128;" ::: "memory"); }
__device__ __forceinline__ bool soft_or(bool v) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r) : "r"(uint32_t(v)) : "memory");
    return r != 0;
}
__device__ __forceinline__ bool soft_and(bool v) { return !soft_or(!v); }

// Over a warp's lanes, 32 values each: lane l gets the maximum or sum of v[l].
// Every round a lane keeps half of its values and takes the partner's half.
template <bool MAX>
__device__ __forceinline__ float over_lanes(float (&v)[32]) {
    const int lane = lane_id();
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            const float got = __shfl_xor_sync(0xffffffffu, send, o);
            v[i] = MAX ? fmaxf(keep, got) : keep + got;
        }
    }
    return v[0];
}

// grid: one CTA per (64 rows of a request, split), the ones with the most keys
// first; CTAs beyond the last one leave at once.
template <bool FP8>
__global__ void __launch_bounds__(kRThreads, 1) paged_rows_kernel(const PagedArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    PagedRowsSmem& S = *reinterpret_cast<PagedRowsSmem*>(smem_raw);
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
    // Behind the tile kernel, which runs other requests of the same call: the
    // inputs are there when that one has started (it is behind the decode
    // kernel), so this one only has to end after it.
    if (!a.behind) grid_dep_wait();
    grid_dep_launch();
    paged_find<kRThreads / 32>(a, blockIdx.x, blockIdx.x == 0, S.work, S.sums);
    if (warp == kRMmaWarp) {
        if (lane == 0) {
            for (int b = 0; b < 4; ++b) mbar_init(&S.empty[b], 1);
            for (int b = 0; b < 2; ++b) mbar_init(&S.full[b], kRProdWarps / 2);
            mbar_init(&S.s_full, 1);
            mbar_init(&S.p_full, kPSoftWarps);
            mbar_init(&S.o_done, 1);
            mbar_init(&S.drain, 1);
            mbar_init_fence();
        }
        __syncwarp();
        tmem_alloc(&S.tmem, 512);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    const int64_t req = S.work.req;
    const PagedReq rq = S.work.rq;
    if (req < 0) {
        if (warp == kRMmaWarp) tmem_dealloc(tmem, 512);
        if (a.behind) grid_dep_wait();
        return;
    }
    const int32_t nt = S.work.nt, key0 = S.work.key0, splits = S.work.splits;
    const int32_t row0 = S.work.item * kRRows;  // of the request
    const int32_t n_row = rq.nq * a.heads - row0 < kRRows ? rq.nq * a.heads - row0 : kRRows;
    const int32_t k_end = rq.len - rq.nq + (row0 + n_row - 1) / a.by_heads + 1;
    const int32_t k_last = key0 + nt * kPN < k_end ? key0 + nt * kPN : k_end;  // end of this CTA's keys

    // ---- Q by the warps that do not bring in latents, one group of 8 rows each
    if (warp < kPSoftWarps || warp >= kRMmaWarp) {
        const int row = 8 * (warp < kPSoftWarps ? warp : warp - kRProdWarps) + (lane & 7), piece = lane >> 3;
        const bool on = row < n_row;
        U32x8 v[8];
        paged_q_load(a, S.work.out0 + row, on, v);
        const int qs = paged_q_exponent(v);
        if (piece == 0) {
            S.row[row] = make_float2(paged_q_scale(a, qs), 0.f);
            // rows behind the last one see nothing
            const int32_t hi = on ? rq.len - rq.nq + (row0 + row) / a.by_heads + 1 : 0;
            S.keys[row] = make_int2(a.window > 0 ? hi - a.window : 0, hi);
            if (row == 0) S.fresh = n_row;
        }
        uint8_t* dst = S.q + (row >> 3) * 8192 + piece * 256 + (row & 7) * 16;
#pragma unroll
        for (int i = 0; i < 8; ++i) paged_q_store(dst + i * 1024, v[i], qs);
        fence_async_smem();
        asm volatile("bar.sync 1, 256;" ::: "memory");
    }

    if (warp < kPSoftWarps) {
        regs_up<kRSoftRegs>();
        // ================= softmax: key = TMEM lane = thread, rows in registers
        const uint32_t tm = tmem + (uint32_t(32 * warp) << 16);
        uint8_t* pd = S.p + (tid >> 3) * 1024 + (tid & 7) * 16;
        float l[kRRows];
#pragma unroll
        for (int c = 0; c < kRRows; ++c) l[c] = 0.f;
        bool ok = true;
        for (int32_t j = 0; j < nt; ++j) {
            ok = soft_and(mbar_wait(&S.s_full, j & 1, a.wlim));
            if (!ok) break;
            tc_fence_after();
            float x[2][32];
            tmem_ld32(tm + kRColS, reinterpret_cast<uint32_t(&)[32]>(x[0]));
            tmem_ld32(tm + kRColS + 32, reinterpret_cast<uint32_t(&)[32]>(x[1]));
            tmem_ld_wait();
            // to the log2 domain, against the row's base
            float top = -INFINITY;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float4 r = *reinterpret_cast<const float4*>(&S.row[32 * h + c]);
                    x[h][c] = fmaf(x[h][c], r.x, -r.y);
                    x[h][c + 1] = fmaf(x[h][c + 1], r.z, -r.w);
                }
            const int32_t key = key0 + j * kPN + tid;
            const PagedFlags *f = S.flags[j & 1];
            const bool hidden = (f[0].hidden[tid >> 4] >> (tid & 15)) & 1;
            const bool nan = ((f[0].nan[tid >> 4] | f[1].nan[tid >> 4]) >> (tid & 15)) & 1;
            // the rows' key ranges are ordered: the first row's end and the last one's start bound all of them (what a row
            // behind the last one sees is of no account)
            const bool inside = key < S.keys[0].y && key >= S.keys[n_row - 1].x;
            if (__any_sync(0xffffffffu, hidden || nan || !inside)) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const int2 k = S.keys[32 * h + c];
                        if (nan) x[h][c] = __uint_as_float(0x7FC00000u);
                        if (hidden || key < k.x || key >= k.y) x[h][c] = -INFINITY;
                    }
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) top = fmaxf(top, fmaxf(x[0][c], x[1][c]));
            if (soft_or(top > kPGrow) || S.fresh > 0) {  // (S.fresh was written before a barrier that all have passed)
                // maxima over the keys; rows with a logit above kPGrow, or that see their first key, move their base
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) v[c] = x[h][c];
                    S.red[warp][32 * h + lane] = over_lanes<true>(v);
                }
                soft_sync();
                const bool was_fresh = S.fresh > 0;  // some row is
                int still = 0;
                if (tid < kRRows) {
                    const float t = fmaxf(fmaxf(S.red[0][tid], S.red[1][tid]), fmaxf(S.red[2][tid], S.red[3][tid]));
                    const float m = S.row[tid].y;
                    // alpha < 0 marks a row that has seen no key before this tile (set below); first tile: all
                    const bool mine = j == 0 || (was_fresh && S.alpha[tid] < 0.f);
                    float d = 0.f, al = 1.f;
                    if (mine) {
                        if (t > -INFINITY) d = t - kPBase, al = 0.f;
                        else al = -1.f;
                    } else if (t > kPGrow) {
                        d = t - kPBase;
                        al = ex2(-d);
                    }
                    still = tid < n_row && al < 0.f;
                    S.row[tid].y = m + d;
                    S.delta[tid] = d;
                    S.alpha[tid] = al;
                }
                soft_sync();
                const uint32_t left = __ballot_sync(0xffffffffu, still);
                if (tid == 0) S.fresh = 0;
                soft_sync();
                if (lane == 0 && left != 0) atomicAdd(&S.fresh, __popc(left));
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 d = *reinterpret_cast<const float4*>(&S.delta[32 * h + c]);
                        const float4 al = *reinterpret_cast<const float4*>(&S.alpha[32 * h + c]);
                        x[h][c] -= d.x, x[h][c + 1] -= d.y, x[h][c + 2] -= d.z, x[h][c + 3] -= d.w;
                        l[32 * h + c] *= fmaxf(al.x, 0.f), l[32 * h + c + 1] *= fmaxf(al.y, 0.f);
                        l[32 * h + c + 2] *= fmaxf(al.z, 0.f), l[32 * h + c + 3] *= fmaxf(al.w, 0.f);
                    }
                if (j > 0) {  // every MMA before this tile's logits is done, the previous O^T among them
#pragma unroll 1
                    for (int b = 0; b < 8; ++b) {
                        uint32_t o[32];
                        tmem_ld32(tm + kRColO + 32 * b, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            o[c] = __float_as_uint(__uint_as_float(o[c]) * fmaxf(S.alpha[32 * (b & 1) + c], 0.f));
                        tmem_st32(tm + kRColO + 32 * b, o);
                    }
                    tmem_st_wait();
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < 32; c += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p0 = ex2(x[h][c + 2 * e]), p1 = ex2(x[h][c + 2 * e + 1]);
                        l[32 * h + c + 2 * e] += p0;
                        l[32 * h + c + 2 * e + 1] += p1;
                        w[e] = f16x2(p0, p1);
                    }
                    *reinterpret_cast<uint4*>(pd + (4 * h + c / 8) * 128) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.p_full);
        }
        if (ok && nt > 0) ok = soft_and(mbar_wait(&S.o_done, 0, a.wlim));
        if (!ok && lane == 0) record(a.st, CSA2_ERR_TIMEOUT, 6, int32_t(req), S.work.item);
        // ---- epilogue: the rows' sums, then O / l row by row in shared memory (the latents' place), and out
        if (ok) {
            tc_fence_after();
            const int64_t out0 = S.work.out0, part0 = S.work.part0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = l[32 * h + c];
                S.red[warp][32 * h + lane] = over_lanes<false>(v);
            }
            soft_sync();
            if (tid < kRRows) {
                const float sum = (S.red[0][tid] + S.red[1][tid]) + (S.red[2][tid] + S.red[3][tid]);
                S.alpha[tid] = sum == 0.f ? 0.f : 1.0f / sum;
                const float lse2 = sum == 0.f ? -INFINITY : S.row[tid].y + log2f(sum);
                if (tid < n_row) {
                    if (splits > 1)
                        a.part_lse[part0 + tid] = lse2;
                    else if (a.lse)
                        a.lse[out0 + tid] = lse2 * kLn2;
                }
            }
            soft_sync();
            const bool whole = splits == 1;
            uint8_t* stage = S.c[0];
#pragma unroll 1
            for (int b = 0; b < 8; ++b) {  // channels 128 (b / 2) + thread, rows 32 (b % 2) ..
                uint32_t o[32];
                if (nt > 0) {
                    tmem_ld32(tm + kRColO + 32 * b, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = 0;
                }
                const int dim = 128 * (b >> 1) + tid;
#pragma unroll
                for (int c = 0; c < 32; c += 4) {  // (all loads before the stores, which could be to the same place for all
                                                   // the compiler knows: 47 clocks a value otherwise)
                    const float4 f = *reinterpret_cast<const float4*>(&S.alpha[32 * (b & 1) + c]);
                    o[c] = __float_as_uint(__uint_as_float(o[c]) * f.x);
                    o[c + 1] = __float_as_uint(__uint_as_float(o[c + 1]) * f.y);
                    o[c + 2] = __float_as_uint(__uint_as_float(o[c + 2]) * f.z);
                    o[c + 3] = __float_as_uint(__uint_as_float(o[c + 3]) * f.w);
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const int r = 32 * (b & 1) + c;
                    const float v = __uint_as_float(o[c]);
                    if (whole)
                        reinterpret_cast<__nv_bfloat16*>(stage)[r * kPD + dim] = __float2bfloat16_rn(v);
                    else
                        reinterpret_cast<float*>(stage)[r * kPD + dim] = v;
                }
            }
            fence_async_smem();
            soft_sync();
            if (tid < n_row) {
                if (whole)
                    bulk_s2g(a.out + (out0 + tid) * kPD * 2, stage + tid * kPD * 2, kPD * 2);
                else
                    bulk_s2g(a.part_o + (part0 + tid) * kPD, stage + tid * kPD * 4, kPD * 4);
                bulk_s2g_wait();
            }
        }
    } else if (warp < kRMmaWarp) {
        regs_down<kRProdRegs>();
        // ================= producers: two teams of four warps, the first with channels 0 .. 255
        // (blocks 0 and 1), the second with the others.  A thread has keys 32 w +
        // 8 i + (lane % 8), i < 4, and the piece lane / 8 of 64 channels.  Loads are
        // whole lines (32 bytes a lane, four lanes a row of 128 bytes; 8 rows of 64
        // bytes an instruction kept the load unit busy for 1200 clocks a tile); a
        // quarter-warp stores 8 keys of one chunk: no bank conflicts.  Keys in
        // eights share a page.
        const int team = (warp - kPSoftWarps) >> 2, w4 = warp & 3, k8 = lane & 7, piece = lane >> 3;
        constexpr int NV = FP8 ? 2 : 1;  // loads per key: 64 channels in 32 bytes (FP4), or 32 (E4M3)
        U32x8 v[4][NV];
        uint32_t sc[4];                  // FP4: the four scales of the thread's channels
        const int32_t* trow = a.table + req * a.max_pages;
        // page ids of the warp's four key groups in 8 tiles, one per lane: a tile's are shuffled out
        int32_t ids = -1;
        uint32_t gone = 0;               // keys of the tile without a row, a bit each
        // place within its page of the first key of the tile that is loaded next; a tile on is 128 keys on
        const int32_t step_off = kPN % a.page;
        int32_t off_t = (key0 + 32 * w4) % a.page + k8;  // groups of 8 keys share a page, so this is below it
        auto load = [&](int32_t j) {
            if ((j & 7) == 0) {
                const int32_t p = key0 + (j + (lane >> 2)) * kPN + 32 * w4 + 8 * (lane & 3);
                ids = p < k_last ? trow[p / a.by_page] : -1;
            }
            int32_t off = off_t;
            gone = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t id = __shfl_sync(0xffffffffu, ids, 4 * (j & 7) + i);
                const bool in = key0 + j * kPN + 32 * w4 + 8 * i + k8 < k_last;
                if (in && id >= 0 && id < a.n_rows_pages) {
                    const int64_t row = int64_t(id) * a.page + off;
                    const uint8_t* src = a.codes + row * (FP8 ? kPD : kPD / 2) + team * (FP8 ? 256 : 128) + 32 * piece;
                    // E4M3: channels 32 piece .. of each 128 of the team's 256
#pragma unroll
                    for (int e = 0; e < NV; ++e) v[i][e] = ldg_32b(src + 128 * e);
                    if (!FP8) sc[i] = __ldg(reinterpret_cast<const uint32_t*>(a.scales + row * (kPD / 16) + 16 * team) + piece);
                } else {
                    if (in && piece == 0 && team == 0) record(a.st, CSA2_ERR_DEVICE_BOUNDS, CHK_PAGE, int32_t(req), id);
                    gone |= 1u << i;
#pragma unroll
                    for (int e = 0; e < NV; ++e)
#pragma unroll
                        for (int x = 0; x < 8; ++x) v[i][e].w[x] = 0;
                    sc[i] = 0;
                }
                off += 8;
                if (off >= a.page) off -= a.page;
            }
            off_t += step_off;
            if (off_t >= a.page) off_t -= a.page;
        };
        load(0);
        bool ok = true;
        for (int32_t j = 0; j < nt && ok; ++j) {
            uint32_t bad = 0;  // a bit per key
            if (j >= 1) {
                ok = __all_sync(0xffffffffu, mbar_wait(&S.empty[2 * team], (j - 1) & 1, a.wlim));
                ok = ok && __all_sync(0xffffffffu, mbar_wait(&S.empty[2 * team + 1], (j - 1) & 1, a.wlim));
                if (!ok) break;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (FP8) {
#pragma unroll
                    for (int e = 0; e < NV; ++e) {  // 32 channels of block 2 team + e
                        uint32_t n4 = 0;
#pragma unroll
                        for (int x = 0; x < 8; ++x) n4 |= e4m3_nan4(v[i][e].w[x]);
                        bad |= (n4 ? 1u : 0u) << i;
                        const uint32_t keep = n4 ? 0u : 0xFFFFFFFFu;
                        uint8_t* dst = S.c[2 * team + e] + (4 * w4 + i) * 2048 + 4 * piece * 128 + k8 * 16;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint32_t o[4];
                            e4m3x4_f16(v[i][e].w[2 * x] & keep, o);
                            e4m3x4_f16(v[i][e].w[2 * x + 1] & keep, o + 2);
                            *reinterpret_cast<uint4*>(dst + x * 128) = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                } else {
                    const uint32_t n4 = e4m3_nan4(sc[i]);
                    bad |= (n4 ? 1u : 0u) << i;
                    uint32_t ss[2];
                    e4m3x4_f16(n4 ? 0u : sc[i], ss);
                    uint8_t* dst = S.c[2 * team + (piece >> 1)] + (4 * w4 + i) * 2048 + 8 * (piece & 1) * 128 + k8 * 16;
#pragma unroll
                    for (int x = 0; x < 8; ++x) {  // 8 channels; a scale serves two
                        const uint32_t s = __byte_perm(ss[x >> 2], 0, x & 2 ? 0x3232 : 0x1010);
                        uint32_t o[4];
                        e2m1x8_f16(v[i][0].w[x], o);
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[e] = mul_f16x2(o[e], s);
                        *reinterpret_cast<uint4*>(dst + x * 128) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
            {  // per key a bit of any of its four lanes, eight keys a byte
                uint32_t nan = 0, hid = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t x = __ballot_sync(0xffffffffu, (bad >> i) & 1u);
                    x |= x >> 16;
                    nan |= ((x | x >> 8) & 0xFFu) << (8 * i);
                    hid |= (__ballot_sync(0xffffffffu, (gone >> i) & 1u) & 0xFFu) << (8 * i);
                }
                if (lane == 0) {
                    reinterpret_cast<uint32_t*>(S.flags[j & 1][team].nan)[w4] = nan;
                    reinterpret_cast<uint32_t*>(S.flags[j & 1][team].hidden)[w4] = hid;
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.full[team]);
            if (j + 1 < nt) load(j + 1);
        }
        if (!ok && lane == 0) record(a.st, CSA2_ERR_TIMEOUT, 7, int32_t(req), S.work.item);
    } else {
        regs_down<kRMmaRegs>();
        if (tid == 32 * kRMmaWarp) {
            // ================= MMA issue
            constexpr uint32_t id_s = idesc_f16(kPN, kRRows, 0, false, false), id_o = idesc_f16(128, kRRows, 0, true, true);
            // descriptors; a step of 16 along K is 256 bytes (K-major) or two 8-key groups (MN-major).  (A value the
            // compiler cannot know: it would keep every step's descriptor of the loop in registers, and spill.)
            auto fresh = [](uint64_t v) {
                asm volatile("" : "+l"(v));
                return v;
            };
            const uint64_t dq0 = umma_desc(smem_u32(S.q), 128, 8192), dp0 = umma_desc(smem_u32(S.p), 1024, 128);
            const uint64_t dk0 = umma_desc(smem_u32(S.c[0]), 128, 2048), dv0 = umma_desc(smem_u32(S.c[0]), 2048, 128);
            bool ok = true;
            auto s_mma = [&](int32_t j, int b) {  // S^T += C_b Q_b^T of tile j
                if ((b & 1) == 0) ok = ok && mbar_wait(&S.full[b >> 1], j & 1, a.wlim);
                if (!ok) return;
                tc_fence_after();
                const uint64_t dk = fresh(dk0) + b * (kRBlock >> 4), dq = fresh(dq0) + b * (2048 >> 4);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_f16_ss(tmem + kRColS, dk + k * (256 >> 4), dq + k * (256 >> 4), id_s, k > 0 || b > 0);
            };
            auto o_mma = [&](int32_t j, int b) {  // O^T_b += C_b^T P^T of tile j
                if (!ok) return;
                const uint64_t dv = fresh(dv0) + b * (kRBlock >> 4), dp = fresh(dp0);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_f16_ss(tmem + kRColO + 64 * b, dv + k * (4096 >> 4), dp + k * (2048 >> 4), id_o, k > 0 || j > 0);
                tc_commit(&S.empty[b]);
            };
            for (int b = 0; b < 4 && nt > 0; ++b) s_mma(0, b);
            if (ok && nt > 0) tc_commit(&S.s_full);
            for (int32_t j = 0; j < nt && ok; ++j) {
                ok = mbar_wait(&S.p_full, j & 1, a.wlim);
                if (!ok) break;
                tc_fence_after();
                const bool next = j + 1 < nt;
                for (int b = 0; b < 4; ++b) o_mma(j, b);
                if (next) {
                    for (int b = 0; b < 4; ++b) s_mma(j + 1, b);
                    if (ok) tc_commit(&S.s_full);
                } else if (ok) {
                    tc_commit(&S.o_done);
                }
            }
            if (!ok) record(a.st, CSA2_ERR_TIMEOUT, 8, int32_t(req), S.work.item);
            if (nt > 0) {  // after a give-up, TMEM and shared memory stay until the MMAs in flight are done
                tc_commit(&S.drain);
                mbar_wait(&S.drain, 0, kDrainNs);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kRMmaWarp) tmem_dealloc(tmem, 512);
    if (a.behind) grid_dep_wait();
}

template <bool FP8>
static csa2_status rows_launch(const PagedArgs& a, unsigned grid, cudaStream_t s) {
    // once per device: the shared memory opt-in, and the register count that the kernel's split of them is made for
    static std::atomic<bool> done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CSA2_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, paged_rows_kernel<FP8>) != cudaSuccess || at.numRegs != kRLaunchRegs ||
            cudaFuncSetAttribute(paged_rows_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(sizeof(PagedRowsSmem))) != cudaSuccess)
            return CSA2_ERR_CUDA;
        done[dev].store(true, std::memory_order_release);
    }
    timer_begin(K_PAGED_ATTN, s);
    const cudaError_t e = launch(paged_rows_kernel<FP8>, dim3(grid), kRThreads, sizeof(PagedRowsSmem), s, 1, a);
    timer_end(K_PAGED_ATTN, s);
    return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

csa2_status paged_rows_launch(const PagedArgs& a, bool fp8, unsigned grid, cudaStream_t s) {
    return fp8 ? rows_launch<true>(a, grid, s) : rows_launch<false>(a, grid, s);
}

}  // namespace csa2
