// Causal attention of each request's new tokens over its paged latents.
//
//   l_p = sm_scale q . c_p,  o = sum_p softmax(l)_p c_p,  c_p a 512-wide
//   latent in FP4 (E2M1, one E4M3 scale per 16 channels) or E4M3
//
// Rows are (token, head) pairs: 128 consecutive rows of a request make a tile
// of the tensor cores' M, whatever the number of heads.  All heads share the
// latents, so a key costs 2048 FLOPs a row against 288 bytes: the tensor cores
// bound the kernel.
//
// The latents are decoded once per call (paged_decode_kernel, at the end of
// this file) to tiles of 128 keys in f16, exact, laid out as shared memory holds
// them.  With the decoding inside the attention kernel every pair of CTAs did
// it again, 12,600 warp instructions a key tile, and 1024 tokens x 64 heads over
// 16K entries took 2.7 ms (csa2_paged_rows.cu still does) instead of 1.84.
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
// 256 channels at once.  Every CTA copies its own 128 KB per tile, 9.0 TB/s from L2
// over the GPU for 1024 tokens over 16K, with plain bulk copies.  Three roles:
//   copy warp  the other half's channels X of a tile first, then, as the logits'
//       MMAs release them, the own half's Y into the same group.  One copy of Y
//       serves S (K-major) and O (MN-major).
//   MMA warp, per tile:  S += Q_X X^T, O += P Y of the previous tile for 128
//       channels, S += Q_Y Y^T, then the other 128 channels of O.  The softmax of
//       a tile runs under the next tile's S_X, the copy of Y under the first half
//       of O, and the read of S out of TMEM under the second (with all of O
//       between the two parts of S the tensor cores waited for that read: 583 us where
//       it was 567, 512 tokens x 64 heads over 8K).
//   softmax (4 warps, a thread per row)  takes S out of TMEM, keeps the
//       running base and sum in fp32, writes P as f16 to shared memory.  O is
//       rescaled only when a logit lies 2^15 above the base (kPGrow).
// P is rounded to f16 (2^-11 relative, an eighth of the step of the bf16
// output); Q goes to f16 times a power of two per row (exact down to 2^-28 of
// the row's maximum).
//
// A tile takes about 4150 clocks, three quarters of them MMAs: a block that is released
// is there again some 1500 clocks later, and S has one place in TMEM, so the next
// logits wait for the softmax to have read it.  512 tokens x 64 heads over 8K
// entries: 523 us, 1090 TFLOP/s without the third product; 1024 tokens over 16K:
// 1.84 ms, 1160 TFLOP/s.
//
// Long axes with few rows are split over CTAs in chunks of key tiles that the
// host sizes; the partial outputs are joined by paged_merge_kernel.
#include "csa2_paged.cuh"
#include "csa2_timer.cuh"

#include <atomic>

namespace csa2 {

constexpr int kPM = 128;                            // rows of a tile
constexpr int kPTileThreads = 32 * (kPSoftWarps + 4);  // softmax, MMA and copy warps (and two that only bring in Q)
constexpr int kPBlockBytes = kPN * 128 * 2;             // of a tile: 128 channels
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 384;

struct PagedTilesSmem {
    uint8_t qx[kPM * kPHalf * 2];      // other half of Q, K-major: 8-row groups of 4096 B, 8-channel chunks of 128 B
    uint8_t c[2][kPN * kPHalf * 2];    // latents: per 128 channels 8-key groups of 2048 B, 8-channel chunks of 128 B
    uint8_t p[kPM * kPN * 2];          // P: 8-row groups of 2048 B, 8-key chunks of 128 B
    PagedFlags flags[2];
    float q_scale[kPM];                // logits' scale of each row (log2 domain)
    uint64_t full_x[2][2], full_y[2][2], empty_x[2][2], empty_o[2][2];
    uint64_t s_full, s_free, p_full, p_free, o_done, q_done, drain;
    uint32_t tmem;
    PagedWork work;
    int64_t sums[2 * kPTileThreads / 32];
};
static_assert(sizeof(PagedTilesSmem) + 1024 <= 227 * 1024, "shared memory of the paged attention");
static_assert(kPM * (kPHalf * 4 + 16) <= 2 * kPN * kPHalf * 2 + kPM * kPN * 2, "the epilogue's rows in the latents' and P's place");

// grid: 4 CTAs (two output halves, two row tiles) per (pair of row tiles, split),
// the ones with the most keys first; CTAs beyond the last one leave at once.
__global__ void __launch_bounds__(kPTileThreads, 1) paged_tiles_kernel(const PagedArgs a) {
    constexpr int kMmaWarp = kPSoftWarps, kCopyWarp = kPSoftWarps + 1;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    PagedTilesSmem& S = *reinterpret_cast<PagedTilesSmem*>(smem_raw);
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
    const int half = (blockIdx.x >> 1) & 1, rank = blockIdx.x & 1;
    grid_dep_launch();
    // The set-up and Q come before the wait for the decode kernel, this launch's
    // predecessor: it starts its dependents only after its own wait, so all that
    // the call's inputs come from is done by then, and nothing but the status word
    // is written before.

    paged_find<kPTileThreads / 32>(a, blockIdx.x >> 2, blockIdx.x == 0, S.work, S.sums);
    __syncthreads();
    const int64_t req = S.work.req;
    const PagedReq rq = S.work.rq;
    const int32_t nt = S.work.nt, key0 = S.work.key0, splits = S.work.splits;
    // the CTA's row tile (an item's second one may be behind the request's rows)
    const int32_t ti = 2 * S.work.item + rank;
    const int32_t n_row = rq.nq * a.heads - ti * kPM < kPM ? rq.nq * a.heads - ti * kPM : kPM;
    if (req < 0 || n_row <= 0) {
        grid_dep_wait();  // (a launch behind this one may rely on the decode kernel's end)
        return;
    }
    const int64_t flat0 = int64_t(rq.q0) * a.heads + int64_t(ti) * kPM;
    const int y_dim = kPHalf * half;

    // ---- Q: two groups of 8 rows per warp; the loads are under way while the CTA sets up
    const int q_groups = (n_row + 7) / 8;  // rows behind the last one stay what they are: they reach no other row
    U32x8 qv[2][8];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int row = 8 * (warp + 8 * n) + (lane & 7);
        if (warp + 8 * n < q_groups) paged_q_load(a, flat0 + row, row < n_row, qv[n]);
    }
    if (tid == 0) {
        for (int g = 0; g < 2; ++g) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(&S.full_x[g][b], 1);
                mbar_init(&S.full_y[g][b], 1);
                mbar_init(&S.empty_x[g][b], 1);
                mbar_init(&S.empty_o[g][b], 1);
            }
        }
        mbar_init(&S.s_full, 1);
        mbar_init(&S.s_free, kPSoftWarps);
        mbar_init(&S.p_full, kPSoftWarps);
        mbar_init(&S.p_free, 1);
        mbar_init(&S.o_done, 1);
        mbar_init(&S.q_done, kPSoftWarps);
        mbar_init(&S.drain, 1);
        mbar_init_fence();
    }
    if (warp == kMmaWarp) tmem_alloc(&S.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;

    // ---- decoded tiles: a block of 128 channels is 2 KB of each of 16 key groups
    const int64_t tile0 = req * a.span + (key0 - paged_base(a, rq)) / kPN;
    auto copy_block = [&](uint64_t* bar, int g, int b, const uint8_t* src, const uint8_t* fl) {
        if (lane == 0) mbar_arrive_expect_tx(bar, kPN * 128 * 2 + (fl ? kPFlagBytes : 0));
        __syncwarp();
        if (lane == 0)
            bulk_g2s(S.c[g] + b * kPBlockBytes, src + b * kPBlockBytes, kPBlockBytes, bar);
        else if (lane == 1 && fl)
            bulk_g2s(&S.flags[g], fl, kPFlagBytes, bar);
        __syncwarp();
    };
    const uint8_t* x_src = a.tiles + tile0 * kPTileBytes + (1 - half) * (kPTileBytes / 2);

    // ---- Q to f16 times a power of two per row: the other half to its place, the
    // own half by way of the second group of latents into TMEM
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        if (warp + 8 * n >= q_groups) continue;
        const int row = 8 * (warp + 8 * n) + (lane & 7), piece = lane >> 3;
        const int qs = paged_q_exponent(qv[n]);
        if (piece == 0) S.q_scale[row] = paged_q_scale(a, qs);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint8_t* dst = (i >= 4) == (half == 1) ? S.c[1] : S.qx;  // channels 256 .. 511 are the own half of half 1
            paged_q_store(dst + (row >> 3) * 4096 + (8 * (i & 3) + 2 * piece) * 128 + (row & 7) * 16, qv[n][i], qs);
        }
    }
    fence_async_smem();
    grid_dep_wait();  // the tiles
    if (warp == kCopyWarp && nt > 0)
        for (int b = 0; b < 2; ++b) copy_block(&S.full_x[0][b], 0, b, x_src, nullptr);
    __syncthreads();

    if (warp < kPSoftWarps) {
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
            mbar_arrive(&S.s_free);  // phase 0: Q is in place
        }

        // ---- key tiles
        int32_t lo_r = 0, hi_r = INT32_MAX;  // the row's keys
        if (row_on) {
            hi_r = rq.len - rq.nq + (ti * kPM + row) / a.by_heads + 1;
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
            const bool grew = top > m + kPGrow;
            if (j > 0) {  // the previous tile's O, which the next products' P and a new base have to come after
                ok = __all_sync(0xffffffffu, mbar_wait(&S.p_free, (j - 1) & 1, a.wlim));
                if (!ok) break;
                tc_fence_after();
            }
            if (__any_sync(0xffffffffu, grew)) {
                const float mn = grew ? top - kPBase : m;
                const float alpha = !grew ? 1.f : m == -INFINITY ? 0.f : ex2(m - mn);
                if (j > 0) {
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
                    bulk_s2g(a.part_o + (S.work.part0 + rank * kPM + row) * kPD + y_dim, stage, kPHalf * 4);
                if (half == 0) {
                    if (!whole)
                        a.part_lse[S.work.part0 + rank * kPM + row] = lse2;
                    else if (a.lse)
                        a.lse[flat] = lse2 * kLn2;
                }
                bulk_s2g_wait();
            }
        }
    } else if (tid == 32 * kMmaWarp) {
        // ================= MMA issue
        constexpr uint32_t id_s = idesc_f16(kPM, kPN, 0, false, false), id_o = idesc_f16(kPM, 128, 0, false, true);
        // descriptors; a step of 16 along K is 256 bytes (K-major) or two 8-key groups (MN-major)
        const uint64_t dq0 = umma_desc(smem_u32(S.qx), 128, 4096), dp0 = umma_desc(smem_u32(S.p), 128, 2048);
        const uint64_t dk[2] = {umma_desc(smem_u32(S.c[0]), 128, 2048), umma_desc(smem_u32(S.c[1]), 128, 2048)};
        const uint64_t dv[2] = {umma_desc(smem_u32(S.c[0]), 2048, 128), umma_desc(smem_u32(S.c[1]), 2048, 128)};
        // (a value the compiler cannot know: it would keep every step's descriptor of the loop in registers, and spill)
        auto fresh = [](uint64_t v) {
            asm volatile("" : "+l"(v));
            return v;
        };
        bool ok = true;
        auto o_mma = [&](int32_t j, int b) {  // O += P Y of tile j, 128 channels
            if (b == 0) ok = ok && mbar_wait(&S.p_full, j & 1, a.wlim);
            if (!ok) return;
            tc_fence_after();
            const uint64_t d = fresh(j & 1 ? dv[1] : dv[0]) + b * (kPBlockBytes >> 4), dp = fresh(dp0);
#pragma unroll
            for (int k = 0; k < kPN / 16; ++k)
                mma_f16_ss(tmem + kColO + 128 * b, dp + k * (256 >> 4), d + k * (4096 >> 4), id_o, k > 0 || j > 0);
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
                    mma_f16_ss(tmem + kColS, dq + (8 * b + k) * (256 >> 4), d + b * (kPBlockBytes >> 4) + k * (256 >> 4), id_s, k > 0 || b > 0);
                tc_commit(&S.empty_x[g][b]);
            }
            if (ok && j > 0) {
                o_mma(j - 1, 0);
                if (ok && j + 1 < nt) tc_commit(&S.empty_o[g ^ 1][0]);
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                ok = ok && mbar_wait(&S.full_y[g][b], ph, a.wlim);
                if (!ok) break;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_f16_ts(tmem + kColS, tmem + kColQ + 8 * (8 * b + k), d + b * (kPBlockBytes >> 4) + k * (256 >> 4), id_s, true);
            }
            if (ok) tc_commit(&S.s_full);
            if (ok && j > 0) {
                o_mma(j - 1, 1);
                tc_commit(&S.p_free);
                if (j + 1 < nt) tc_commit(&S.empty_o[g ^ 1][1]);
            }
        }
        if (nt > 0) {
            for (int b = 0; b < 2; ++b) o_mma(nt - 1, b);
            if (ok) tc_commit(&S.o_done);
            if (!ok) record(a.st, CSA2_ERR_TIMEOUT, 8, int32_t(req), ti);
            // after a give-up anywhere, TMEM and shared memory stay until the MMAs in flight are done
            tc_commit(&S.drain);
            mbar_wait(&S.drain, 0, kDrainNs);
        }
    } else if (warp == kCopyWarp) {
        // ================= tile copies (the first X blocks are under way)
        const uint8_t* y_src = a.tiles + tile0 * kPTileBytes + half * (kPTileBytes / 2);
        const uint8_t* flags = a.flags + tile0 * kPFlagBytes;
        bool ok = true;
        int32_t last_x[2][2] = {{-1, -1}, {-1, -1}}, last_y[2][2] = {{-1, -1}, {-1, -1}};  // tiles copied last
        for (int32_t j = 0; j < nt && ok; ++j) {
            const int g = j & 1;
            const uint32_t ph = (j >> 1) & 1;
            for (int b = 0; b < 2; ++b) {
                if (j == 1 && b == 0) ok = __all_sync(0xffffffffu, mbar_wait(&S.q_done, 0, a.wlim));
                if (j > 1) ok = __all_sync(0xffffffffu, mbar_wait(&S.empty_o[g][b], ph ^ 1, a.wlim));
                if (!ok) break;
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
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Decodes the pages of every request once into tiles of 128 keys (layout:
// kPTileBytes).  1.8 KB of traffic per FP4 key: 1 % of the attention's time at 512
// tokens x 64 heads.  grid (blocks of a request, requests).  A block takes 32 keys
// at a time, a warp 8 keys and half of their channels: with whole tiles per
// block, calls of a few tiles took 3 us longer.  The requests' real lengths are
// not the host's, and the few-row kernel's requests have no tiles: the blocks of
// a request walk over its tiles, since 17,000 blocks, most of them without work,
// cost 13 us.
template <bool FP8>
__global__ void __launch_bounds__(256) paged_decode_kernel(const PagedArgs a) {
    __shared__ uint32_t s_nan[2], s_hidden[2];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t req = blockIdx.y;
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5, k8 = lane & 7, piece = lane >> 3;
    PagedReq rq;
    if (!paged_request(a, req, rq, nullptr) || !paged_mine(a, rq)) return;
    const int32_t base = paged_base(a, rq), quarters = (rq.len - base + 31) / 32;
    if (tid < 2) s_nan[tid] = s_hidden[tid] = 0;
    __syncthreads();
    int par = 0;
    for (int32_t n = blockIdx.x; n < ((quarters + 3) & ~3); n += gridDim.x, par ^= 1) {
        const int32_t j = n >> 2, quarter = n & 3;
        const int key = 32 * quarter + 8 * (warp >> 1) + k8, half = warp & 1;
        uint8_t* dst = a.tiles + (req * a.span + j) * kPTileBytes + half * (kPTileBytes / 2) + (key >> 3) * 2048 + k8 * 16;
        const int32_t p = base + j * kPN + key;
        int64_t row = -1;
        if (p < rq.len) {
            const int32_t page = p / a.by_page, id = a.table[req * a.max_pages + page];
            if (id >= 0 && id < a.n_rows_pages)
                row = int64_t(id) * a.page + (p - page * a.page);
            else if (piece == 0 && half == 0)
                record(a.st, CSA2_ERR_DEVICE_BOUNDS, CHK_PAGE, int32_t(req), id);
        }
        constexpr int NP = FP8 ? 4 : 2;  // 64-byte parts of the half row; a lane has 16 bytes of each
        uint4 v[NP], sc = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < NP; ++e)
            v[e] = row >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.codes + row * (FP8 ? kPD : kPD / 2) + 64 * (NP * half + e)) + piece)
                            : make_uint4(0, 0, 0, 0);
        if (!FP8 && row >= 0) sc = __ldg(reinterpret_cast<const uint4*>(a.scales + row * (kPD / 16)) + half);
        uint32_t bad = 0;
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            const uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
            // chunks of 8 channels: FP4 4 piece .. of each 16, FP8 2 piece .. of each 8
            constexpr int NC = FP8 ? 2 : 4;
            uint8_t* to = dst + (FP8 ? (e >> 1) * kPBlockBytes + (8 * (e & 1) + 2 * piece) * 128 : e * kPBlockBytes + 4 * piece * 128);
            uint32_t o[4 * NC];
            if (FP8) {
                const uint32_t n4 = e4m3_nan4(w[0]) | e4m3_nan4(w[1]) | e4m3_nan4(w[2]) | e4m3_nan4(w[3]);
                bad |= n4;
#pragma unroll
                for (int m = 0; m < 4; ++m) e4m3x4_f16(n4 ? 0u : w[m], o + 2 * m);
            } else {
                const uint32_t lo = e ? sc.z : sc.x, hi = e ? sc.w : sc.y;  // the 8 scales of 128 channels
                const uint32_t s2 = ((piece & 2 ? hi : lo) >> (16 * (piece & 1))) & 0xFFFFu;
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
                *reinterpret_cast<uint4*>(to + c * 128) = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
        if (bad) atomicOr(&s_nan[par], 1u << (key & 31));
        if (row < 0) atomicOr(&s_hidden[par], 1u << (key & 31));
        __syncthreads();
        if (tid == 0) {  // (the next 32 keys use the other pair)
            uint32_t* fl = reinterpret_cast<uint32_t*>(a.flags + (req * a.span + j) * kPFlagBytes);
            fl[quarter] = s_hidden[par], fl[4 + quarter] = s_nan[par];
            s_hidden[par] = s_nan[par] = 0;
        }
    }
}

csa2_status paged_tiles_launch(const PagedArgs& a, bool fp8, unsigned grid, cudaStream_t s) {
    static std::atomic<bool> done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CSA2_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(paged_tiles_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(sizeof(PagedTilesSmem))) != cudaSuccess)
            return CSA2_ERR_CUDA;
        done[dev].store(true, std::memory_order_release);
    }
    timer_begin(K_PAGED_DECODE, s);
    const int64_t quarters = int64_t(a.span) * 4, some = 4096 / a.n_req > 32 ? 4096 / a.n_req : 32;
    const cudaError_t e1 = launch(fp8 ? paged_decode_kernel<true> : paged_decode_kernel<false>,
                                  dim3(unsigned(quarters < some ? quarters : some), unsigned(a.n_req)), 256, 0, s, 1, a);
    timer_end(K_PAGED_DECODE, s);
    if (e1 != cudaSuccess) return CSA2_ERR_CUDA;
    timer_begin(K_PAGED_ATTN, s);
    const cudaError_t e2 = launch(paged_tiles_kernel, dim3(grid), kPTileThreads, sizeof(PagedTilesSmem), s, 1, a);
    timer_end(K_PAGED_ATTN, s);
    return e2 == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

}  // namespace csa2
