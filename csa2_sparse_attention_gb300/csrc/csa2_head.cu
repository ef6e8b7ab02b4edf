// Norms of every head's query and of the latents, and their rotation by
// position, in one pass: queries leave in bf16, latents as rows of the cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w,   (y_2i, y_2i+1) turned by p theta^(-2i/512)
//
// HBM bound: 1 KB in and 1 KB out per (token, head).  A warp has a row of 512
// channels, 16 contiguous ones a lane (one 32-byte load and store), so that the
// norm is one warp's sum.  Latents have a warp each.
//
// Latents are rounded to 4 or 8 bits as 64-bit arithmetic would: the fp32
// result carries a bound of its error, and a scale or a code that lies nearer to
// a border than that is computed again in fp64.
//
// Measured, norm and rotation: 4096 tokens x 64 heads 83 us (6.1 TB/s, 90 % of the
// card's copy rate; the norm or the rotation alone 79 and 80), 512 x 64 16.4 us,
// 16 x 64 4.8 us, 1 x 64 2.7 us (a launch is 2.2).
#include "csa2_common.cuh"
#include "csa2_round.cuh"
#include "csa2_timer.cuh"

#include <algorithm>
#include <cfloat>
#include <climits>

namespace csa2 {

constexpr int kHD = CSA2_LATENT_DIM;
constexpr int kHWarps = 8;

struct HeadArgs {
    const uint8_t* q;
    const uint8_t* q_weight;
    uint8_t* q_out;
    const uint8_t* lat;
    const uint8_t* lat_weight;
    const int64_t* pos;
    const float2* table;   // null: no rotation
    const int64_t* dst;
    uint8_t* codes;
    uint8_t* scales;
    Status* st;
    int64_t q_stride, lat_stride, n, max_pos, n_rows;  // strides in elements
    int64_t lat_blocks;                                // blocks that take latents,
    uint32_t lat_every;                                // each at a multiple of this
    int32_t heads, per_unit, warps;                    // heads of a warp, warps of a token in a block
    int32_t tokens, parts;                             // tokens of a block, blocks of a token
    int32_t n_hi;
    float eps;
};

struct Row32 {
    uint32_t w[8];
};
// 32 bytes from or to a 16-byte aligned address: one access where it is 32-byte
// aligned.  (Plain loads: the outputs may be the inputs.)
__device__ __forceinline__ Row32 load32(const uint8_t* p) {
    Row32 v;
    if ((reinterpret_cast<uintptr_t>(p) & 16) == 0) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                       "=r"(v.w[7])
                     : "l"(p));
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 16);
        v.w[0] = a.x, v.w[1] = a.y, v.w[2] = a.z, v.w[3] = a.w, v.w[4] = b.x, v.w[5] = b.y, v.w[6] = b.z, v.w[7] = b.w;
    }
    return v;
}
__device__ __forceinline__ void store32(uint8_t* p, const Row32& v) {
    if ((reinterpret_cast<uintptr_t>(p) & 16) == 0) {
        asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]),
                     "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7]), "l"(p) : "memory");
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
        *reinterpret_cast<uint4*>(p + 16) = make_uint4(v.w[4], v.w[5], v.w[6], v.w[7]);
    }
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Sum of a lane's 16 squares, in pairs: off by 5 * 2^-24 of it at most.
__device__ __forceinline__ float squares(const Row32& x) {
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = fmaf(bf16_lo(x.w[e]), bf16_lo(x.w[e]), bf16_hi(x.w[e]) * bf16_hi(x.w[e]));
    return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}
// 1 / sqrt(mean + eps); a row of zeros stays one, also where eps is 0.
__device__ __forceinline__ float root_of(float ss, float eps) { return ss == 0.f ? 0.f : 1.0f / sqrtf(fmaf(ss, 1.0f / kHD, eps)); }

// Cosines and sines of a lane's 8 pairs at position p (csa2_rope_table_init's
// table: the angle of p = 1024 hi + lo by addition).
__device__ __forceinline__ void turns(const HeadArgs& a, int64_t p, int lane, float (&c)[8], float (&s)[8]) {
    const float4* th = reinterpret_cast<const float4*>(a.table + (p >> 10) * (kHD / 2) + 8 * lane);
    const float4* tl = reinterpret_cast<const float4*>(a.table + (int64_t(a.n_hi) + (p & 1023)) * (kHD / 2) + 8 * lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 h = __ldg(th + j), l = __ldg(tl + j);
        c[2 * j] = fmaf(h.x, l.x, -h.y * l.y), s[2 * j] = fmaf(h.y, l.x, h.x * l.y);
        c[2 * j + 1] = fmaf(h.z, l.z, -h.w * l.w), s[2 * j + 1] = fmaf(h.w, l.z, h.z * l.w);
    }
}

template <bool NORM, bool TURN>
struct HeadTurns {
    float4 v[TURN ? kHWarps : 1][TURN && NORM ? 8 : TURN ? 4 : 1][TURN ? 32 : 1];
};

// Queries of a block: of one token, or of a few where it has few heads; a token's
// warps take per_unit heads each.  What a token's heads are multiplied by stands
// in shared memory, made by a thread a pair, so that a lane's own registers hold
// nothing but rows and 32 warps fit a multiprocessor (cosines, sines and weights
// in registers, 24 warps: 95 us at 4096 tokens x 64 heads; so: 83):
//   norm and rotation  (w0 c, w0 s, w1 c, w1 s) of a pair,
//   rotation alone     (c, s) of two pairs.
// 16 bytes a lane at a time, without conflicts.  1 / sqrt(mean + eps) comes last,
// so that the products need not wait for the warp's sum.
template <bool NORM, bool TURN>
__device__ __forceinline__ void head_queries(const HeadArgs& a, int64_t block, HeadTurns<NORM, TURN>& of) {
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
    const int slot = warp / a.warps;  // the token's place in the block
    const int64_t t0 = a.tokens > 1 ? block * a.tokens : int64_t(uint32_t(block) / uint32_t(a.parts)), t = t0 + slot;
    const int unit = a.tokens > 1 ? warp - slot * a.warps : int(block - t0 * a.parts) * kHWarps + warp;
    const int h0 = unit * a.per_unit, h1 = h0 + a.per_unit < a.heads ? h0 + a.per_unit : a.heads;
    const bool on = t < a.n && h0 < a.heads;
    const uint8_t* src = a.q + (t * a.q_stride + int64_t(h0) * kHD) * 2 + 32 * lane;
    uint8_t* dst = a.q_out + (t * a.heads + h0) * int64_t(kHD * 2) + 32 * lane;
    Row32 x, ahead, w;  // the next two heads are under way
    if (on) {
        x = load32(src);
        if (h0 + 1 < h1) ahead = load32(src + kHD * 2);
        if (NORM && !TURN) w = load32(a.q_weight + 32 * lane);
    }
    const int64_t p = on && a.pos != nullptr ? __ldg(a.pos + t) : 0;
    if (TURN) {  // cosine and sine by addition of the table's two angles
        const uint32_t wp = NORM ? *reinterpret_cast<const uint32_t*>(a.q_weight + 4 * tid) : 0;
        for (int i = 0; i < a.tokens; ++i) {
            if (t0 + i >= a.n) break;
            const int64_t at = __ldg(a.pos + t0 + i);
            if (at < 0 || at >= a.max_pos) continue;
            const float2 h = __ldg(a.table + (at >> 10) * (kHD / 2) + tid), l = __ldg(a.table + (int64_t(a.n_hi) + (at & 1023)) * (kHD / 2) + tid);
            const float c = fmaf(h.x, l.x, -h.y * l.y), s = fmaf(h.y, l.x, h.x * l.y);
            if (NORM)
                of.v[i][tid & 7][tid >> 3] = make_float4(bf16_lo(wp) * c, bf16_lo(wp) * s, bf16_hi(wp) * c, bf16_hi(wp) * s);
            else
                reinterpret_cast<float2*>(&of.v[i][(tid & 7) >> 1][tid >> 3])[tid & 1] = make_float2(c, s);
        }
        __syncthreads();
    }
    if (!on) return;
    if (p < 0 || (TURN && p >= a.max_pos)) {
        if (p != -1 && h0 == 0 && lane == 0) record(a.st, CSA2_ERR_DEVICE_BOUNDS, CHK_POSITION, int32_t(t), int32_t(p));
        return;
    }
    for (int h = h0; h < h1; ++h) {
        Row32 v = x;
        x = ahead;
        if (h + 2 < h1) ahead = load32(src + 2 * kHD * 2);
        src += kHD * 2;
        const float rs = NORM ? root_of(sum_lanes(squares(v)), a.eps) : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x0 = bf16_lo(v.w[e]), x1 = bf16_hi(v.w[e]);
            float y0, y1;
            if (NORM && TURN) {
                const float4 c = of.v[slot][e][lane];
                y0 = fmaf(x0, c.x, -x1 * c.w) * rs, y1 = fmaf(x0, c.y, x1 * c.z) * rs;
            } else if (TURN) {
                const float2 c = reinterpret_cast<const float2*>(&of.v[slot][e >> 1][lane])[e & 1];
                y0 = fmaf(x0, c.x, -x1 * c.y), y1 = fmaf(x0, c.y, x1 * c.x);
            } else {
                y0 = NORM ? x0 * bf16_lo(w.w[e]) * rs : x0, y1 = NORM ? x1 * bf16_hi(w.w[e]) * rs : x1;
            }
            v.w[e] = bf16x2_of(y0, y1);
        }
        store32(dst, v);
        dst += kHD * 2;
    }
}

// 1 / sqrt(mean + eps) in fp64, by the warp: rs, off by 2^-21 at most, improved by
// two of Newton's steps (the error becomes 1.5 times its square each time).
__device__ __forceinline__ double root_of64(const Row32& x, float rs, float eps) {
    double ss[2] = {0.0, 0.0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // (the square of a bf16 number is exact in fp32)
        ss[e & 1] += double(bf16_lo(x.w[e]) * bf16_lo(x.w[e]));
        ss[e & 1] += double(bf16_hi(x.w[e]) * bf16_hi(x.w[e]));
    }
    double v = ss[0] + ss[1];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (v == 0.0) return 0.0;
    v = fma(v, 1.0 / kHD, double(eps));
    double r = double(rs);
#pragma unroll
    for (int i = 0; i < 2; ++i) r = fma(r, 0.5 * fma(-v * r, r, 1.0), r);
    return r;
}

// A token's latent.  The error of y, relative to |h0| + |h1| of its pair (h the
// normed values): the sum of squares 10 * 2^-24 (5 in a lane, 5 over lanes), so
// its root 5; mean and eps, root and reciprocal 2 together; the product 1 (x w
// is exact); the rotation 5 (cosines within 1.5 * 2^-23 of their values after the
// angles' addition, two roundings).  13 * 2^-24 < 2^-20.
//
// Where the values within that error of y have different codes, that value is
// computed again in fp64: in a few of a thousand groups.  (All 16 of the group took
// 8 us, which a call of 16 tokens as often had as not.)
template <bool FP8>
__device__ __forceinline__ void head_latent(const HeadArgs& a, int64_t t) {
    const int lane = lane_id();
    const Row32 x = load32(a.lat + t * a.lat_stride * 2 + 32 * lane);
    const bool norm = a.lat_weight != nullptr, turn = a.table != nullptr;
    Row32 w;
#pragma unroll
    for (int e = 0; e < 8; ++e) w.w[e] = 0x3F803F80u;
    if (norm) w = load32(a.lat_weight + 32 * lane);
    const int64_t p = a.pos != nullptr ? __ldg(a.pos + t) : 0, row = a.dst != nullptr ? __ldg(a.dst + t) : t;
    if (p < 0 || (turn && p >= a.max_pos)) {
        if (p != -1 && lane == 0) record(a.st, CSA2_ERR_DEVICE_BOUNDS, CHK_POSITION, int32_t(t), int32_t(p));
        return;
    }
    if (row < 0 || row >= a.n_rows) {
        if (row != -1 && lane == 0) record(a.st, CSA2_ERR_DEVICE_BOUNDS, CHK_DST_ROW, int32_t(t), int32_t(row));
        return;
    }
    const float rs = norm ? root_of(sum_lanes(squares(x)), a.eps) : 1.f;
    float y[16], bnd[8];  // bnd[j]: how far pair j's values may be off
    float c[8], s[8];
    if (turn) turns(a, p, lane, c, s);
    bool whole = true;  // no NaN or infinity
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float h0 = bf16_lo(x.w[e]) * bf16_lo(w.w[e]) * rs, h1 = bf16_hi(x.w[e]) * bf16_hi(w.w[e]) * rs;
        bnd[e] = norm || turn ? 0x1p-20f * (fabsf(h0) + fabsf(h1)) : 0.f;
        y[2 * e] = turn ? fmaf(h0, c[e], -h1 * s[e]) : h0;
        y[2 * e + 1] = turn ? fmaf(h0, s[e], h1 * c[e]) : h1;
        whole = whole && fabsf(y[2 * e]) <= FLT_MAX && fabsf(y[2 * e + 1]) <= FLT_MAX && bnd[e] <= FLT_MAX;
    }
    double rs64 = -1.0;  // not there yet
    auto need64 = [&](bool some) {  // by the whole warp
        if (rs64 >= 0.0 || !__any_sync(0xffffffffu, some)) return;
        rs64 = norm ? root_of64(x, rs, a.eps) : 1.0;
    };
    auto exact = [&](int e) {  // value e of the lane in fp64
        uint32_t xw = x.w[0], ww = w.w[0];
#pragma unroll
        for (int j = 1; j < 8; ++j)
            if (j == e >> 1) xw = x.w[j], ww = w.w[j];
        const double h0 = double(bf16_lo(xw) * bf16_lo(ww)) * rs64, h1 = double(bf16_hi(xw) * bf16_hi(ww)) * rs64;
        if (!turn) return e & 1 ? h1 : h0;
        const double2* t64 = reinterpret_cast<const double2*>(a.table + int64_t(a.n_hi + 1024) * (kHD / 2));
        const int j = 8 * lane + (e >> 1);
        const double2 h = t64[(p >> 10) * (kHD / 2) + j], l = t64[(int64_t(a.n_hi) + (p & 1023)) * (kHD / 2) + j];
        const double c64 = fma(h.x, l.x, -h.y * l.y), s64 = fma(h.y, l.x, h.x * l.y);
        return e & 1 ? fma(h0, s64, h1 * c64) : fma(h0, c64, -h1 * s64);
    };
    uint32_t sb = 0, cw[4] = {0, 0, 0, 0}, risky = 0;  // risky: a bit per value
    if (FP8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cw[j >> 1] |= e4m3x2_rn_sat(y[2 * j], y[2 * j + 1]) << (16 * (j & 1));
            const float a0 = fabsf(y[2 * j]), a1 = fabsf(y[2 * j + 1]);
            const uint32_t differ = e4m3x2_rn_sat(fmaxf(a0 - bnd[j], 0.f), fmaxf(a1 - bnd[j], 0.f)) ^ e4m3x2_rn_sat(a0 + bnd[j], a1 + bnd[j]);
            if (whole) risky |= (differ & 0xFF ? 1u : 0u) << (2 * j) | (differ >> 8 ? 1u : 0u) << (2 * j + 1);
        }
        need64(risky != 0);
        for (; risky != 0; risky &= risky - 1) {
            const int e = __ffs(risky) - 1;
            const double z = exact(e);
            const uint32_t code = e4m3_rne_f64(fabs(z)) | (signbit(z) ? 0x80u : 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i == e >> 2) cw[i] = (cw[i] & ~(0xFFu << (8 * (e & 3)))) | code << (8 * (e & 3));
        }
    } else {
        float amax = 0.f, bmax = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(y[e]));
#pragma unroll
        for (int j = 0; j < 8; ++j) bmax = fmaxf(bmax, bnd[j]);
        // amax / 6 by a multiply: its error (< 2^-22 relative) sits inside mq
        const float q6 = amax * (1.0f / 6.0f), mq = fmaf(q6, 0x1p-20f, bmax * (1.0f / 6.0f) * 1.001f);
        const uint32_t span = e4m3x2_rn_sat(fmaxf(q6 - mq, 0.f), q6 + mq), lo = span & 0xFF, hi = span >> 8;
        sb = whole ? e4m3x2_rn_sat(q6, 0.f) & 0xFF : 0x7Fu;  // a scale of NaN: what attends to the latent gets NaN
        const bool unsure = whole && lo != hi;
        need64(unsure);
        if (unsure) {  // the largest of those that may be the largest one
            double top = 0.0;
#pragma unroll
            for (int e = 0; e < 16; ++e) risky |= (fabsf(y[e]) + 2.f * bmax >= amax ? 1u : 0u) << e;
            for (; risky != 0; risky &= risky - 1) top = fmax(top, fabs(exact(__ffs(risky) - 1)));
            sb = e4m3_rne_f64(top / 6.0);
        }
        const float sc = e4m3_value(sb);
        float inv = 0.f;
        if (sc > 0.f) {
            inv = __frcp_rn(sc);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float r0 = y[2 * j] * inv, r1 = y[2 * j + 1] * inv;
                cw[j >> 2] |= e2m1x2_rn_sat(r0, r1) << (8 * (j & 3));
                const float a0 = fabsf(r0), a1 = fabsf(r1);
                const float m0 = fmaf(a0, 0x1p-22f, bnd[j] * inv * 1.001f), m1 = fmaf(a1, 0x1p-22f, bnd[j] * inv * 1.001f);
                const uint32_t differ = e2m1x2_rn_sat(fmaxf(a0 - m0, 0.f), fmaxf(a1 - m1, 0.f)) ^ e2m1x2_rn_sat(a0 + m0, a1 + m1);
                risky |= (differ & 0xF ? 1u : 0u) << (2 * j) | (differ >> 4 ? 1u : 0u) << (2 * j + 1);
            }
        }
        need64(risky != 0);
        for (; risky != 0; risky &= risky - 1) {
            const int e = __ffs(risky) - 1;
            const double z = exact(e);
            const uint32_t code = e2m1_code_f64(z, double(sc));
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i == e >> 3) cw[i] = (cw[i] & ~(0xFu << (4 * (e & 7)))) | code << (4 * (e & 7));
        }
    }
    if (FP8) {
        *reinterpret_cast<uint4*>(a.codes + row * kHD + 16 * lane) = make_uint4(cw[0], cw[1], cw[2], cw[3]);
    } else {
        *reinterpret_cast<uint2*>(a.codes + row * (kHD / 2) + 8 * lane) = make_uint2(cw[0], cw[1]);
        a.scales[row * (kHD / 16) + lane] = uint8_t(sb);
    }
}

template <bool NORM, bool TURN, bool FP8>
__global__ void __launch_bounds__(32 * kHWarps, 4) head_norm_rope_kernel(const HeadArgs a) {
    __shared__ HeadTurns<NORM, TURN> q_turns;
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t at = blockIdx.x / a.lat_every, lat_blocks = uint32_t(a.lat_blocks);
    if (at < lat_blocks && at * a.lat_every == blockIdx.x) {
        const int64_t t = int64_t(at) * kHWarps + (threadIdx.x >> 5);
        if (t < a.n) head_latent<FP8>(a, t);
        return;
    }
    head_queries<NORM, TURN>(a, blockIdx.x - (at + 1 < lat_blocks ? at + 1 : lat_blocks), q_turns);
}

}  // namespace csa2

using namespace csa2;

extern "C" csa2_status csa2_head_norm_rope(const void* q, int64_t q_stride, int n_heads, const void* q_weight, void* q_out,
                                           const void* latents, int64_t lat_stride, const void* lat_weight, int64_t n, float eps,
                                           const int64_t* pos, const void* rope_table, int64_t rope_max_pos, int fmt,
                                           const int64_t* dst_row, int64_t n_rows, uint8_t* dst_codes, uint8_t* dst_scales,
                                           void* ws, size_t ws_bytes, csa2_stream_t stream) {
    if (n < 0 || n_rows < 0 || !(eps >= 0.f) || !(eps <= FLT_MAX)) return CSA2_ERR_INVALID_ARG;
    if (!ws || ws_bytes < CSA2_STATUS_BYTES || !aligned16(ws)) return CSA2_ERR_WORKSPACE;
    if (!q && !latents) return CSA2_ERR_INVALID_ARG;
    if (n > (int64_t(1) << 22)) return CSA2_ERR_UNSUPPORTED;
    if ((q == nullptr) != (q_out == nullptr) || (!q && q_weight) || (!latents && lat_weight)) return CSA2_ERR_INVALID_ARG;
    for (const void* p : {q, q_weight, static_cast<const void*>(q_out), latents, lat_weight, static_cast<const void*>(pos), rope_table,
                          static_cast<const void*>(dst_row), static_cast<const void*>(dst_codes),
                          static_cast<const void*>(dst_scales)})
        if (!aligned16(p)) return CSA2_ERR_INVALID_ARG;
    if (rope_table && (!pos || rope_max_pos <= 0 || rope_max_pos > (int64_t(1) << 31))) return CSA2_ERR_INVALID_ARG;
    if (q) {
        if (n_heads < 1 || n_heads > 128) return CSA2_ERR_UNSUPPORTED;
        const int64_t row = int64_t(n_heads) * kHD;
        if (q_stride < row || q_stride % 8 || q_stride > (int64_t(1) << 31)) return CSA2_ERR_INVALID_ARG;
    }
    if (latents) {
        if (fmt != CSA2_FMT_FP4 && fmt != CSA2_FMT_FP8) return CSA2_ERR_UNSUPPORTED;
        if (lat_stride < kHD || lat_stride % 8 || lat_stride > (int64_t(1) << 31)) return CSA2_ERR_INVALID_ARG;
        if (!dst_codes || (fmt == CSA2_FMT_FP4) != (dst_scales != nullptr)) return CSA2_ERR_INVALID_ARG;
        if (!dst_row && n > n_rows) return CSA2_ERR_INVALID_ARG;
    }
    if (n == 0) return CSA2_OK;
    // what is written lies apart from what is read and from each other; or the queries are turned in place
    const int64_t q_row = q ? int64_t(n_heads) * kHD : 0;
    const bool in_place = q == q_out && q_stride == q_row;
    const int64_t row_codes = fmt == CSA2_FMT_FP4 ? kHD / 2 : kHD, cells = latents ? n_rows : 0;
    const Span outs[] = {{q_out, n * q_row * 2}, {dst_codes, cells * row_codes}, {dst_scales, cells * (kHD / 16)}};
    const int64_t positions = rope_table ? ceil_div<int64_t>(rope_max_pos, 1024) + 1024 : 0;
    const Span ins[] = {{in_place ? nullptr : q, q ? ((n - 1) * q_stride + q_row) * 2 : 0},
                        {latents, latents ? ((n - 1) * lat_stride + kHD) * 2 : 0},
                        {q_weight, kHD * 2},
                        {lat_weight, kHD * 2},
                        {pos, n * 8},
                        {dst_row, n * 8},
                        {rope_table, positions * (kHD / 2) * 24}};
    if (!apart(outs, ins)) return CSA2_ERR_INVALID_ARG;
    HeadArgs a{};
    a.q = static_cast<const uint8_t*>(q);
    a.q_weight = static_cast<const uint8_t*>(q_weight);
    a.q_out = static_cast<uint8_t*>(q_out);
    a.lat = static_cast<const uint8_t*>(latents);
    a.lat_weight = static_cast<const uint8_t*>(lat_weight);
    a.pos = pos;
    a.table = static_cast<const float2*>(rope_table);
    a.dst = dst_row;
    a.codes = dst_codes;
    a.scales = dst_scales;
    a.st = static_cast<Status*>(ws);
    a.q_stride = q_stride;
    a.lat_stride = lat_stride;
    a.n = n;
    a.max_pos = rope_max_pos;
    a.n_rows = n_rows;
    a.n_hi = rope_table ? int(ceil_div<int64_t>(rope_max_pos, 1024)) : 0;
    a.eps = eps;
    a.lat_blocks = latents ? ceil_div<int64_t>(n, kHWarps) : 0;
    int64_t q_blocks = 0;
    if (q) {
        // A power of two of heads to a warp, as many as leave every multiprocessor
        // twice the warps it holds: 4096 tokens x 64 heads with 4 / 8 / 16 of them
        // 89 / 83 / 87 us; 4096 x 16 with 4 of them 30 us, with 6 (a warp of every
        // four has no head) 31.  A block has a token's warps, or several tokens'.
        a.heads = n_heads;
        a.per_unit = 1;
        while (a.per_unit < 8 && n * n_heads >= int64_t(sm_count()) * 64 * 2 * a.per_unit) a.per_unit *= 2;
        const int32_t units = ceil_div(a.heads, a.per_unit);
        a.warps = kHWarps;
        while (a.warps / 2 >= units) a.warps /= 2;
        a.tokens = kHWarps / a.warps;
        a.parts = ceil_div(units, kHWarps);
        q_blocks = a.tokens > 1 ? ceil_div<int64_t>(n, a.tokens) : n * a.parts;
    }
    if (a.lat_blocks + q_blocks > INT32_MAX) return CSA2_ERR_UNSUPPORTED;
    const dim3 grid(unsigned(a.lat_blocks + q_blocks));
    // Latents wait for more than they move: every third block has them, until they are done (4096 tokens x 64 and x 16
    // heads, 512 x 64: 82.6, 28.9, 17.3 us; all first 84.6, 30.9, 17.2; over three quarters of the grid 82.2, 29.1, 18.4).
    a.lat_every = a.lat_blocks > 0 ? unsigned(std::min<int64_t>(3, (a.lat_blocks + q_blocks) / a.lat_blocks)) : 1;
    cudaStream_t s = cudaStream_t(stream);
    timer_begin(K_HEAD, s);
    auto go = [&](auto kernel) { launch(kernel, grid, 32 * kHWarps, 0, s, 1, a); };
    const bool f8 = fmt == CSA2_FMT_FP8;
    if (a.q_weight && a.table) f8 ? go(head_norm_rope_kernel<true, true, true>) : go(head_norm_rope_kernel<true, true, false>);
    else if (a.q_weight) f8 ? go(head_norm_rope_kernel<true, false, true>) : go(head_norm_rope_kernel<true, false, false>);
    else if (a.table) f8 ? go(head_norm_rope_kernel<false, true, true>) : go(head_norm_rope_kernel<false, true, false>);
    else f8 ? go(head_norm_rope_kernel<false, false, true>) : go(head_norm_rope_kernel<false, false, false>);
    timer_end(K_HEAD, s);
    return launch_status();
}
