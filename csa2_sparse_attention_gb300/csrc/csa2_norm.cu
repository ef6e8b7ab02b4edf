// Residual addition, root-mean-square norm and E4M3 output with scales.
//
//   h = bf16(x + residual),  y = h * rsqrt(mean(h^2) + eps) * w,
//   s = max|y| / 448 per row or per 128 channels,  code = E4M3(y / s)
//
// HBM bound: 7 bytes per channel with a residual (x, residual in and out,
// code), 3 without.  A row is read once and stays in the registers of the
// threads that loaded it (16-byte chunks of 8 channels) through both
// reductions.  Rows of more than 1024 channels take a block, two chunks per
// thread, that walks over the rows and loads the next one before it reduces
// this one: the two block barriers of a row then cost no memory time.  4096 rows
// of 7168 with a residual, scales per 128: 57.8 us without that, 37.8 us with it
// (5.5 TB/s, 81 % of the copy rate).
//
// Codes are those of the exact quotient y / s (the root cancels in it): y times
// a rounded reciprocal of s, 37.3 us, put a code in ten thousand on the wrong
// side of a border, since products of bf16 numbers lie on borders that often.
#include "csa2_common.cuh"
#include "csa2_timer.cuh"

#include <cfloat>

namespace csa2 {

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float rcp_near(float x) {  // off by 2^-23
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two floats in one register pair, and their products: half of the issue slots.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// WPR warps per row, chunks t, t + 32 WPR, ... (NCH of them) of the row in
// thread t of the row's warps.
template <int WPR, int NCH, bool GROUPS>
__global__ void __launch_bounds__(WPR > 1 ? 32 * WPR : 256, WPR > 1 ? 1024 / (32 * WPR) : 1) rmsnorm_fp8_kernel(
    const uint4* __restrict__ x, int64_t x_stride, const uint4* residual, uint4* residual_out,
    const uint4* __restrict__ weight, int64_t n, int dim, float eps, uint2* __restrict__ codes, float* __restrict__ scales,
    uint4* __restrict__ y_bf16) {
    constexpr int T = 32 * WPR, RPB = WPR > 1 ? 1 : 256 / T;
    __shared__ float red[2][2][32];
    grid_dep_wait();
    grid_dep_launch();
    const int t = threadIdx.x % T, rw = threadIdx.x / T, lane = lane_id();
    const int chunks = dim / 8;
    const int64_t step = int64_t(gridDim.x) * RPB;
    int par = 0;
    // reduction over the row's warps (one, or the whole block's); the two rows in turn use two buffers, so
    // that one barrier per reduction is enough
    auto over_row = [&](float v, bool is_max, int slot) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float u = __shfl_xor_sync(0xffffffffu, v, o);
            v = is_max ? max_nan(v, u) : v + u;
        }
        if (WPR > 1) {
            if (lane == 0) red[par][slot][threadIdx.x >> 5] = v;
            __syncthreads();
            v = lane < WPR ? red[par][slot][lane] : 0.f;  // (0 is neutral for both: maxima are of absolute values)
#pragma unroll
            for (int o = WPR / 2; o; o >>= 1) {
                const float u = __shfl_xor_sync(0xffffffffu, v, o);
                v = is_max ? max_nan(v, u) : v + u;
            }
            v = __shfl_sync(0xffffffffu, v, 0);
        }
        return v;
    };
    uint4 wv[NCH], xv[NCH], rv[NCH];  // weight; the next row's x and residual
#pragma unroll
    for (int j = 0; j < NCH; ++j) wv[j] = t + T * j < chunks ? __ldg(weight + t + T * j) : make_uint4(0, 0, 0, 0);
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = t + T * j;
            const bool on = row < n && c < chunks;
            xv[j] = on ? __ldg(x + row * (x_stride / 8) + c) : make_uint4(0, 0, 0, 0);
            rv[j] = on && residual != nullptr ? residual[row * chunks + c] : make_uint4(0, 0, 0, 0);
        }
    };
    if (WPR > 1) fetch(int64_t(blockIdx.x) * RPB + rw);
    for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < n; row0 += step, par ^= 1) {
        const int64_t row = row0 + rw;
        const bool live = row < n;
        if (WPR == 1) fetch(row);
        uint4 h[NCH];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = t + T * j;
            uint32_t a[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
            const uint32_t r[4] = {rv[j].x, rv[j].y, rv[j].z, rv[j].w};
            if (residual != nullptr) {
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = bf16x2_rn(bf16_lo(a[e]) + bf16_lo(r[e]), bf16_hi(a[e]) + bf16_hi(r[e]));
            }
            h[j] = make_uint4(a[0], a[1], a[2], a[3]);
            if (residual != nullptr && live && c < chunks) residual_out[row * chunks + c] = h[j];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ss = fmaf(bf16_lo(a[e]), bf16_lo(a[e]), ss);
                ss = fmaf(bf16_hi(a[e]), bf16_hi(a[e]), ss);
            }
        }
        if (WPR > 1) fetch(row + step);
        ss = over_row(ss, false, 0);
        const float rs = 1.0f / sqrtf(ss / float(dim) + eps);
        // rs = p2 f with a power of two p2: a = h p2 w is exact (16 bits), y = a f
        const uint32_t rb = __float_as_uint(rs);
        const bool plain = (rb >> 23) - 1u < 254u;
        const float p2 = plain ? __uint_as_float(rb & 0x7F800000u) : 1.0f;
        const float f = plain ? __uint_as_float((rb & 0x007FFFFFu) | 0x3F800000u) : rs;
        const uint64_t pp = pair(p2, p2);
        uint64_t y[NCH][4];  // a
        float am = 0.f, cm[NCH];  // maxima of |a|
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const uint32_t a[4] = {h[j].x, h[j].y, h[j].z, h[j].w}, w[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w};
            cm[j] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[j][e] = mul_pair(mul_pair(pair(bf16_lo(a[e]), bf16_hi(a[e])), pp), pair(bf16_lo(w[e]), bf16_hi(w[e])));
                float lo, hi;
                unpair(y[j][e], lo, hi);
                cm[j] = max_nan(cm[j], max_nan(fabsf(lo), fabsf(hi)));
            }
            if (GROUPS) {  // 16 chunks = 128 channels: half a warp
#pragma unroll
                for (int o = 8; o; o >>= 1) cm[j] = max_nan(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], o));
            } else {
                am = max_nan(am, cm[j]);
            }
        }
        if (!GROUPS) am = over_row(am, true, 1);
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = t + T * j;
            if (!live || c >= chunks) continue;
            // y / s = 448 a / max|a|, a quotient of numbers of 19 and 16 bits: it lies on a border of two codes, or 2^-21 of
            // it away or more.  Times a reciprocal of twice the bits it is off by 2^-24 and exact where it has few bits
            // itself, so the codes are those of the exact quotient.
            const float top = GROUPS ? cm[j] : am, inv0 = rcp_near(top), inv = 448.0f * inv0;
            const float inv2 = fmaf(-top, inv, 448.0f) * inv0, s = top * (f * (1.0f / 448.0f));
            float v[8];
            const uint64_t i1 = pair(inv, inv), i2 = pair(inv2, inv2);
#pragma unroll
            for (int e = 0; e < 4; ++e) unpair(fma_pair(y[j][e], i1, mul_pair(y[j][e], i2)), v[2 * e], v[2 * e + 1]);
            if (!(plain && top >= 0x1p-90f && top <= 0x1p90f)) {  // infinities, NaN, zeros (0 / 0 is 0), the ends of the range
                const uint64_t ff = pair(f, f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float lo, hi;
                    unpair(mul_pair(y[j][e], ff), lo, hi);
                    v[2 * e] = s == 0.f ? 0.f : __fdiv_rn(lo, s);
                    v[2 * e + 1] = s == 0.f ? 0.f : __fdiv_rn(hi, s);
                }
            }
            uint2 o;
            o.x = e4m3x2_rn_sat(v[0], v[1]) | (e4m3x2_rn_sat(v[2], v[3]) << 16);
            o.y = e4m3x2_rn_sat(v[4], v[5]) | (e4m3x2_rn_sat(v[6], v[7]) << 16);
            codes[row * chunks + c] = o;
            if (y_bf16 != nullptr) {
                const uint64_t ff = pair(f, f);
                uint32_t b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float lo, hi;
                    unpair(mul_pair(y[j][e], ff), lo, hi);
                    b[e] = bf16x2_rn(lo, hi);
                }
                y_bf16[row * chunks + c] = make_uint4(b[0], b[1], b[2], b[3]);
            }
            if (GROUPS) {
                if ((c & 15) == 0) scales[row * (chunks / 16) + c / 16] = s;
            } else if (c == 0) {
                scales[row] = s;
            }
        }
    }
}

}  // namespace csa2

using namespace csa2;

extern "C" csa2_status csa2_rmsnorm_fp8(const void* x, int64_t x_stride, const void* residual, void* residual_out,
                                        const void* weight, int64_t n, int dim, float eps, int group, uint8_t* codes,
                                        float* scales, void* y_bf16, csa2_stream_t stream) {
    if (n < 0 || dim < 1 || !(eps >= 0.f) || !(eps <= FLT_MAX)) return CSA2_ERR_INVALID_ARG;
    if (dim % 8 || dim > 16384 || (group != 0 && group != 128) || (group == 128 && dim % 128)) return CSA2_ERR_UNSUPPORTED;
    if (x_stride < dim || x_stride % 8) return CSA2_ERR_INVALID_ARG;
    if ((residual == nullptr) != (residual_out == nullptr)) return CSA2_ERR_INVALID_ARG;
    if (!x || !weight || !codes || !scales) return CSA2_ERR_INVALID_ARG;
    for (const void* p : {x, residual, static_cast<const void*>(residual_out), weight, static_cast<const void*>(codes),
                          static_cast<const void*>(scales), static_cast<const void*>(y_bf16)})
        if (!aligned16(p)) return CSA2_ERR_INVALID_ARG;
    if (n == 0) return CSA2_OK;
    cudaStream_t s = cudaStream_t(stream);
    const int chunks = dim / 8;
    const bool wide = chunks > 128;
    const int threads = !wide || chunks <= 512 ? 256 : chunks <= 1024 ? 512 : 1024;
    // wide rows: the blocks that are resident at once, which then walk over the rows
    const int64_t cap = int64_t(sm_count()) * (wide ? 1024 / threads : 8), want = wide ? n : ceil_div<int64_t>(n, 8);
    const dim3 grid(unsigned(want < cap ? want : cap));
    timer_begin(K_RMSNORM, s);
    auto go = [&](auto kernel) {
        launch(kernel, grid, threads, 0, s, 1, static_cast<const uint4*>(x), x_stride, static_cast<const uint4*>(residual),
               static_cast<uint4*>(residual_out), static_cast<const uint4*>(weight), n, dim, eps,
               reinterpret_cast<uint2*>(codes), scales, static_cast<uint4*>(y_bf16));
    };
#define CSA2_NORM(W, C) \
    if (group) go(rmsnorm_fp8_kernel<W, C, true>); \
    else go(rmsnorm_fp8_kernel<W, C, false>)
    if (chunks <= 64) { CSA2_NORM(1, 2); }
    else if (!wide) { CSA2_NORM(1, 4); }
    else if (threads == 256) { CSA2_NORM(8, 2); }
    else if (threads == 512) { CSA2_NORM(16, 2); }
    else { CSA2_NORM(32, 2); }
#undef CSA2_NORM
    timer_end(K_RMSNORM, s);
    return launch_status();
}
