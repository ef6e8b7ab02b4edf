// Residual addition, root-mean-square norm and E4M3 output with scales.
//
//   h = bf16(x + residual),  y = h * rsqrt(mean(h^2) + eps) * w,
//   s = max|y| / 448 per row or per 128 channels,  code = E4M3(y / s)
//
// HBM bound: 7 bytes per channel with a residual (x, residual in and out, code), 3
// without.  A row is read once: its values stay in the registers of the
// threads that loaded them (16 bytes, 8 channels, a chunk) through both
// reductions.
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

// WPR warps per row, chunks t, t + 32 WPR, ... (NCH of them) of the row in
// thread t of the row's warps.
template <int WPR, int NCH, bool GROUPS>
__global__ void __launch_bounds__(256) rmsnorm_fp8_kernel(const uint4* __restrict__ x, int64_t x_stride, const uint4* residual,
                                                          uint4* residual_out, const uint4* __restrict__ weight, int64_t n,
                                                          int dim, float eps, uint2* __restrict__ codes,
                                                          float* __restrict__ scales, uint4* __restrict__ y_bf16) {
    constexpr int T = 32 * WPR, RPB = 256 / T;
    __shared__ float red[2][8];
    grid_dep_wait();
    grid_dep_launch();
    const int t = threadIdx.x % T, rw = threadIdx.x / T, lane = lane_id();
    const int chunks = dim / 8;
    // block reduction over the row's warps (a row has one warp, or all eight)
    auto over_row = [&](float v, bool is_max, int slot) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float u = __shfl_xor_sync(0xffffffffu, v, o);
            v = is_max ? max_nan(v, u) : v + u;
        }
        if (WPR > 1) {
            if (lane == 0) red[slot][threadIdx.x >> 5] = v;
            __syncthreads();
            v = red[slot][0];
#pragma unroll
            for (int w = 1; w < WPR; ++w) v = is_max ? max_nan(v, red[slot][w]) : v + red[slot][w];
        }
        return v;
    };
    for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < n; row0 += int64_t(gridDim.x) * RPB) {
        const int64_t row = row0 + rw;
        const bool live = row < n;
        float h[NCH][8];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = t + T * j;
            const bool on = live && c < chunks;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (on) {
                v = __ldg(x + row * (x_stride / 8) + c);
                if (residual != nullptr) {
                    const uint4 u = residual[row * chunks + c];
                    uint32_t* a = &v.x;
                    const uint32_t* b = &u.x;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        a[e] = bf16x2_rn(bf16_lo(a[e]) + bf16_lo(b[e]), bf16_hi(a[e]) + bf16_hi(b[e]));
                    residual_out[row * chunks + c] = v;
                }
            }
            const uint32_t* a = &v.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[j][2 * e] = bf16_lo(a[e]);
                h[j][2 * e + 1] = bf16_hi(a[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(h[j][e], h[j][e], ss);
        }
        ss = over_row(ss, false, 0);
        const float rs = 1.0f / sqrtf(ss / float(dim) + eps);
        float am = 0.f, cm[NCH];
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = t + T * j;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (c < chunks) w = __ldg(weight + c);
            const uint32_t* a = &w.x;
            cm[j] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[j][2 * e] = h[j][2 * e] * rs * bf16_lo(a[e]);
                h[j][2 * e + 1] = h[j][2 * e + 1] * rs * bf16_hi(a[e]);
                if (c < chunks) cm[j] = max_nan(cm[j], max_nan(fabsf(h[j][2 * e]), fabsf(h[j][2 * e + 1])));
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
            const float s = __fdiv_rn(GROUPS ? cm[j] : am, 448.0f);
            const float inv = __frcp_rn(s);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = h[j][e] * inv;
                // the reciprocal overflows for the smallest scales; 0 / 0 is 0
                if (!(inv <= FLT_MAX)) v[e] = s == 0.f ? 0.f : __fdiv_rn(h[j][e], s);
            }
            uint2 o;
            o.x = e4m3x2_rn_sat(v[0], v[1]) | (e4m3x2_rn_sat(v[2], v[3]) << 16);
            o.y = e4m3x2_rn_sat(v[4], v[5]) | (e4m3x2_rn_sat(v[6], v[7]) << 16);
            codes[row * chunks + c] = o;
            if (y_bf16 != nullptr)
                y_bf16[row * chunks + c] = make_uint4(bf16x2_rn(h[j][0], h[j][1]), bf16x2_rn(h[j][2], h[j][3]),
                                                      bf16x2_rn(h[j][4], h[j][5]), bf16x2_rn(h[j][6], h[j][7]));
            if (GROUPS) {
                if ((c & 15) == 0) scales[row * (chunks / 16) + c / 16] = s;
            } else if (c == 0) {
                scales[row] = s;
            }
        }
        if (WPR > 1) __syncthreads();  // `red` is free for the next row
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
    const int nch = ceil_div(chunks, wide ? 256 : 32);
    const int64_t cap = int64_t(sm_count()) * 8, want = wide ? n : ceil_div<int64_t>(n, 8);
    const dim3 grid(unsigned(want < cap ? want : cap));
    timer_begin(K_RMSNORM, s);
    auto go = [&](auto kernel) {
        launch(kernel, grid, 256, 0, s, 1, static_cast<const uint4*>(x), x_stride, static_cast<const uint4*>(residual),
               static_cast<uint4*>(residual_out), static_cast<const uint4*>(weight), n, dim, eps,
               reinterpret_cast<uint2*>(codes), scales, static_cast<uint4*>(y_bf16));
    };
#define CSA2_NORM(W, C) \
    if (group) go(rmsnorm_fp8_kernel<W, C, true>); \
    else go(rmsnorm_fp8_kernel<W, C, false>)
    if (!wide) {
        if (nch <= 2) { CSA2_NORM(1, 2); }
        else { CSA2_NORM(1, 4); }
    } else {
        if (nch <= 2) { CSA2_NORM(8, 2); }
        else if (nch <= 4) { CSA2_NORM(8, 4); }
        else { CSA2_NORM(8, 8); }
    }
#undef CSA2_NORM
    timer_end(K_RMSNORM, s);
    return launch_status();
}
