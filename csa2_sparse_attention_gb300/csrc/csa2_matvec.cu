// Products of a few rows with FP4 weights (E2M1 codes, one E4M3 scale per 16
// channels): out[i][j] = alpha * sum_c x[i][c] W[j][c].
//
// One warp per output channel and 8 rows of x; lanes take groups of 16 weights.
#include "csa2_common.cuh"
#include "csa2_timer.cuh"

#include <cfloat>

namespace csa2 {

constexpr int kMvRows = 8;

template <bool FP8>
__global__ void __launch_bounds__(256) fp4_matvec_kernel(const uint8_t* __restrict__ x, const float* __restrict__ x_scales,
                                                         int64_t x_stride, int64_t n, int k, const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int64_t n_out, float alpha,
                                                         void* __restrict__ out, bool out_f32) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = lane_id();
    const int64_t i0 = int64_t(blockIdx.y) * kMvRows;
    const int rows = int(n - i0 < kMvRows ? n - i0 : kMvRows);
    for (int64_t j = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); j < n_out; j += int64_t(gridDim.x) * 8) {
        float acc[kMvRows] = {};
        for (int g = lane; g < k / 16; g += 32) {
            const uint2 cw = __ldg(reinterpret_cast<const uint2*>(codes + j * (k / 2)) + g);
            const float s = e4m3_value(scales[j * (k / 16) + g]);
            float w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t c = ((e < 8 ? cw.x : cw.y) >> (4 * (e & 7))) & 15u;
                const uint32_t m = c & 7u;
                const float v = m < 2 ? 0.5f * float(m) : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
                w[e] = (c & 8u ? -v : v) * s;
            }
            for (int i = 0; i < rows; ++i) {
                const int64_t at = (i0 + i) * x_stride + 16 * g;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float xv = FP8 ? e4m3_value(x[at + e])
                                         : __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(x)[at + e]) << 16);
                    acc[i] = fmaf(xv, w[e], acc[i]);
                }
            }
        }
        for (int i = 0; i < rows; ++i) {
            float v = acc[i];
#pragma unroll
            for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            v *= FP8 ? alpha * x_scales[i0 + i] : alpha;
            if (lane == 0) {
                if (out_f32)
                    static_cast<float*>(out)[(i0 + i) * n_out + j] = v;
                else
                    static_cast<__nv_bfloat16*>(out)[(i0 + i) * n_out + j] = __float2bfloat16_rn(v);
            }
        }
    }
}

static bool matvec_sizes(int64_t n, int k, int64_t n_out) {
    return n >= 0 && n <= (int64_t(1) << 20) && k >= 128 && k <= 65536 && k % 128 == 0 && n_out >= 1 && n_out <= INT32_MAX;
}

}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_fp4_matvec_workspace_bytes(int64_t n, int k, int64_t n_out) {
    return matvec_sizes(n, k, n_out) ? CSA2_STATUS_BYTES : 0;
}

extern "C" csa2_status csa2_fp4_matvec(const void* x, int x_fmt, const float* x_scales, int64_t x_stride, int64_t n, int k,
                                       const uint8_t* codes, const uint8_t* scales, int64_t n_out, float alpha, void* out,
                                       int out_dtype, void* ws, size_t ws_bytes, csa2_stream_t stream) {
    if (x_fmt != CSA2_X_BF16 && x_fmt != CSA2_X_E4M3) return CSA2_ERR_UNSUPPORTED;
    if (out_dtype != CSA2_OUT_BF16 && out_dtype != CSA2_OUT_F32) return CSA2_ERR_INVALID_ARG;
    if (n < 0 || n_out < 0 || !(fabsf(alpha) <= FLT_MAX)) return CSA2_ERR_INVALID_ARG;
    if (!matvec_sizes(n, k, n_out)) return CSA2_ERR_UNSUPPORTED;
    if (x_stride < k || x_stride % 16) return CSA2_ERR_INVALID_ARG;
    if ((x_fmt == CSA2_X_E4M3) != (x_scales != nullptr)) return CSA2_ERR_INVALID_ARG;
    if (!x || !codes || !scales || !out) return CSA2_ERR_INVALID_ARG;
    for (const void* p : {x, static_cast<const void*>(codes), static_cast<const void*>(scales),
                          static_cast<const void*>(out), static_cast<const void*>(x_scales)})
        if (!aligned16(p)) return CSA2_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws) || ws_bytes < csa2_fp4_matvec_workspace_bytes(n, k, n_out)) return CSA2_ERR_WORKSPACE;
    if (n == 0) return CSA2_OK;
    cudaStream_t s = cudaStream_t(stream);
    const int64_t want = ceil_div<int64_t>(n_out, 8), cap = int64_t(sm_count()) * 8;
    const dim3 grid(unsigned(want < cap ? want : cap), unsigned(ceil_div<int64_t>(n, kMvRows)));
    timer_begin(K_MATVEC, s);
    launch(x_fmt == CSA2_X_E4M3 ? fp4_matvec_kernel<true> : fp4_matvec_kernel<false>, grid, 256, 0, s, 1,
           static_cast<const uint8_t*>(x), x_scales, x_stride, n, k, codes, scales, n_out, alpha, out,
           out_dtype == CSA2_OUT_F32);
    timer_end(K_MATVEC, s);
    return launch_status();
}
