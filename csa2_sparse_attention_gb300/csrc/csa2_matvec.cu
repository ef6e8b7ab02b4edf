// Products of a few rows with FP4 weights (E2M1 codes, one E4M3 scale per 16
// channels): out[i][j] = alpha * sum_c x[i][c] W[j][c].
//
// 0.5625 bytes per weight and 2 FLOPs per weight and row: HBM bounds it for
// any number of rows a call takes at once (16), as long as the weights are
// decoded cheaply.  mma.sync m16n8k16 takes 16 output channels x 16 channels
// of W as the A operand (code times scale has at most 6 significant bits:
// exact in f16) and up to 8 rows of x as B, with fp32 accumulators; a warp-wide
// dot product would spend an FMA per weight and row, the MMA two conversions
// and a multiply per two weights for all rows together.
//
// x goes to f16 in shared memory once per CTA, each row times a power of two
// (exact down to 2^-28 of the row's maximum), in the order in which a lane
// needs it.  The sum over channels is in any order as long as A and B agree:
// lane t of a quad takes 64 consecutive channels of a 256-channel step (32
// bytes of codes in one load, 128 contiguous bytes per weight row) and feeds
// them four at a time to the 16 MMAs of the step, so the loads are whole lines
// and the decoded codes need no exchange.  A CTA keeps its x and walks over the
// output channels; its warps split the channels of x (and rows of W) and add up
// in shared memory in a fixed order.  Three steps of loads (7 KB a warp) are
// in flight.
#include "csa2_common.cuh"
#include "csa2_timer.cuh"
#include "csa2_layout.cuh"

#include <atomic>
#include <cfloat>

namespace csa2 {

constexpr int kMvThreads = 256, kMvWarps = kMvThreads / 32;
constexpr int kMvStep = 256;                  // channels per step
constexpr int kMvDepth = 3;                   // steps in flight
constexpr size_t kMvXBytes = 200 * 1024;      // x in shared memory, per CTA

struct MatvecArgs {
    const uint8_t* x;
    const float* x_scales;
    const uint8_t* codes;
    const uint8_t* scales;
    void* out;
    float* part;         // [slices][n][n_out] partial sums, or null
    int64_t n, x_stride, n_out, tiles;
    int32_t k, slice;    // channels; channels per slice (a multiple of 256)
    int32_t wk;          // warps over the channels; the others go over rows of W
    float alpha;
    int32_t out_f32;
};

struct Mv256 {
    uint32_t w[8];
};
// 32 bytes that no one reads again soon
__device__ __forceinline__ Mv256 ldg256(const uint8_t* p) {
    Mv256 v;
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                   "=r"(v.w[7])
                 : "l"(p));
    return v;
}
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mv_codes(uint32_t w, uint32_t s, uint32_t (&o)[4]) {  // 8 codes times their scale
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n"
        " mul.rn.f16x2 %0, %0, %5;\n mul.rn.f16x2 %1, %1, %5;\n mul.rn.f16x2 %2, %2, %5;\n mul.rn.f16x2 %3, %3, %5;\n}\n"
        : "=&r"(o[0]), "=&r"(o[1]), "=&r"(o[2]), "=&r"(o[3]) : "r"(w), "r"(s));
}
__device__ __forceinline__ void mv_scales(uint32_t w, uint32_t (&o)[4]) {  // four E4M3 scales, each as f16x2
    uint32_t a, b;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n"
        " cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;\n}\n" : "=r"(a), "=r"(b) : "r"(w));
    o[0] = __byte_perm(a, 0, 0x1010);
    o[1] = __byte_perm(a, 0, 0x3232);
    o[2] = __byte_perm(b, 0, 0x1010);
    o[3] = __byte_perm(b, 0, 0x3232);
}

// grid (CTAs over W's rows, slices of x's channels, groups of 16 rows of x)
template <bool FP8, int NT>
__global__ void __launch_bounds__(kMvThreads, 2) fp4_matvec_kernel(const MatvecArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ uint32_t s_max[16];
    __shared__ float s_mul[16];
    __shared__ float s_red[2][kMvWarps][16 * NT * 8];
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
    const int64_t i0 = int64_t(blockIdx.z) * 16;
    const int rows = int(a.n - i0 < 16 ? a.n - i0 : 16);  // rows of x (NT = 1: up to 8)
    const int32_t k0 = blockIdx.y * a.slice, kn = a.k - k0 < a.slice ? a.k - k0 : a.slice;
    const int steps = (kn + kMvStep - 1) / kMvStep;
    const int wk = a.wk, wm = kMvWarps / wk, my_k = warp % wk, my_m = warp / wk;
    const int per_tile = (steps + wk - 1) / wk;  // steps of a warp per tile of 16 wm rows of W
    if (tid < 16) s_max[tid] = 0;
    grid_dep_wait();
    grid_dep_launch();

    // ---- weights: step u of this warp is step my_k + wk (u % per_tile) of
    // the channels, of tile blockIdx.x + gridDim.x (u / per_tile)
    const int g = lane >> 2, t = lane & 3;
    const int64_t my_tiles = (a.tiles - blockIdx.x + gridDim.x - 1) / gridDim.x;
    const int64_t units = my_tiles * per_tile;
    Mv256 cw[kMvDepth][2];
    uint32_t sw[kMvDepth][2];
    int64_t f_tile = blockIdx.x;  // the unit to be loaded next
    int f_k = 0;
    auto fetch = [&](int d) {
        const int32_t c = (my_k + wk * f_k) * kMvStep + 64 * t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = (f_tile * wm + my_m) * 16 + g + 8 * h;
            if (f_tile < a.tiles && row < a.n_out && c < kn) {
                cw[d][h] = ldg256(a.codes + (row * a.k + k0 + c) / 2);
                sw[d][h] = __ldg(reinterpret_cast<const uint32_t*>(a.scales + (row * a.k + k0 + c) / 16));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) cw[d][h].w[e] = 0;
                sw[d][h] = 0;
            }
        }
        if (++f_k == per_tile) f_k = 0, f_tile += gridDim.x;
    };
#pragma unroll
    for (int d = 0; d < kMvDepth; ++d) fetch(d);

    // ---- x: f16 in the lanes' order, [step][8-channel piece i][row][t]
    const int pieces = steps * (kMvStep / 8);  // per row, of 8 channels
    auto x_piece = [&](int r, int p) {
        const int64_t at = (i0 + r) * a.x_stride + k0 + 8 * p;
        if (FP8) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(a.x + at));
            uint4 o;
            asm("{\n .reg .b16 a, b, c, d;\n mov.b32 {a, b}, %4;\n mov.b32 {c, d}, %5;\n"
                " cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n"
                " cvt.rn.f16x2.e4m3x2 %2, c;\n cvt.rn.f16x2.e4m3x2 %3, d;\n}\n"
                : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w) : "r"(v.x), "r"(v.y));
            return o;
        }
        return __ldg(reinterpret_cast<const uint4*>(a.x + 2 * at));
    };
    const int threads_per_row = kMvThreads / (rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : rows <= 8 ? 8 : 16);
    const int xr = tid / threads_per_row, xt = tid % threads_per_row;
    __syncthreads();  // s_max is zero
    if (!FP8 && xr < rows) {
        uint32_t m = 0;
        for (int p = xt; 8 * p < kn; p += threads_per_row) {
            const uint4 v = x_piece(xr, p);
            m = __vmaxu2(m, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu));
            m = __vmaxu2(m, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
        }
        m = max(m & 0xFFFFu, m >> 16);
        atomicMax(&s_max[xr], m);
    }
    __syncthreads();
    if (xr < rows) {
        float qf = 1.f;
        if (!FP8) {
            int qs = s_max[xr] != 0 ? int(s_max[xr] >> 7) - 127 - 14 : 0;  // max |x| 2^-qs in [2^14, 2^15)
            qs = qs < -126 ? -126 : (qs > 126 ? 126 : qs);
            qf = __uint_as_float(uint32_t(127 - qs) << 23);
            if (xt == 0) s_mul[xr] = __uint_as_float(uint32_t(127 + qs) << 23);
        } else if (xt == 0) {
            s_mul[xr] = a.x_scales[i0 + xr];
        }
        for (int p = xt; p < pieces; p += threads_per_row) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (8 * p < kn) {
                v = x_piece(xr, p);
                if (!FP8) {
                    uint32_t* w = &v.x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __half2 h = __floats2half2_rn(bf16_lo(w[e]) * qf, bf16_hi(w[e]) * qf);
                        w[e] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                }
            }
            const int c = p >> 5, pt = (p >> 3) & 3, i = p & 7;
            *reinterpret_cast<uint4*>(smem_raw + (size_t((c * 8 + i) * rows + xr) * 4 + pt) * 16) = v;
        }
    }
    __syncthreads();

    // ---- the walk
    uint32_t xoff[NT];  // this lane's row of x (a missing row reads another; its sums are dropped)
#pragma unroll
    for (int q = 0; q < NT; ++q) xoff[q] = uint32_t((8 * q + g < rows ? 8 * q + g : 0) * 4 + t) * 16;
    const uint32_t xstride = uint32_t(rows) * 64;
    float acc[NT][4] = {};
    int64_t tile = blockIdx.x;
    int kk = 0, par = 0;
    for (int64_t u0 = 0; u0 < units; u0 += kMvDepth) {
#pragma unroll
        for (int d = 0; d < kMvDepth; ++d) {
            if (u0 + d >= units) break;
            const int step = my_k + wk * kk;
            if (step < steps) {
                const uint8_t* xs = smem_raw + size_t(step) * 8 * xstride;
                uint32_t s0[4], s1[4];
                mv_scales(sw[d][0], s0);
                mv_scales(sw[d][1], s1);
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    uint32_t r0[4], r1[4];
                    mv_codes(cw[d][0].w[w], s0[w >> 1], r0);
                    mv_codes(cw[d][1].w[w], s1[w >> 1], r1);
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        const uint4 b = *reinterpret_cast<const uint4*>(xs + w * xstride + xoff[q]);
                        mma_16816(acc[q], r0[0], r1[0], r0[1], r1[1], b.x, b.y);
                        mma_16816(acc[q], r0[2], r1[2], r0[3], r1[3], b.z, b.w);
                    }
                }
            }
            fetch(d);
            if (++kk == per_tile) {  // the tile is done: add up the warps' parts and write
                kk = 0;
                float* mine = s_red[par][warp];
#pragma unroll
                for (int q = 0; q < NT; ++q) {
                    const int col = 8 * q + 2 * t;
                    mine[col * 16 + g] = acc[q][0];
                    mine[(col + 1) * 16 + g] = acc[q][1];
                    mine[col * 16 + g + 8] = acc[q][2];
                    mine[(col + 1) * 16 + g + 8] = acc[q][3];
                    acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
                }
                __syncthreads();
                const int width = 16 * wm;
                for (int e = tid; e < rows * width; e += kMvThreads) {
                    const int i = e / width, j = e - i * width, m = j >> 4;
                    float v = 0.f;
                    for (int q = 0; q < wk; ++q) v += s_red[par][m * wk + q][i * 16 + (j & 15)];
                    v *= s_mul[i];
                    const int64_t row = tile * width + j;
                    if (row < a.n_out) {
                        if (a.part)
                            a.part[(int64_t(blockIdx.y) * a.n + i0 + i) * a.n_out + row] = v;
                        else if (a.out_f32)
                            static_cast<float*>(a.out)[(i0 + i) * a.n_out + row] = a.alpha * v;
                        else
                            static_cast<__nv_bfloat16*>(a.out)[(i0 + i) * a.n_out + row] = __float2bfloat16_rn(a.alpha * v);
                    }
                }
                par ^= 1;  // the next tile's parts go to the other buffer: one barrier per tile
                tile += gridDim.x;
            }
        }
    }
}

// Adds the slices' partial sums in order.
__global__ void __launch_bounds__(256) matvec_join_kernel(const float* __restrict__ part, int slices, int64_t count, float alpha,
                                                          void* __restrict__ out, int out_f32) {
    grid_dep_wait();
    grid_dep_launch();
    for (int64_t e = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; e < count; e += int64_t(gridDim.x) * blockDim.x) {
        float v = 0.f;
        for (int s = 0; s < slices; ++s) v += part[s * count + e];
        if (out_f32)
            static_cast<float*>(out)[e] = alpha * v;
        else
            static_cast<__nv_bfloat16*>(out)[e] = __float2bfloat16_rn(alpha * v);
    }
}

struct MatvecPlan {
    int32_t slice, slices, wk;
    size_t x_bytes, total;
};
static MatvecPlan matvec_plan(int64_t n, int k, int64_t n_out) {
    MatvecPlan p{};
    const int rows = n < 16 ? int(n > 0 ? n : 1) : 16;
    const int steps = (k + kMvStep - 1) / kMvStep;
    const size_t step_bytes = size_t(rows) * kMvStep * 2;
    const int fit = int(kMvXBytes / step_bytes);  // steps of x that a CTA can hold (25 at 16 rows)
    p.slices = (steps + fit - 1) / fit;
    const int per = (steps + p.slices - 1) / p.slices;
    p.slices = (steps + per - 1) / per;
    p.slice = per * kMvStep;
    p.x_bytes = per * step_bytes;
    // at least two steps of a warp per tile, so that the join over the warps stays a small part
    p.wk = per >= 16 ? 8 : per >= 8 ? 4 : per >= 4 ? 2 : 1;
    p.total = CSA2_STATUS_BYTES;
    if (p.slices > 1) p.total = align256(p.total + size_t(p.slices) * size_t(n) * size_t(n_out) * 4);
    return p;
}

template <bool FP8, int NT>
static csa2_status matvec_launch(const MatvecArgs& a, const MatvecPlan& p, cudaStream_t s) {
    static std::atomic<bool> done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CSA2_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(fp4_matvec_kernel<FP8, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMvXBytes)) !=
            cudaSuccess) {
            cudaGetLastError();
            return CSA2_ERR_CUDA;
        }
        done[dev].store(true, std::memory_order_release);
    }
    // two CTAs per SM where both fit into its shared memory
    const int per_sm = p.x_bytes + 20 * 1024 <= 113 * 1024 ? 2 : 1;
    const int64_t groups = ceil_div<int64_t>(a.n, 16);
    int64_t cap = int64_t(sm_count()) * per_sm / (p.slices * groups);
    cap = cap < 1 ? 1 : cap;
    const dim3 grid(unsigned(a.tiles < cap ? a.tiles : cap), unsigned(p.slices), unsigned(groups));
    const cudaError_t e = launch(fp4_matvec_kernel<FP8, NT>, grid, kMvThreads, p.x_bytes, s, 1, a);
    return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

static bool matvec_sizes(int64_t n, int k, int64_t n_out) {
    return n >= 0 && n <= (int64_t(1) << 16) && k >= 128 && k <= 65536 && k % 128 == 0 && n_out >= 1 && n_out <= INT32_MAX;
}

}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_fp4_matvec_workspace_bytes(int64_t n, int k, int64_t n_out) {
    return matvec_sizes(n, k, n_out) ? matvec_plan(n, k, n_out).total : 0;
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
    const MatvecPlan p = matvec_plan(n, k, n_out);
    MatvecArgs a{};
    a.x = static_cast<const uint8_t*>(x);
    a.x_scales = x_scales;
    a.codes = codes;
    a.scales = scales;
    a.out = out;
    a.part = p.slices > 1 ? reinterpret_cast<float*>(static_cast<char*>(ws) + CSA2_STATUS_BYTES) : nullptr;
    a.n = n;
    a.x_stride = x_stride;
    a.n_out = n_out;
    a.tiles = ceil_div<int64_t>(n_out, 16 * (kMvWarps / p.wk));
    a.k = k;
    a.slice = p.slice;
    a.wk = p.wk;
    a.alpha = alpha;
    a.out_f32 = out_dtype == CSA2_OUT_F32;
    timer_begin(K_MATVEC, s);
    const bool two = n > 8;
    const csa2_status e = x_fmt == CSA2_X_E4M3 ? (two ? matvec_launch<true, 2>(a, p, s) : matvec_launch<true, 1>(a, p, s))
                                               : (two ? matvec_launch<false, 2>(a, p, s) : matvec_launch<false, 1>(a, p, s));
    timer_end(K_MATVEC, s);
    if (e != CSA2_OK) {
        cudaGetLastError();
        return e;
    }
    if (p.slices > 1) {
        const int64_t count = n * n_out, blocks = ceil_div<int64_t>(count, 1024), cap = int64_t(sm_count()) * 8;
        launch(matvec_join_kernel, dim3(unsigned(blocks < cap ? blocks : cap)), 256, 0, s, 1, a.part, p.slices, count, alpha, out,
               int(a.out_f32));
    }
    return launch_status();
}
