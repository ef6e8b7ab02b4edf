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
// lane t of a quad takes 32 consecutive channels of 128 (16 bytes of codes, 64
// contiguous bytes per weight row) and feeds them four at a time to 8 MMAs, so
// the decoded codes need no exchange.  A warp takes 32 rows of W, so that one
// read of x from shared memory serves two MMAs.
//
// Weights come by 16-byte asynchronous copies through a ring of a warp's own
// (2.25 KB a step, up to four steps for each of 16 warps): loads into
// registers reached 3.1 TB/s, since a warp's six scoreboards make it wait for
// the youngest load with the oldest.  A CTA keeps its x and walks over the
// output channels; its warps split the channels of x (and rows of W) and add up
// in shared memory in a fixed order.
#include "csa2_common.cuh"
#include "csa2_timer.cuh"
#include "csa2_layout.cuh"

#include <atomic>
#include <cfloat>

namespace csa2 {

constexpr int kMvThreads = 512, kMvWarps = kMvThreads / 32;
constexpr int kMvStep = 128, kMvRows = 32;    // channels and rows of W per step of a warp
constexpr int kMvStage = kMvRows * (kMvStep / 2 + kMvStep / 16);  // bytes of a step: codes, then scales
constexpr int kMvSumStride = 36;              // a column's rows of a warp's sums: no bank conflicts
constexpr int kMvMaxStages = 4;
constexpr int kMvHeld = 8;                    // pieces of x that a thread holds from its first loads on
constexpr int kMvSms = 152;                   // multiprocessors the split is planned for
constexpr size_t kMvSmem = 208 * 1024;        // x and the rings, per CTA (and the warps' sums, 18 or 36 KB)

struct MatvecArgs {
    const uint8_t* x;
    const float* x_scales;
    const uint8_t* codes;
    const uint8_t* scales;
    void* out;
    float* part;         // [slices][n][n_out] partial sums, or null
    int64_t n, x_stride, n_out, tiles;
    int32_t k, slice;    // channels; channels per slice (a multiple of 128)
    int32_t wk, wm;      // warps over the channels, warps over rows of W (what is left of 16 idles)
    int32_t by_wm;       // 65536 / wm + 1: n * by_wm >> 16 is n / wm for n < 256
    int32_t x_e4m3;
    float alpha;
    int32_t out_f32;
};

// 16 bytes into shared memory past L1 (weights, read once), or 8 through it
// (scales: the rest of the sector is other steps'); zeros where !on.
__device__ __forceinline__ void cp16_cg(void* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp8_ca(void* dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(on ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
__device__ __forceinline__ void mv_scales(uint32_t w, uint32_t& s0, uint32_t& s1) {  // two E4M3 scales, each as f16x2
    uint32_t a;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"(uint16_t(w)));
    s0 = __byte_perm(a, 0, 0x1010);
    s1 = __byte_perm(a, 0, 0x3232);
}

// grid (CTAs over W's rows, slices of x's channels, groups of 16 rows of x)
template <int NT, int STAGES>
__global__ void __launch_bounds__(kMvThreads, 1) fp4_matvec_kernel(const MatvecArgs a) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ uint32_t s_max[16];
    __shared__ float s_mul[16];
    const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
    const int64_t i0 = int64_t(blockIdx.z) * 16;
    const int rows = int(a.n - i0 < 16 ? a.n - i0 : 16);  // rows of x (NT = 1: up to 8)
    const int32_t k0 = blockIdx.y * a.slice, kn = a.k - k0 < a.slice ? a.k - k0 : a.slice;
    const int steps = (kn + kMvStep - 1) / kMvStep;
    const int wk = a.wk, wm = a.wm, my_k = warp % wk, my_m = warp / wk;
    const int my_steps = my_m < wm ? steps : 0;    // (an idle warp has none)
    const int per_tile = (steps + wk - 1) / wk;  // steps of a warp per tile of 32 wm rows of W
    // shared memory: rings, then the warps' sums [warp][8 NT columns][36: 32 rows], then x
    uint8_t* ring = smem_raw + warp * (STAGES * kMvStage);
    float* s_red = reinterpret_cast<float*>(smem_raw + kMvWarps * STAGES * kMvStage);
    constexpr int kRed = 8 * NT * kMvSumStride;
    uint8_t* s_x = reinterpret_cast<uint8_t*>(s_red + kMvWarps * kRed);
    if (tid < 16) s_max[tid] = 0;
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();

    // ---- x: the first pieces of 8 channels of this thread's row, ahead of the
    // weights in the load unit's queue
    const int threads_per_row = kMvThreads / (rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : rows <= 8 ? 8 : 16);
    const int xr = tid / threads_per_row, xt = tid % threads_per_row;
    const bool x_on = xr < rows;
    auto x_raw = [&](int p) {  // 8 bf16, or 8 E4M3 in the first half
        const int64_t at = (i0 + xr) * a.x_stride + k0 + 8 * p;
        if (!a.x_e4m3) return __ldg(reinterpret_cast<const uint4*>(a.x + 2 * at));
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(a.x + at));
        return make_uint4(v.x, v.y, 0, 0);
    };
    uint4 xv[kMvHeld];
#pragma unroll
    for (int e = 0; e < kMvHeld; ++e) {
        const int p = xt + e * threads_per_row;
        xv[e] = x_on && p < kn / 8 ? x_raw(p) : make_uint4(0, 0, 0, 0);
    }

    // ---- weights: step u of this warp is step my_k + wk (u % per_tile) of
    // the channels, of tile blockIdx.x + gridDim.x (u / per_tile)
    const int g = lane >> 2, t = lane & 3;
    const int64_t my_tiles = (a.tiles - blockIdx.x + gridDim.x - 1) / gridDim.x;
    const int64_t units = my_tiles * per_tile;
    const int64_t row8 = int64_t(a.k) * 4;  // bytes of 8 rows' codes
    int64_t f_tile = blockIdx.x;            // the unit to be loaded next
    int f_k = 0, f_stage = 0;
    const uint8_t *f_code = nullptr, *f_scale = nullptr;
    int f_left = 0;                         // rows of W from this lane's first one on
    bool f_scale_on = false;
    auto f_rows = [&]() {
        const int64_t r = (f_tile * wm + my_m) * kMvRows;
        f_left = f_tile < a.tiles ? int(a.n_out - r - g < kMvRows ? a.n_out - r - g : kMvRows) : 0;
        f_code = a.codes + ((r + g) * a.k + k0) / 2 + 16 * t;
        f_scale = a.scales + ((r + lane) * a.k + k0) / 16;
        f_scale_on = f_tile < a.tiles && r + lane < a.n_out;
    };
    f_rows();
    auto fetch = [&]() {
        const int step = my_k + wk * f_k;
        uint8_t* dst = ring + f_stage * kMvStage + lane * 16;
        const uint8_t* src = f_code + step * (kMvStep / 2);
        const bool in = step < my_steps;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const bool on = in && 8 * h < f_left;
            cp16_cg(dst + h * 512, on ? src + h * row8 : a.codes, on);
        }
        const bool son = in && f_scale_on;  // a row's 8 scales per lane
        cp8_ca(ring + f_stage * kMvStage + 4 * 512 + lane * 8, son ? f_scale + step * (kMvStep / 16) : a.scales, son);
        f_stage = f_stage + 1 == STAGES ? 0 : f_stage + 1;
        if (++f_k == per_tile) {
            f_k = 0;
            f_tile += gridDim.x;
            f_rows();
        }
    };
#pragma unroll
    for (int d = 0; d < STAGES - 1; ++d) {
        fetch();
        cp_commit();
    }

    // ---- x: f16 in the lanes' order, [128 channels][8-channel piece i][row][t]
    if (!a.x_e4m3) {
        if (x_on) {
            uint32_t m = 0;
            auto take = [&](uint4 v) {
                m = __vmaxu2(m, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu));
                m = __vmaxu2(m, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
            };
#pragma unroll
            for (int e = 0; e < kMvHeld; ++e) take(xv[e]);
#pragma unroll 4
            for (int p = xt + kMvHeld * threads_per_row; p < kn / 8; p += threads_per_row) take(x_raw(p));
            m = max(m & 0xFFFFu, m >> 16);
            atomicMax(&s_max[xr], m);
        }
        __syncthreads();
    }
    if (x_on) {
        float qf = 1.f;
        if (!a.x_e4m3) {
            int qs = s_max[xr] != 0 ? int(s_max[xr] >> 7) - 127 - 14 : 0;  // max |x| 2^-qs in [2^14, 2^15)
            qs = qs < -126 ? -126 : (qs > 126 ? 126 : qs);
            qf = __uint_as_float(uint32_t(127 - qs) << 23);
            if (xt == 0) s_mul[xr] = __uint_as_float(uint32_t(127 + qs) << 23);
        } else if (xt == 0) {
            s_mul[xr] = a.x_scales[i0 + xr];
        }
        auto put = [&](int p, uint4 v) {
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (a.x_e4m3) {
                asm("{\n .reg .b16 a, b, c, d;\n mov.b32 {a, b}, %4;\n mov.b32 {c, d}, %5;\n"
                    " cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n"
                    " cvt.rn.f16x2.e4m3x2 %2, c;\n cvt.rn.f16x2.e4m3x2 %3, d;\n}\n"
                    : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(v.x), "r"(v.y));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __half2 h = __floats2half2_rn(bf16_lo(w[e]) * qf, bf16_hi(w[e]) * qf);
                    w[e] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
            const int c = p >> 4, pt = (p >> 2) & 3, i = p & 3;
            *reinterpret_cast<uint4*>(s_x + ((c * 4 + i) * rows + xr) * 64 + pt * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        };
#pragma unroll
        for (int e = 0; e < kMvHeld; ++e)
            if (xt + e * threads_per_row < kn / 8) put(xt + e * threads_per_row, xv[e]);
#pragma unroll 4
        for (int p = xt + kMvHeld * threads_per_row; p < kn / 8; p += threads_per_row) put(p, x_raw(p));
    }
    if (tid < rows * 16) reinterpret_cast<uint4*>(s_x + steps * rows * 256)[tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();

    // ---- the walk
    uint32_t xoff[NT];  // this lane's row of x (a missing row reads another; its sums are dropped)
#pragma unroll
    for (int q = 0; q < NT; ++q) xoff[q] = uint32_t((8 * q + g < rows ? 8 * q + g : 0) * 4 + t) * 16;
    const uint32_t xstride = uint32_t(rows) * 64;
    float acc[2][NT][4] = {};
    int64_t tile = blockIdx.x;
    int kk = 0, stage = 0;
    for (int64_t u = 0; u < units; ++u) {
        cp_wait<STAGES - 2>();
        __syncwarp();  // the step's copies of every lane are in; every lane is done with the stage refilled here
        fetch();
        cp_commit();
        const int step = my_k + wk * kk;
        const uint8_t* cs = ring + stage * kMvStage;
        stage = stage + 1 == STAGES ? 0 : stage + 1;
        // (without a branch the loads run ahead of the products: a step behind the last one has zero weights, and reads
        // the zeros behind x; 4 x 8192 -> 28672 28.2 -> 27.2 us)
        uint4 cw[4];
        uint32_t sc[4][2];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            cw[h] = *reinterpret_cast<const uint4*>(cs + h * 512 + lane * 16);
            mv_scales(*reinterpret_cast<const uint16_t*>(cs + 4 * 512 + (8 * h + g) * 8 + 2 * t), sc[h][0], sc[h][1]);
        }
        const uint8_t* xs = s_x + (step < steps ? step : steps) * 4 * xstride;
#pragma unroll
        for (int w = 0; w < 4; ++w) {  // 8 of the lane's 32 channels
            uint4 b[NT];
#pragma unroll
            for (int q = 0; q < NT; ++q) b[q] = *reinterpret_cast<const uint4*>(xs + w * xstride + xoff[q]);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint32_t r0[4], r1[4];
                const uint4 c0 = cw[2 * m], c1 = cw[2 * m + 1];
                mv_codes(w == 0 ? c0.x : w == 1 ? c0.y : w == 2 ? c0.z : c0.w, sc[2 * m][w >> 1], r0);
                mv_codes(w == 0 ? c1.x : w == 1 ? c1.y : w == 2 ? c1.z : c1.w, sc[2 * m + 1][w >> 1], r1);
#pragma unroll
                for (int q = 0; q < NT; ++q) {
                    mma_16816(acc[m][q], r0[0], r1[0], r0[1], r1[1], b[q].x, b[q].y);
                    mma_16816(acc[m][q], r0[2], r1[2], r0[3], r1[3], b[q].z, b[q].w);
                }
            }
        }
        if (++kk == per_tile) {  // the tile is done: add up the warps' parts and write
            kk = 0;
            float* mine = s_red + warp * kRed;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int q = 0; q < NT; ++q) {
                    const int col = 8 * q + 2 * t, r = 16 * m + g;
                    mine[col * kMvSumStride + r] = acc[m][q][0];
                    mine[(col + 1) * kMvSumStride + r] = acc[m][q][1];
                    mine[col * kMvSumStride + r + 8] = acc[m][q][2];
                    mine[(col + 1) * kMvSumStride + r + 8] = acc[m][q][3];
                    acc[m][q][0] = acc[m][q][1] = acc[m][q][2] = acc[m][q][3] = 0.f;
                }
            __syncthreads();
            const int width = kMvRows * wm;
            for (int e = tid; e < rows * width; e += kMvThreads) {
                const int i = ((e >> 5) * a.by_wm) >> 16, j = e - i * width;
                const float* from = s_red + (j >> 5) * wk * kRed + i * kMvSumStride + (j & 31);
                float v = 0.f;
                for (int q = 0; q < wk; ++q) v += from[q * kRed];
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
            __syncthreads();
            tile += gridDim.x;
        }
    }
    cp_wait<0>();
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
    int32_t slice, slices, wk, wm, stages;
    int64_t tiles, grid;
    size_t smem, total;
};
static MatvecPlan matvec_plan(int64_t n, int k, int64_t n_out) {
    MatvecPlan p{};
    const int rows = n < 16 ? int(n > 0 ? n : 1) : 16, nt = n > 8 ? 2 : 1;
    const int steps = (k + kMvStep - 1) / kMvStep;
    const size_t step_x = size_t(rows) * kMvStep * 2, red = size_t(kMvWarps) * 8 * nt * kMvSumStride * 4;
    // x's channels per CTA and a step of zeros: what fits beside two stages (24 steps of 128 at 16 rows)
    const int fit = int((kMvSmem - red - 2 * kMvWarps * kMvStage) / step_x) - 1;
    p.slices = (steps + fit - 1) / fit;
    const int per = (steps + p.slices - 1) / p.slices;
    p.slices = (steps + per - 1) / per;
    p.slice = per * kMvStep;
    p.stages = int((kMvSmem - red - (per + 1) * step_x) / (kMvWarps * kMvStage));
    p.stages = p.stages < kMvMaxStages ? p.stages : kMvMaxStages;
    p.smem = size_t(p.stages) * kMvWarps * kMvStage + red + (per + 1) * step_x;
    // warps over channels and rows: the fewest steps of the busiest CTA, half a
    // step for each join, and less the fewer warps share the issue slots.  (With 16
    // warps always, powers of two each way: 5 x 896 -> 20000 8.0 us, 1 x 4096 ->
    // 12288 11.4 us; so 7.0 and 11.0.)
    const int64_t groups = (n + 15) / 16;
    int64_t ctas = kMvSms / (p.slices * (groups > 0 ? groups : 1));
    ctas = ctas < 1 ? 1 : ctas;
    double best = 1e30;
    for (int wk = 1; wk <= kMvWarps; ++wk) {
        const int64_t blocks = (n_out + kMvRows - 1) / kMvRows, most = ctas * (kMvWarps / wk);
        const int64_t rounds = (blocks + most - 1) / most;
        const int64_t wm = (blocks + ctas * rounds - 1) / (ctas * rounds);  // no more than these rounds need
        const double cost = double(rounds) * ((per + wk - 1) / wk + 0.5) * (0.7 + 0.3 * double(wk * wm) / kMvWarps);
        if (cost < best) {
            best = cost;
            p.wk = wk;
            p.wm = int(wm);
        }
    }
    p.tiles = (n_out + kMvRows * p.wm - 1) / (kMvRows * p.wm);
    p.grid = p.tiles < ctas ? p.tiles : ctas;
    p.total = CSA2_STATUS_BYTES;
    if (p.slices > 1) p.total = align256(p.total + size_t(p.slices) * size_t(n) * size_t(n_out) * 4);
    return p;
}

template <int NT, int STAGES>
static csa2_status matvec_launch(const MatvecArgs& a, const MatvecPlan& p, cudaStream_t s) {
    static std::atomic<bool> done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CSA2_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(fp4_matvec_kernel<NT, STAGES>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMvSmem)) !=
            cudaSuccess)
            return CSA2_ERR_CUDA;
        done[dev].store(true, std::memory_order_release);
    }
    const dim3 grid(unsigned(p.grid), unsigned(p.slices), unsigned(ceil_div<int64_t>(a.n, 16)));
    return launch(fp4_matvec_kernel<NT, STAGES>, grid, kMvThreads, p.smem, s, 1, a) == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
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
    const MatvecPlan p = matvec_plan(n, k, n_out);
    if (!ws || !aligned16(ws) || ws_bytes < p.total) return CSA2_ERR_WORKSPACE;
    if (n == 0) return CSA2_OK;
    const char *x0 = static_cast<const char*>(x), *o0 = static_cast<const char*>(out);
    if (o0 < x0 + (size_t(n - 1) * x_stride + k) * (x_fmt == CSA2_X_BF16 ? 2 : 1) &&
        x0 < o0 + size_t(n) * n_out * (out_dtype == CSA2_OUT_F32 ? 4 : 2))
        return CSA2_ERR_INVALID_ARG;
    cudaStream_t s = cudaStream_t(stream);
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
    a.tiles = p.tiles;
    a.x_e4m3 = x_fmt == CSA2_X_E4M3;
    a.k = k;
    a.slice = p.slice;
    a.wk = p.wk;
    a.wm = p.wm;
    a.by_wm = 65536 / p.wm + 1;
    a.alpha = alpha;
    a.out_f32 = out_dtype == CSA2_OUT_F32;
    timer_begin(K_MATVEC, s);
    const bool two = n > 8;
    const csa2_status e = p.stages >= 4   ? (two ? matvec_launch<2, 4>(a, p, s) : matvec_launch<1, 4>(a, p, s))
                          : p.stages == 3 ? (two ? matvec_launch<2, 3>(a, p, s) : matvec_launch<1, 3>(a, p, s))
                                          : (two ? matvec_launch<2, 2>(a, p, s) : matvec_launch<1, 2>(a, p, s));
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
