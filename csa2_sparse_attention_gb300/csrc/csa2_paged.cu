// Causal attention of each request's new tokens over its paged latents.
//
//   l_p = sm_scale q . c_p,  o = sum_p softmax(l)_p c_p,  c_p a 512-wide
//   latent in FP4 (E2M1, one E4M3 scale per 16 channels) or E4M3
//
// One warp per (token, head): each lane holds 16 channels, the logits are warp
// sums, and one pass over the keys keeps a running maximum and sum.
#include "csa2_common.cuh"
#include "csa2_timer.cuh"

#include <cfloat>

namespace csa2 {

constexpr int kPD = CSA2_LATENT_DIM;

template <bool FP8>
__global__ void __launch_bounds__(256) paged_attn_kernel(
    const uint8_t* __restrict__ q, int64_t n_tokens, int heads, const int32_t* __restrict__ q_start,
    const int32_t* __restrict__ kv_len, int64_t n_req, int32_t max_q, int32_t max_kv, const uint8_t* __restrict__ codes,
    const uint8_t* __restrict__ scales, int64_t n_rows, const int32_t* __restrict__ table, int64_t max_pages, int page,
    int window, float sm_scale, uint8_t* __restrict__ out, float* __restrict__ out_lse, Status* st) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = lane_id();
    const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t tok = row / heads;
    if (tok >= n_tokens) return;
    int64_t lo = 0, hi = n_req;  // the request: the last one that starts at or before the token
    while (hi - lo > 1) {
        const int64_t m = (lo + hi) / 2;
        if (q_start[m] <= tok) lo = m;
        else hi = m;
    }
    const int64_t r = lo;
    if (n_req == 0 || tok < q_start[r] || tok >= q_start[r + 1]) return;
    const int32_t nq = q_start[r + 1] - q_start[r];
    if (q_start[r] < 0 || q_start[r + 1] > n_tokens || nq > max_q) {
        if (lane == 0) record(st, CSA2_ERR_DEVICE_BOUNDS, CHK_LENGTH, int32_t(r), nq);
        return;
    }
    int32_t len = kv_len[r];
    if (len < 0 || len > max_kv || len > max_pages * page) {
        if (lane == 0) record(st, CSA2_ERR_DEVICE_BOUNDS, CHK_LENGTH, int32_t(r), len);
        len = 0;
    }
    const int64_t t = int64_t(len) - nq + (tok - q_start[r]);
    float qv[16], o[16] = {};
    {
        const uint4* src = reinterpret_cast<const uint4*>(q + (row * kPD + 16 * lane) * 2);
        const uint4 a = src[0], b = src[1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) qv[2 * e] = bf16_lo(w[e]), qv[2 * e + 1] = bf16_hi(w[e]);
    }
    float m = -INFINITY, l = 0.f;
    const int64_t first = window && t + 1 > window ? t + 1 - window : 0;
    for (int64_t p = first; len > 0 && p <= t; ++p) {
        const int32_t id = table[r * max_pages + p / page];
        const int64_t at = int64_t(id) * page + p % page;
        if (id < 0 || at >= n_rows / page * page) {
            if (lane == 0) record(st, CSA2_ERR_DEVICE_BOUNDS, CHK_PAGE, int32_t(r), id);
            continue;
        }
        float c[16];
        if (FP8) {
            const uint4 v = *reinterpret_cast<const uint4*>(codes + at * kPD + 16 * lane);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 16; ++e) c[e] = e4m3_value((w[e / 4] >> (8 * (e & 3))) & 255u);
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(codes + at * (kPD / 2) + 8 * lane);
            const float s = e4m3_value(scales[at * (kPD / 16) + lane]);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t cc = ((e < 8 ? v.x : v.y) >> (4 * (e & 7))) & 15u, mm = cc & 7u;
                const float f = mm < 2 ? 0.5f * float(mm) : __uint_as_float(((mm >> 1) + 126u) << 23 | (mm & 1u) << 22);
                c[e] = (cc & 8u ? -f : f) * s;
            }
        }
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) x = fmaf(qv[e], c[e], x);
#pragma unroll
        for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
        x *= sm_scale;
        const float mn = fmaxf(m, x);
        const float f = m == -INFINITY ? 0.f : expf(m - mn), e1 = expf(x - mn);
        m = mn;
        l = l * f + e1;
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = fmaf(e1, c[e], o[e] * f);
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
        w[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    uint4* dst = reinterpret_cast<uint4*>(out + (row * kPD + 16 * lane) * 2);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (out_lse && lane == 0) out_lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

static bool paged_sizes(int64_t n_tokens, int n_heads, int64_t n_req, int32_t max_q, int32_t max_kv, int window) {
    return n_tokens >= 0 && n_tokens <= (int64_t(1) << 24) && n_heads >= 1 && n_heads <= 128 && n_req >= 0 &&
           n_req <= (1 << 20) && max_q >= 0 && max_kv >= 0 && window >= 0;
}

}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_paged_attn_workspace_bytes(int64_t n_tokens, int n_heads, int64_t n_req, int32_t max_q,
                                                  int32_t max_kv, int window) {
    return paged_sizes(n_tokens, n_heads, n_req, max_q, max_kv, window) ? CSA2_STATUS_BYTES : 0;
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
    timer_begin(K_PAGED_ATTN, s);
    launch(fmt == CSA2_FMT_FP8 ? paged_attn_kernel<true> : paged_attn_kernel<false>,
           dim3(unsigned(ceil_div<int64_t>(n_tokens * n_heads, 8))), 256, 0, s, 1, static_cast<const uint8_t*>(q_bf16),
           n_tokens, n_heads, q_start, kv_len, n_req, max_q, max_kv, codes, scales, n_rows, table, max_pages, page_size,
           window, sm_scale, static_cast<uint8_t*>(out), out_lse, static_cast<Status*>(ws));
    timer_end(K_PAGED_ATTN, s);
    return launch_status();
}
