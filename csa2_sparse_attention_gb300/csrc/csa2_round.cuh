// Roundings to E4M3 and E2M1 beyond the hardware's conversions of one float:
// exact ones of numbers held in fp64, and of a pair to E2M1 at once.
#pragma once

#include "csa2_common.cuh"

namespace csa2 {

// Nearest-even E4M3 byte of v >= 0 held in fp64, saturating at 448: the
// fp32-rounded guess is off by at most one step; the midpoint test 2v vs
// a + b is exact in fp64.
__device__ __forceinline__ uint32_t e4m3_rne_f64(double v) {
    if (v >= 448.0) return 0x7E;
    const uint32_t g = e4m3x2_rn_sat(float(v), 0.f) & 0x7F;
    uint32_t best = g;
    double bv = double(e4m3_value(g));
#pragma unroll
    for (int d = -1; d <= 1; d += 2) {
        const int c = int(g) + d;
        if (c < 0 || c > 0x7E) continue;
        const double cv = double(e4m3_value(uint32_t(c)));
        // exact: compare 2v with the sum of the two candidates
        const bool closer = (cv < bv) ? (2.0 * v < cv + bv) : (2.0 * v > cv + bv);
        const bool tie = (2.0 * v == cv + bv);
        if (closer || (tie && (c & 1) == 0)) { best = uint32_t(c); bv = cv; }
    }
    return best;
}

// E2M1 code of x / s for s > 0 by exact fp64 comparisons (ties to even).
__device__ __forceinline__ uint32_t e2m1_code_f64(double x, double s) {
    const double a = fabs(x);
    uint32_t c = 0;
    c += (a > 0.25 * s);
    c += (a >= 0.75 * s);
    c += (a > 1.25 * s);
    c += (a >= 1.75 * s);
    c += (a > 2.5 * s);
    c += (a >= 3.5 * s);
    c += (a > 5.0 * s);
    return c | (signbit(x) ? 8u : 0u);
}

// E2M1 pair via the hardware conversion (nearest-even, saturating at 6, sign
// kept): low nibble from `lo`.
__device__ __forceinline__ uint32_t e2m1x2_rn_sat(float lo, float hi) {
    uint16_t r;
    asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u16.u8 %0, t;\n}\n"
        : "=h"(r) : "f"(hi), "f"(lo));
    return r & 0xFF;
}

}  // namespace csa2
