// cap.cuh -- scores capped by a tanh: s -> cap * tanh(s / cap), the score
// s = softmax scale * (q . k), applied before the mask.
//
// The kernels keep scores in the log2 domain: u = sl * x for a dot product x,
// capped c2 * tanh(y) with y = u / c2 and c2 = cap * log2(e) (CapArgs).  The cap
// is increasing, so a row's largest capped score is the capped largest dot
// product.
//
// tanh in three forms:
//   * CUDA's tanhf (fp32 outputs);
//   * 1 - 2 / (1 + e^2y), two SFU operations, absolute error a few 1e-7 (below
//     |y| = 1/16, where that would be much of a small y, y - y^3 / 3): relative
//     error up to 6e-6, any y;
//   * poly_fma2: y * P(y^2) on the FMA pipe for |y| <= 0.7, where nearly all
//     scores of a trained model lie (|s| <= 0.7 cap); P has four coefficients,
//     fitted here to the smallest largest relative error there, 6.8e-6: at a
//     cap of 50 at most 2.1e-4 of a weight, far below the 2^-8 of its rounding
//     to bf16.  The tensor-core kernels use it for a warp's part of a tile when
//     every |y| there is in range: their SFU share (the exponentials) is
//     already as large as the MMAs' time.
// Under a cap far above the scores y may leave fp32's normal range where its
// score does not (a cap of 1e38 has y = 1e-38 for a score of 1).  There
// (CapArgs::far) the first two take small scores from u, not from c2 * tanh(y).
// The third is used for caps up to 65,536 softmax scales.
#pragma once

#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace duo {

// 2^x and 1/x on the SFU (PTX approximations)
__device__ __forceinline__ float sfu_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sfu_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The capped score of x, and its tanh: u = sl * x, y = k * x.
struct Capped {
    float s, t;
};
template <bool FAR = true>   // false: CapArgs::far is known to be 0, one operation less
__device__ __forceinline__ Capped cap_sfu(float x, float sl, float k, float c2) {
    // e^2y overflows to inf for large y (1 / inf = 0: tanh = 1) and underflows
    // to 0 for small y (tanh = -1)
    const float y = x * k, e = sfu_exp2(y * (2.f * kLog2e));
    const float t = fmaf(-2.f, sfu_rcp(1.f + e), 1.f);
    const bool small = fabsf(y) < 0.0625f;
    if constexpr (FAR) {
        const float u = x * sl, near = fmaf(y * y, -1.f / 3.f, 1.f);
        return {small ? u * near : c2 * t, small ? y * near : t};
    }
    const float v = small ? fmaf(y * y * y, -1.f / 3.f, y) : t;
    return {__fmul_rn(c2, v), v};   // a score of its own, not the half of a fused sum
}
template <bool FAR>
__device__ __forceinline__ Capped cap_exact(float x, float sl, const CapArgs& cap) {
    if constexpr (FAR) {
        // below the bound the cap moves u by less than half a step of fp32
        const float u = x * sl, y = u * cap.rc2, t = tanhf(y);
        return {fabsf(y) < 0x1p-12f ? u : cap.c2 * t, t};
    }
    const float t = tanhf(x * cap.k);
    return {cap.c2 * t, t};
}

constexpr float kTanh0 = 0.9999933242797852f, kTanh1 = -0.33289048075675964f, kTanh2 = 0.12864212691783905f,
                kTanh3 = -0.037290528416633606f;

// f * tanh(k x), k = sl / c2, of a pair of dot products with |x| in range: the
// polynomial's coefficients times f and the powers of k, so that it takes x
// itself; u is x^2.  A kernel parameter: every constant is a pair of equal
// halves, as the packed instructions take them, read from the parameter bank
// instead of held in registers.
struct TanhPoly {
    float2 a0, a1, a2, a3;
    float2 c2, minus1;     // c2 = cap log2(e); -1
    float x_max, x2_max;   // the largest |x| in range, and its square; negative: none
};
inline TanhPoly tanh_poly(const CapArgs& cap, float f) {
    auto two = [](double x) { return make_float2((float)x, (float)x); };
    if (!cap.on) return {two(0.0), two(0.0), two(0.0), two(0.0), two(0.0), two(-1.0), -1.f, -1.f};
    const double k = cap.k, k2 = k * k, s0 = f * k, s1 = s0 * k2, s2 = s1 * k2;
    TanhPoly p{two(kTanh0 * s0), two(kTanh1 * s1), two(kTanh2 * s2), two(kTanh3 * s2 * k2), two(cap.c2), two(-1.0), -1.f, -1.f};
    // not with a k whose powers leave fp32's normal range
    if (k >= 0x1p-16 && std::isfinite(p.a0.x) && std::isfinite(p.a3.x)) {
        p.x_max = (float)(0.7 / k);
        p.x2_max = p.x_max * p.x_max;
    }
    return p;
}
__device__ __forceinline__ float2 poly_fma2(float2 x, float2 u, const TanhPoly& c) {
    float2 p = ffma2(u, c.a3, c.a2);
    p = ffma2(p, u, c.a1);
    p = ffma2(p, u, c.a0);
    return fmul2(p, x);
}
__device__ __forceinline__ float2 poly_fma2(float2 x, const TanhPoly& c) { return poly_fma2(x, fmul2(x, x), c); }

// The largest |x|, in four chains.
template <int W>
__device__ __forceinline__ float largest(const float* x) {
    static_assert(W % 8 == 0, "pairs for four chains");
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < W; c += 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = fmax3(m[i], fabsf(x[c + 2 * i]), fabsf(x[c + 2 * i + 1]));
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// The log2-domain score of a dot product: x * sl, or capped.
template <bool CAP, bool FAR = true>
__device__ __forceinline__ float score_log2(float x, float sl, const CapArgs& cap) {
    if constexpr (!CAP) return x * sl;
    return cap_sfu<FAR>(x, sl, cap.k, cap.c2).s;
}

}  // namespace duo
