// cap.cuh -- scores capped by a tanh: s -> cap * tanh(s / cap), the score
// s = softmax scale * (q . k), applied before the mask.
//
// The kernels keep scores in the log2 domain, so the capped score of a dot
// product x is c2 * tanh(x * k) with k = scale / cap and c2 = cap * log2(e)
// (CapArgs).  The cap is increasing, so a row's largest capped score is the
// capped largest dot product.
//
// tanh in two forms:
//   * tanh_sfu: 1 - 2 / (1 + e^2y), two SFU operations, absolute error a few
//     1e-7; below |y| = 1/16, where that would be much of a small y (a large
//     cap scales it back up), y - y^3 / 3.  Relative error up to 6e-6, any y.
//   * poly_fma2: y * P(y^2) on the FMA pipe for |y| <= 0.7, where nearly all
//     scores of a trained model lie (|s| <= 0.7 cap); P has four coefficients,
//     fitted here to the smallest largest relative error there, 6.8e-6: at a
//     cap of 50 at most 2.1e-4 of a weight, far below the 2^-8 of its rounding
//     to bf16.  The tensor-core kernels use it for a warp's part of a tile when
//     every |y| there is in range: their SFU share (the exponentials) is
//     already as large as the MMAs' time.
#pragma once

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

__device__ __forceinline__ float tanh_sfu(float y) {
    // e^2y overflows to inf for large y (1 / inf = 0: tanh = 1) and underflows
    // to 0 for small y (tanh = -1)
    const float e = sfu_exp2(y * (2.f * kLog2e));
    const float t = fmaf(-2.f, sfu_rcp(1.f + e), 1.f);
    return fabsf(y) < 0.0625f ? fmaf(y * y * y, -1.f / 3.f, y) : t;
}

constexpr float kTanhRange = 0.7f;   // of |y|
constexpr float kTanh0 = 0.9999933242797852f, kTanh1 = -0.33289048075675964f, kTanh2 = 0.12864212691783905f,
                kTanh3 = -0.037290528416633606f;

// f * tanh(k x) of a pair of dot products with |k x| in range: the
// polynomial's coefficients times f and the powers of k, so that it takes x
// itself; u is x^2.  A kernel parameter: every constant is a pair of equal
// halves, as the packed instructions take them, read from the parameter bank
// instead of held in registers.
struct TanhPoly {
    float2 a0, a1, a2, a3;
    float2 c2, minus1;   // c2 = cap log2(e); -1
    float x2_max;        // the largest x^2 in range
};
inline TanhPoly tanh_poly(const CapArgs& cap, float f) {
    const float k = cap.k, k2 = k * k, s0 = f * k, s1 = s0 * k2, s2 = s1 * k2;
    auto two = [](float x) { return make_float2(x, x); };
    return {two(kTanh0 * s0), two(kTanh1 * s1), two(kTanh2 * s2), two(kTanh3 * (s2 * k2)),
            two(cap.c2),      two(-1.f),        cap.on ? (kTanhRange / k) * (kTanhRange / k) : 0.f};
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

// The log2-domain score of a dot product: x * sl, or capped.  EXACT takes
// CUDA's tanhf (the fp32 paths).
template <bool CAP, bool EXACT = false>
__device__ __forceinline__ float score_log2(float x, float sl, const CapArgs& cap) {
    if constexpr (!CAP) return x * sl;
    return cap.c2 * (EXACT ? tanhf(x * cap.k) : tanh_sfu(x * cap.k));
}

}  // namespace duo
