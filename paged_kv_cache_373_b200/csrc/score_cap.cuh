// score_cap.cuh -- attention scores capped by a tanh: cap tanh(x / cap), in the
// log2 domain, shared by the decode and the chunked-prefill kernels.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// tanh y, |relative error| < 2^-22: below 1/2 an odd polynomial (a minimax fit
// of (tanh y) / y - 1 in y^2, off by 1.5e-8 at most), above it
// 1 - 2 / (1 + e^2|y|) with the hardware's 2^x and reciprocal, whose sum is at
// least 0.46 there and loses no digits to the subtraction.  y = +-inf gives +-1.
__device__ __forceinline__ float tanh_poly(float y) {
    const float z = y * y;
    float q = fmaf(z, 0.01724149100482464f, -0.05304549261927605f);
    q = fmaf(z, q, 0.13325878977775574f);
    q = fmaf(z, q, -0.333331435918808f);
    return fmaf(y * z, q, y);
}
__device__ __forceinline__ float tanh_exp(float y) {
    const float e = ex2(fabsf(y) * 2.885390081777927f);  // e^(2|y|)
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return copysignf(fmaf(-2.f, r, 1.f), y);
}

// N scores in place: x -> cap2 tanh(x pre), pre = (scale to the log2 domain) /
// cap2.  Which form of tanh is decided per lane for all its scores: the
// exponential form costs two more of the special-function unit's operations per
// score, and scores past half the cap are rare.
template <int N>
__device__ __forceinline__ void cap_scores(float (&x)[N], float pre, float cap2) {
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] *= pre;
        big = fmaxf(big, fabsf(x[i]));
    }
    if (big < 0.5f) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = cap2 * tanh_poly(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = cap2 * (fabsf(x[i]) < 0.5f ? tanh_poly(x[i]) : tanh_exp(x[i]));
    }
}

// The same without the final factor, N scores by pairs: x -> tanh(x pre).
template <int N>
__device__ __forceinline__ void cap_pairs(float (&x)[N], float pre) {
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) big = fmaxf(big, fabsf(x[i]));
    const F2 p2 = f2(pre, pre);
    if (big * pre < 0.5f) {
        const F2 c4 = f2(0.01724149100482464f, 0.01724149100482464f), c3 = f2(-0.05304549261927605f, -0.05304549261927605f),
                 c2 = f2(0.13325878977775574f, 0.13325878977775574f), c1 = f2(-0.333331435918808f, -0.333331435918808f);
#pragma unroll
        for (int i = 0; i < N; i += 2) {  // tanh_poly on two values
            const F2 y = f2_mul(f2(x[i], x[i + 1]), p2), z = f2_mul(y, y);
            const F2 q = f2_fma(z, f2_fma(z, f2_fma(z, c4, c3), c2), c1);
            const float2 r = f2_get(f2_fma(f2_mul(y, z), q, y));
            x[i] = r.x;
            x[i + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = x[i] * pre;
            x[i] = fabsf(y) < 0.5f ? tanh_poly(y) : tanh_exp(y);
        }
    }
}

}  // namespace pkv
