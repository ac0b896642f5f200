// score_cap.cuh -- attention scores capped by a tanh: cap tanh(x / cap), in the
// log2 domain, shared by the decode and the chunked-prefill kernels.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// tanh y, |relative error| below 2.1 * 2^-22: below 1/2 an odd polynomial (a minimax
// fit of (tanh y) / y - 1 in y^2, off by 1.6e-8 at most; with its roundings 0.4 *
// 2^-22), above it 1 - 2 / (1 + e^2|y|) with the hardware's 2^x (documented to 2^-22)
// and reciprocal (one unit in the last place).  That is worst at 1/2, where e^2|y|'s
// error counts 0.39, the reciprocal's 2^-24 and the roundings of 1 + e and of the
// difference 2^-25 in all, over a result of 0.46.  y = +-inf gives +-1.
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

// The same for many raw scores per lane, as few operations as the prefill
// kernel can spend: x -> tanh(x pre) / pre.  While every |x pre| < 0.35 that is
// x (1 + z q(z)) with z = x^2 and the polynomial's powers of pre in its
// coefficients (a minimax fit of degree 3 in y^2, off by 4.1e-8 at most): 5
// operations a score.  Otherwise, and for a pre whose sixth power leaves fp32, as
// above.
struct CapCoef {
    F2 c1, c2, c3;
    float pre, inv_pre, lim;  // lim: largest |x| for the polynomial (0: never)
};
__device__ __forceinline__ CapCoef cap_coef(float pre, float inv_pre) {
    CapCoef k;
    const float p2 = pre * pre;
    const float a = -0.33332663774490356f * p2, b = 0.1329982578754425f * p2 * p2, c = -0.049148499965667725f * p2 * p2 * p2;
    k.c1 = f2(a, a);
    k.c2 = f2(b, b);
    k.c3 = f2(c, c);
    k.pre = pre;
    k.inv_pre = inv_pre;
    k.lim = pre > 0x1p-14f && pre < 0x1p14f ? 0.35f / pre : 0.f;
    return k;
}
template <int N>
__device__ __forceinline__ void cap_pairs(float (&x)[N], const CapCoef& k) {
    float big[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; i += 2) big[(i >> 1) & 1] = fmaxf(big[(i >> 1) & 1], fmaxf(fabsf(x[i]), fabsf(x[i + 1])));
    if (fmaxf(big[0], big[1]) < k.lim) {
        const F2 one = f2(1.f, 1.f);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const F2 v = f2(x[i], x[i + 1]), z = f2_mul(v, v);
            const float2 r = f2_get(f2_mul(v, f2_fma(z, f2_fma(z, f2_fma(z, k.c3, k.c2), k.c1), one)));
            x[i] = r.x;
            x[i + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = x[i] * k.pre;
            x[i] = (fabsf(y) < 0.5f ? tanh_poly(y) : tanh_exp(y)) * k.inv_pre;
        }
    }
}

}  // namespace pkv
