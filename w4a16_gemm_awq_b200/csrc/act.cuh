// act.cuh -- the activations of the feed-forward operators and their derivatives, in fp32.
//
//   SILU       p sg(p);                derivative sg + p sg (1 - sg),   sg(p) = 1 / (1 + e^-p)
//   GELU       p Phi(p);               derivative Phi + p phi,          Phi = (1 + erf(p / sqrt 2)) / 2
//   GELU_TANH  p (1 + tanh z) / 2 = p sg(2 z), z = sqrt(2 / pi) (p + 0.044715 p^3);
//              derivative sg + p sg (1 - sg) 2 z'
// The sigmoid is 1 / (1 + e^-p) by the fast exponential, within 2 + 1.173 |p| units of its last place, and the
// fast division, within 2.  For p >= 0 that is a relative error below 2^-20; for negative p, where e^-p decides,
// at most (5 + 1.2 |p|) 2^-23 (2^-18 at p = -20, 2^-16 where it underflows), far inside the bf16 rounding that
// every result goes through.  It saturates without a NaN: e^-p
// overflows to infinity for p below -88 and 1 / inf is 0, and p * 0 is 0 for every finite p.
#pragma once

#include <cuda_runtime.h>

#include "w4a16.h"

namespace w4a16 {

__device__ __forceinline__ float sigmoid_fast(float p) { return __fdividef(1.0f, 1.0f + __expf(-p)); }

template <int ACT>
__device__ __forceinline__ float act_value(float p) {
    if constexpr (ACT == W4A16_ACT_RELU) return p > 0.0f ? p : (p == p ? 0.0f : p);
    if constexpr (ACT == W4A16_ACT_SILU) return p * sigmoid_fast(p);
    if constexpr (ACT == W4A16_ACT_GELU) return 0.5f * p * (1.0f + erff(p * 0.70710678118654752f));
    if constexpr (ACT == W4A16_ACT_GELU_TANH)
        return p * sigmoid_fast(1.5957691216057308f * fmaf(0.044715f * p * p, p, p));
    return p;
}

template <int ACT>
__device__ __forceinline__ float act_grad(float p) {
    if constexpr (ACT == W4A16_ACT_RELU) return p > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == W4A16_ACT_SILU) {
        const float sg = sigmoid_fast(p);
        return fmaf(p * sg, 1.0f - sg, sg);
    }
    if constexpr (ACT == W4A16_ACT_GELU) {
        // Phi by formula 7.1.26 of Abramowitz and Stegun, "Handbook of Mathematical Functions" (erf to
        // 1.5e-7), which shares phi's exponential: 0.75e-7 absolute in a derivative of order 1.
        const float e = __expf(-0.5f * p * p), t = __fdividef(1.0f, fmaf(0.23164189f, fabsf(p), 1.0f));
        float c = fmaf(t, 1.061405429f, -1.453152027f);
        c = fmaf(t, c, 1.421413741f);
        c = fmaf(t, c, -0.284496736f);
        c = fmaf(t, c, 0.254829592f);
        const float tail = 0.5f * t * c * e;  // 1 - Phi(|p|)
        return fmaf(p * 0.39894228040143268f, e, p > 0.0f ? 1.0f - tail : tail);
    }
    if constexpr (ACT == W4A16_ACT_GELU_TANH) {
        const float sg = sigmoid_fast(1.5957691216057308f * fmaf(0.044715f * p * p, p, p));
        const float q = fminf(fabsf(p), 32.0f);  // beyond, sg is 0 or 1, and q^2 must not become infinite beside it
        return fmaf(p * sg, (1.0f - sg) * 1.5957691216057308f * fmaf(0.134145f * q, q, 1.0f), sg);
    }
    return 1.0f;
}

// The activation of C values held in registers, the choice made once for all of them: a choice per
// value makes C copies of every activation's code, which then comes from the instruction cache's
// misses (a GEMM epilogue of 32 values took 6000 cycles that way).
template <int C, int ACT>
__device__ __forceinline__ void act_each(float (&v)[C]) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = act_value<ACT>(v[i]);
}

template <int C>
__device__ __forceinline__ void act_values(int act, float (&v)[C]) {
    switch (act) {
        case W4A16_ACT_RELU: act_each<C, W4A16_ACT_RELU>(v); break;
        case W4A16_ACT_SILU: act_each<C, W4A16_ACT_SILU>(v); break;
        case W4A16_ACT_GELU: act_each<C, W4A16_ACT_GELU>(v); break;
        case W4A16_ACT_GELU_TANH: act_each<C, W4A16_ACT_GELU_TANH>(v); break;
        default: break;
    }
}

}  // namespace w4a16
