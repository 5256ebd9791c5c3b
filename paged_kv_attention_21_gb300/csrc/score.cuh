// score.cuh -- the score rule of the pkv_score_* entry points (sm_103a).
//
// With s = q.k (fp32, from the MMA), the logit in log2 units is
//     x = log2(e) (cap tanh(sm_scale s / cap) - slope |p - t|)
// (without a cap: log2(e) sm_scale s), for a query at position p and key t.
#pragma once

#include "common.cuh"

namespace pkv {

// |y| up to which tanh is taken from its polynomial.
constexpr float kTanhPoly = 0.7f;

// tanh(y) = y (1 + z P(z)), z = y^2, for |y| <= 0.7: P is the fit of least
// relative error (reweighted least squares on Chebyshev nodes), off by 1.5e-8;
// with fp32 arithmetic 8.5e-8 of the value.  1 - 2 / (e^2y + 1), used beyond,
// is off by about 1.5e-7 of 1 wherever it is evaluated: near 0 that would be an
// absolute error of 1.5e-7 cap in every logit, 7e-6 for a cap of 50.
constexpr float kTanhC0 = -0.3333319127559662f;
constexpr float kTanhC1 = 0.1332911103963852f;
constexpr float kTanhC2 = -0.05355885997414589f;
constexpr float kTanhC3 = 0.020091967657208443f;
constexpr float kTanhC4 = -0.005138659384101629f;

__device__ __forceinline__ float tanh_poly(float y) {
    const float z = y * y;
    float p = fmaf(z, kTanhC4, kTanhC3);
    p = fmaf(z, p, kTanhC2);
    p = fmaf(z, p, kTanhC1);
    p = fmaf(z, p, kTanhC0);
    return fmaf(y * z, p, y);
}

// For any y: e^2|y| overflows to inf from |y| = 44 on, where tanh is 1 to fp32.
__device__ __forceinline__ float tanh_exp(float y) {
    const float e = fast_exp2(fabsf(y) * 2.8853900817779268f);
    return copysignf(1.f - __fdividef(2.f, e + 1.f), y);
}

__device__ __forceinline__ float tanh_any(float y) { return fabsf(y) <= kTanhPoly ? tanh_poly(y) : tanh_exp(y); }

constexpr float kLog2e = 1.4426950408889634f;

// What a kernel needs of the rule for one KV head (kscale: the head's e4m3 scale, or 1).
struct ScoreScale {
    float in;    // s -> y = sm_scale s / cap with a cap, else s -> log2 units
    float out;   // cap log2(e) with a cap, else 0
    __device__ __forceinline__ ScoreScale(float sm_scale, float cap, float kscale) {
        in = cap > 0.f ? sm_scale * kscale / cap : sm_scale * kLog2e * kscale;
        out = cap > 0.f ? cap * kLog2e : 0.f;
    }
    __device__ __forceinline__ float operator()(float s) const {
        const float y = s * in;
        return out > 0.f ? out * tanh_any(y) : y;
    }
};

}  // namespace pkv
