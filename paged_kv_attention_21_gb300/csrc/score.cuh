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
// with fp32 arithmetic 1e-7 of the value.  1 - 2 / (e^2y + 1), used beyond,
// is off by about 1.5e-7 of 1 wherever it is evaluated: near 0 that would be an
// absolute error of 1.5e-7 cap in every logit, 7e-6 for a cap of 50.
constexpr float kTanhC0 = -0.3333319127559662f;
constexpr float kTanhC1 = 0.1332911103963852f;
constexpr float kTanhC2 = -0.05355885997414589f;
constexpr float kTanhC3 = 0.020091967657208443f;
constexpr float kTanhC4 = -0.005138659384101629f;

// The same for |y| <= 0.3, off by 1.2e-8: three coefficients serve where all of a tile's
// scores are that small.  Logits of standard deviation 2 are under a cap of 50 (8 x 512 tokens
// over up to 8704 keys: prefill 362 us, weights 250), under one of 20 they are not (393, 282),
// and under one of 10 and of 6.7 ever more tiles hold a score past kTanhPoly (639 and 862; 429
// and 565).
constexpr float kTanhNear = 0.3f;
constexpr float kTanhN0 = -0.33333060145378113f;
constexpr float kTanhN1 = 0.13314832746982574f;
constexpr float kTanhN2 = -0.05036623775959015f;

// For any y: e^2|y| overflows to inf from |y| = 44 on, where tanh is 1 to fp32.
__device__ __forceinline__ float tanh_exp(float y) {
    const float e = fast_exp2(fabsf(y) * 2.8853900817779268f);
    return copysignf(1.f - __fdividef(2.f, e + 1.f), y);
}

constexpr float kLog2e = 1.4426950408889634f;

// What a kernel needs of the rule for one KV head (kscale: the head's e4m3 scale, or 1).
// A score's logit has the same bits whichever of the forms below computes it, but for
// TanhPair::near: which form does may depend on the scores beside it.
struct ScoreScale {
    float in;    // s -> y = sm_scale s / cap with a cap, else s -> log2 units
    float out;   // cap log2(e) with a cap, else 0
    __device__ __forceinline__ ScoreScale(float sm_scale, float cap, float kscale) {
        in = cap > 0.f ? sm_scale * kscale / cap : sm_scale * kLog2e * kscale;
        out = cap > 0.f ? cap * kLog2e : 0.f;
    }
    // out tanh(y) / y for |y| <= kTanhPoly: the factor `out` is in the coefficients
    __device__ __forceinline__ float factor(float y) const {
        const float z = y * y;
        float p = fmaf(z, kTanhC4 * out, kTanhC3 * out);
        p = fmaf(z, p, kTanhC2 * out);
        p = fmaf(z, p, kTanhC1 * out);
        p = fmaf(z, p, kTanhC0 * out);
        return fmaf(z, p, out);
    }
    __device__ __forceinline__ float capped(float s) const {
        const float y = s * in;
        return fabsf(y) <= kTanhPoly ? y * factor(y) : out * tanh_exp(y);
    }
    __device__ __forceinline__ float capped(float s, float c) const {
        const float y = s * in;
        return fabsf(y) <= kTanhPoly ? fmaf(y, factor(y), c) : fmaf(out, tanh_exp(y), c);
    }
    __device__ __forceinline__ float operator()(float s) const { return out > 0.f ? capped(s) : s * in; }
    __device__ __forceinline__ float operator()(float s, float c) const { return out > 0.f ? capped(s, c) : fmaf(s, in, c); }
};

// ScoreScale's capped(), two logits at a time, where every |y| <= kTanhPoly.
struct TanhPair {
    uint64_t in, c0, c1, c2, c3, c4, one, n0, n1, n2;
    __device__ __forceinline__ explicit TanhPair(const ScoreScale& sc) {
        in = pack_f32x2(sc.in, sc.in);
        auto twice = [&](float k) { return pack_f32x2(k * sc.out, k * sc.out); };
        one = twice(1.f), c0 = twice(kTanhC0), c1 = twice(kTanhC1), c2 = twice(kTanhC2);
        c3 = twice(kTanhC3), c4 = twice(kTanhC4);
        n0 = twice(kTanhN0), n1 = twice(kTanhN1), n2 = twice(kTanhN2);
    }
    // |y| <= kTanhNear.  Chosen by scores that are the sequence's own, so that a call repeats its bits
    __device__ __forceinline__ uint64_t near(uint64_t s, uint64_t c) const {
        const uint64_t y = mul_f32x2(s, in), z = mul_f32x2(y, y);
        return fma_f32x2(y, fma_f32x2(z, fma_f32x2(z, fma_f32x2(z, n2, n1), n0), one), c);
    }
    __device__ __forceinline__ uint64_t factor(uint64_t y) const {  // out tanh(y) / y
        const uint64_t z = mul_f32x2(y, y);
        uint64_t p = fma_f32x2(z, c4, c3);
        p = fma_f32x2(z, p, c2);
        p = fma_f32x2(z, p, c1);
        p = fma_f32x2(z, p, c0);
        return fma_f32x2(z, p, one);
    }
    __device__ __forceinline__ uint64_t operator()(uint64_t s) const {
        const uint64_t y = mul_f32x2(s, in);
        return mul_f32x2(y, factor(y));
    }
    __device__ __forceinline__ uint64_t operator()(uint64_t s, uint64_t c) const {
        const uint64_t y = mul_f32x2(s, in);
        return fma_f32x2(y, factor(y), c);
    }
};

// ScoreScale's capped(s) and capped(s, c) of two scores of every lane of the warp: the
// pair's polynomial, and where some lane's |y| lies past it, capped() as well.
__device__ __forceinline__ bool past_poly(const ScoreScale& sc, float s0, float s1) {
    return __any_sync(0xFFFFFFFFu, !(fabsf(s0) * sc.in <= kTanhPoly && fabsf(s1) * sc.in <= kTanhPoly));
}
__device__ __forceinline__ void capped_pair(const ScoreScale& sc, const TanhPair& tp, float s0, float s1, float& x0,
                                            float& x1) {
    unpack_f32x2(tp(pack_f32x2(s0, s1)), x0, x1);
    if (past_poly(sc, s0, s1)) {
        x0 = sc.capped(s0);
        x1 = sc.capped(s1);
    }
}
__device__ __forceinline__ void capped_pair(const ScoreScale& sc, const TanhPair& tp, float s0, float s1, float c,
                                            float& x0, float& x1) {
    unpack_f32x2(tp(pack_f32x2(s0, s1), pack_f32x2(c, c)), x0, x1);
    if (past_poly(sc, s0, s1)) {
        x0 = sc.capped(s0, c);
        x1 = sc.capped(s1, c);
    }
}

// The largest |y| of N scores (a NaN: not looked at).
template <int N>
__device__ __forceinline__ float largest(const float (&v)[N], float in) {
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < N; e += 2) m[(e >> 1) & 3] = fmax3(m[(e >> 1) & 3], fabsf(v[e]), fabsf(v[e + 1]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * in;
}

}  // namespace pkv
