// quant.cuh -- the records of the quantised pools (int8 with a scale per row,
// 4-bit e2m1 with an e4m3 scale per 16 dims): where a row's codes and scales
// sit, and the rounding of a row into them.  include/pkv.h states the format.
#pragma once

#include <cuda_fp4.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {

template <int D, bool kFp4>
struct QuantRecord {
    static constexpr int kRowBytes = kFp4 ? D / 2 : D;            // a row's codes
    static constexpr int kScaleBytes = kFp4 ? D / kBlockSize : 4;  // a row's scales
    static constexpr int kScales = kBlockSize * kRowBytes;         // offset of the scales
    static constexpr int kBytes = kScales + kBlockSize * kScaleBytes;
    static constexpr int kChunks = kRowBytes / 16;
};

// Offset of 16-byte chunk c of row r's codes in a record.
template <int kRowBytes>
__host__ __device__ __forceinline__ constexpr int quant_chunk(int r, int c) {
    return r * kRowBytes + ((c ^ ((r * kRowBytes / 128) & (kRowBytes / 16 - 1))) << 4);
}

// Offset of byte b of row r's codes.
template <int kRowBytes>
__host__ __device__ __forceinline__ constexpr int quant_byte(int r, int b) {
    return quant_chunk<kRowBytes>(r, b >> 4) + (b & 15);
}

// The magnitude that counts towards a scale: NaN and infinities do not.
__device__ __forceinline__ float finite_magnitude(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;
}

// x[e] / t rounded to nearest for 8 elements, a NaN (and any x over t = 0) as 0.
//
// One correctly rounded reciprocal r serves all: q = x r is within 2 ulp of x / t, a step
// q + (x - q t) r brings it within 1, and by Markstein's theorem (P. W. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990) another such step
// from within 1 ulp, with r = RN(1 / t) and the remainder exact, is the rounded quotient.
// t within 2^+-90 keeps the remainders of all quotients above 2^-12 normal, hence exact;
// smaller quotients become code 0 however they round.  The remainder is taken as q t - x
// so that a zero keeps its sign.  Rows with NaN, infinities or such t divide one by one.
// (With a division per value the append of 4096 tokens of 32 + 8 heads of 128 took 36 us.)
__device__ __forceinline__ bool plain_divisor(float t) {
    return t >= 8.077935669463161e-28f && t <= 1.2379400392853803e27f;  // 2^-90, 2^90
}
__device__ __forceinline__ float divisor_reciprocal(float t) { return __frcp_rn(plain_divisor(t) ? t : 1.f); }
// r: divisor_reciprocal(t)
__device__ __forceinline__ void quotients(const float (&x)[8], float t, float r, float (&y)[8]) {
    const uint64_t rr = pack_f32x2(r, r), tt = pack_f32x2(t, t), nr = pack_f32x2(-r, -r), m1 = pack_f32x2(-1.f, -1.f);
    uint64_t sums = 0;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint64_t xx = pack_f32x2(x[e], x[e + 1]), nx = mul_f32x2(xx, m1);
        uint64_t q = mul_f32x2(xx, rr);
        q = fma_f32x2(fma_f32x2(q, tt, nx), nr, q);
        q = fma_f32x2(fma_f32x2(q, tt, nx), nr, q);
        unpack_f32x2(q, y[e], y[e + 1]);
        sums = add_f32x2(sums, q);
    }
    float sum, sum1;
    unpack_f32x2(sums, sum, sum1);
    sum += sum1;
    if (!plain_divisor(t) || sum - sum != 0.f) {  // an infinity's remainder is a NaN, and an overflowed sum is taken along
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = t > 0.f ? __fdiv_rn(x[e], t) : 0.f;
            y[e] = q != q ? 0.f : q;
        }
    }
}

// 8 quotients -> bytes of code + 128, rounded to nearest even: 1.5 2^23 + 128 + y has the
// code in its low byte.
__device__ __forceinline__ uint2 int8_codes(const float (&y)[8]) {
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = __float_as_uint(__fadd_rn(fminf(fmaxf(y[e], -127.f), 127.f), 12583040.f));
    return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}

// Two quotients -> a byte, the first in the low nibble.
__device__ __forceinline__ uint32_t fp4_pair(float lo, float hi) {
    return __nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}

// The e4m3 scale of 16 dims with largest finite magnitude amax.
__device__ __forceinline__ uint32_t fp4_scale_code(float amax, float g) {
    return __nv_cvt_float_to_fp8(fminf(__fdiv_rn(amax, __fmul_rn(6.f, g)), 448.f), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float e4m3_float(uint32_t code) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
    return __half2float(__half(h));
}

// A byte's two e2m1 values, packed f16 (exact), the low nibble's in the low half.
__device__ __forceinline__ uint32_t fp4x2_to_f16x2(uint32_t byte) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
    return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}

}  // namespace pkv
