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

// code + 128 of x under the row's scale.
__device__ __forceinline__ uint32_t int8_code(float x, float scale) {
    if (!(scale > 0.f)) return 128u;
    const float y = __fdiv_rn(x, scale);
    if (y != y) return 128u;
    return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(y), -127.f), 127.f)) + 128);
}

// x / t as e2m1's converter takes it (a NaN is stored as 0).
__device__ __forceinline__ float fp4_quotient(float x, float t) {
    if (!(t > 0.f)) return 0.f;
    const float y = __fdiv_rn(x, t);
    return y != y ? 0.f : y;
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
