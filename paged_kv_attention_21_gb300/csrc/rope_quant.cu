// rope_quant.cu -- rotary positions in both pair layouts, and the quantised
// pools' append, row read and block widening (formats: include/pkv.h).
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace pkv {

namespace {

// ------------------------------------------------------------- rotation --
//
// One thread per (token, head, element pair or passing element).

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
    return static_cast<float>(x);
}
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
    return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// x' = (a c - b s, b c + a s), each op rounded
__device__ __forceinline__ float2 turn(float a, float b, float c, float s) {
    return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

template <typename T>
__global__ void __launch_bounds__(256) rope_rotate_kernel(RotateArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int half = a.rotary / 2;
    const int items = a.d - half;  // pairs, then the dims that pass
    const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int it = static_cast<int>(idx % items);
    const long long row = idx / items;
    const int heads = a.q.num_heads + a.k.num_heads;
    const long long i = row / heads;
    int h = static_cast<int>(row % heads);
    if (i >= a.num_tokens) return;
    const int p = a.positions[i];
    if (p < 0) return;
    if (p >= a.max_pos) {
        if (it == 0) flag_error(a.err, PKV_DEVERR_POSITION);
        return;
    }
    const bool is_k = h >= a.q.num_heads;
    const RotateRows& r = is_k ? a.k : a.q;
    if (is_k) h -= a.q.num_heads;
    const T* in = static_cast<const T*>(r.in) + i * r.in_token + h * r.in_head;
    T* out = static_cast<T*>(r.out) + i * r.out_token + h * r.out_head;
    if (it >= half) {
        out[it + half] = in[it + half];
        return;
    }
    const float* cs = a.cos_sin + (static_cast<size_t>(p) * half + it) * 2;
    const int e0 = a.interleaved ? 2 * it : it;
    const int e1 = a.interleaved ? 2 * it + 1 : it + half;
    const float2 y = turn(to_f32(in[e0]), to_f32(in[e1]), cs[0], a.inverse ? -cs[1] : cs[1]);
    out[e0] = from_f32<T>(y.x);
    out[e1] = from_f32<T>(y.y);
}

// --------------------------------------------------------------- append --
//
// One warp per (token, row); rows are the Hkv K heads, the Hkv V heads and
// the Hq query heads.  Lane l owns dims [l D/32, (l + 1) D/32).

// The block and slot of a token: false for padding and for a bad position or
// block id (flagged by `report`).
__device__ __forceinline__ bool quant_slot(const QuantArgs& a, int i, bool report, int* blk, int* row) {
    const int s = a.token_to_seq[i];
    if (s < 0) return false;
    const int p = a.positions[i];
    const int tb = a.ring > 0 ? (p / kBlockSize) % a.ring : p / kBlockSize;
    if (s >= a.num_seqs || p < 0 || tb >= a.mbps || (a.cos_sin != nullptr && p >= a.max_pos)) {
        if (report) flag_error(a.err, PKV_DEVERR_POSITION);
        return false;
    }
    *row = p % kBlockSize;
    *blk = a.block_tables[static_cast<size_t>(s) * a.mbps + tb];
    if (*blk < 0 || *blk >= a.num_blocks) {
        if (report) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
        return false;
    }
    return true;
}

template <int D, bool kFp4>
__global__ void __launch_bounds__(256) quant_append_kernel(QuantArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    using R = QuantRecord<D, kFp4>;
    constexpr int E = D / 32;  // dims of a lane
    const int lane = threadIdx.x & 31;
    const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int rows = 2 * a.hkv + (a.q ? a.hq : 0);
    const long long i = w / rows;
    int r = static_cast<int>(w % rows);
    if (i >= a.num_tokens) return;
    int blk, row;
    if (!quant_slot(a, static_cast<int>(i), lane == 0, &blk, &row)) return;
    const int p = a.positions[i];
    const bool is_k = r < a.hkv, is_q = r >= 2 * a.hkv;
    const int h = is_q ? r - 2 * a.hkv : is_k ? r : r - a.hkv;
    const __nv_bfloat16* x =
        is_q ? static_cast<const __nv_bfloat16*>(a.q) + i * a.q_stride + static_cast<size_t>(h) * D
             : static_cast<const __nv_bfloat16*>(is_k ? a.k_new : a.v_new) + i * a.new_stride + static_cast<size_t>(h) * D;
    float v[E];
    const int half = a.rotary / 2;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int d = lane * E + e;
        v[e] = __bfloat162float(x[d]);
        if (a.cos_sin && (is_k || is_q) && d < a.rotary) {
            const bool second = a.interleaved ? (d & 1) : d >= half;
            const int j = a.interleaved ? d >> 1 : second ? d - half : d;
            const int mate = a.interleaved ? d ^ 1 : second ? d - half : d + half;
            const float* cs = a.cos_sin + (static_cast<size_t>(p) * half + j) * 2;
            const float m = __bfloat162float(x[mate]);
            const float s = a.inverse ? -cs[1] : cs[1];
            v[e] = second ? turn(m, v[e], cs[0], s).y : turn(v[e], m, cs[0], s).x;
        }
    }
    __syncwarp();  // q in place: every lane has read its pairs
    if (is_q) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.q_out) + i * a.q_out_stride + static_cast<size_t>(h) * D;
#pragma unroll
        for (int e = 0; e < E; ++e) o[lane * E + e] = __float2bfloat16_rn(v[e]);
        return;
    }
    uint8_t* rec = static_cast<uint8_t*>(is_k ? a.k_pool : a.v_pool) + (static_cast<size_t>(blk) * a.hkv + h) * R::kBytes;
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) amax = fmaxf(amax, finite_magnitude(v[e]));
    if constexpr (kFp4) {
        constexpr int kLanes = 16 / E;  // lanes of one scale
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const float g = (is_k ? a.k_scale : a.v_scale)[h];
        const uint32_t sc = fp4_scale_code(amax, g);
        const float t = __fmul_rn(e4m3_float(sc), g);
#pragma unroll
        for (int e = 0; e < E; e += 2)
            rec[quant_byte<R::kRowBytes>(row, (lane * E + e) / 2)] =
                static_cast<uint8_t>(fp4_pair(fp4_quotient(v[e], t), fp4_quotient(v[e + 1], t)));
        if (lane % kLanes == 0) rec[R::kScales + row * R::kScaleBytes + lane / kLanes] = static_cast<uint8_t>(sc);
    } else {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const float sc = __fdiv_rn(amax, 127.f);
#pragma unroll
        for (int e = 0; e < E; ++e)
            rec[quant_byte<R::kRowBytes>(row, lane * E + e)] = static_cast<uint8_t>(int8_code(v[e], sc));
        if (lane == 0) *reinterpret_cast<float*>(rec + R::kScales + row * 4) = sc;
    }
}

// ----------------------------------------------------------------- read --

template <int D, bool kFp4>
__global__ void __launch_bounds__(256) quant_read_kernel(QuantArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int d = static_cast<int>(idx % D);
    const int h = static_cast<int>((idx / D) % a.hkv);
    const long long i = idx / D / a.hkv;
    if (i >= a.num_tokens) return;
    int blk, row;
    if (!quant_slot(a, static_cast<int>(i), d == 0, &blk, &row)) return;
    const size_t at = (static_cast<size_t>(blk) * a.hkv + h) * QuantRecord<D, kFp4>::kBytes;
    const size_t to = (static_cast<size_t>(i) * a.hkv + h) * D + d;
#pragma unroll
    for (int pool = 0; pool < 2; ++pool) {
        const void* src = pool ? a.v_pool : a.k_pool;
        void* dst = pool ? a.v_out : a.k_out;
        if (!dst) continue;
        const float g = kFp4 ? (pool ? a.v_scale : a.k_scale)[h] : 1.f;
        const float v = quant_value<D, kFp4>(static_cast<const uint8_t*>(src) + at, row, d, g);
        if (a.out_f32)
            static_cast<float*>(dst)[to] = v;
        else
            static_cast<__nv_bfloat16*>(dst)[to] = __float2bfloat16_rn(v);
    }
}

template <int D, bool kFp4>
__global__ void __launch_bounds__(256) quant_load_kernel(QuantArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int i = blockIdx.x;
    const int h = blockIdx.y;
    const int src = a.src_blocks[i], dst = a.dst_blocks[i];
    if (src < 0 || src >= a.num_blocks || dst < 0 || dst >= a.dst_num_blocks) {
        if (threadIdx.x == 0) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
        return;
    }
    const uint8_t* rec = static_cast<const uint8_t*>(blockIdx.z ? a.v_pool : a.k_pool) +
                         (static_cast<size_t>(src) * a.hkv + h) * QuantRecord<D, kFp4>::kBytes;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(blockIdx.z ? a.v_out : a.k_out) +
                         (static_cast<size_t>(dst) * a.hkv + h) * kBlockSize * D;
    const float g = kFp4 ? (blockIdx.z ? a.v_scale : a.k_scale)[h] : 1.f;
    for (int e = threadIdx.x; e < kBlockSize * D; e += blockDim.x)
        out[e] = __float2bfloat16_rn(quant_value<D, kFp4>(rec, e / D, e % D, g));
}

cudaError_t grid_of(long long threads, dim3* grid) {
    const long long blocks = (threads + 255) / 256;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    *grid = dim3(static_cast<unsigned>(blocks));
    return cudaSuccess;
}

template <template <int, bool> class F>
cudaError_t by_format(const QuantArgs& a) {
    if (a.d == 64) return a.fp4 ? F<64, true>::go(a) : F<64, false>::go(a);
    return a.fp4 ? F<128, true>::go(a) : F<128, false>::go(a);
}

template <int D, bool kFp4>
struct AppendLaunch {
    static cudaError_t go(const QuantArgs& a) {
        dim3 grid;
        const cudaError_t e = grid_of(32LL * a.num_tokens * (2 * a.hkv + (a.q ? a.hq : 0)), &grid);
        return e != cudaSuccess ? e : launch_pdl(quant_append_kernel<D, kFp4>, grid, dim3(256), 0, a.stream, a);
    }
};
template <int D, bool kFp4>
struct ReadLaunch {
    static cudaError_t go(const QuantArgs& a) {
        dim3 grid;
        const cudaError_t e = grid_of(static_cast<long long>(a.num_tokens) * a.hkv * D, &grid);
        return e != cudaSuccess ? e : launch_pdl(quant_read_kernel<D, kFp4>, grid, dim3(256), 0, a.stream, a);
    }
};
template <int D, bool kFp4>
struct LoadLaunch {
    static cudaError_t go(const QuantArgs& a) {
        return launch_pdl(quant_load_kernel<D, kFp4>, dim3(a.num_tokens, a.hkv, 2), dim3(256), 0, a.stream, a);
    }
};

}  // namespace

int quant_record_bytes(int d, int fp4) {
    if (d == 64) return fp4 ? QuantRecord<64, true>::kBytes : QuantRecord<64, false>::kBytes;
    return fp4 ? QuantRecord<128, true>::kBytes : QuantRecord<128, false>::kBytes;
}

cudaError_t launch_rope_rotate(const RotateArgs& a, cudaStream_t stream) {
    dim3 grid;
    const cudaError_t e = grid_of(static_cast<long long>(a.num_tokens) * (a.q.num_heads + a.k.num_heads) *
                                      (a.d - a.rotary / 2), &grid);
    if (e != cudaSuccess) return e;
    switch (a.dtype) {
        case PKV_BF16: return launch_pdl(rope_rotate_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, a);
        case PKV_F16: return launch_pdl(rope_rotate_kernel<__half>, grid, dim3(256), 0, stream, a);
        default: return launch_pdl(rope_rotate_kernel<float>, grid, dim3(256), 0, stream, a);
    }
}

cudaError_t launch_quant_append(const QuantArgs& a) { return by_format<AppendLaunch>(a); }
cudaError_t launch_quant_read(const QuantArgs& a) { return by_format<ReadLaunch>(a); }
cudaError_t launch_quant_load(const QuantArgs& a) { return by_format<LoadLaunch>(a); }

}  // namespace pkv
