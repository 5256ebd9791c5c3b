// rope_quant.cu -- rotary positions in both pair layouts, and the quantised
// pools' append, row read and block widening (formats: include/pkv.h).
//
// All four move bytes: each lane handles 16 bytes of 16-bit values (8 dims) at a
// time, so that a warp's loads and stores of a row are whole lines, and several
// rows per thread, all loads ahead of the first use, so that enough bytes are in
// flight.  The rotation's (cos, sin) pairs are read once per thread and used for
// all of its rows.
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace pkv {

namespace {

// ---------------------------------------------------------- conversions --

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

// The 16 / sizeof(T) elements of a 16-byte vector.
template <typename T, int N>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[N]) {
    static_assert(N * sizeof(T) == 16, "one vector");
    const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(e[i]);
}
template <typename T, int N>
__device__ __forceinline__ uint4 pack(const float (&x)[N]) {
    uint4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = from_f32<T>(x[i]);
    return v;
}

// x' = (a c - b s, b c + a s), each op rounded
__device__ __forceinline__ float2 turn(float a, float b, float c, float s) {
    return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

// ------------------------------------------------------------- rotation --
//
// Rows by strides.  A thread takes one vector position of kRows heads of a token:
// with half-split pairs the vectors at j and j + r/2, with interleaved pairs one
// vector; positions past the rotary dims copy a vector (out of place only).

struct RotateRow {
    const uint8_t* in;
    uint8_t* out;
};

template <typename T>
__device__ __forceinline__ RotateRow rotate_row(const RotateArgs& a, long long i, int h) {
    const bool is_k = h >= a.q.num_heads;
    const RotateRows& r = is_k ? a.k : a.q;
    if (is_k) h -= a.q.num_heads;
    return RotateRow{static_cast<const uint8_t*>(r.in) + (i * r.in_token + h * r.in_head) * static_cast<long long>(sizeof(T)),
                     static_cast<uint8_t*>(r.out) + (i * r.out_token + h * r.out_head) * static_cast<long long>(sizeof(T))};
}

template <typename T, bool kHalf, int kRows>
__global__ void __launch_bounds__(256) rope_vector_kernel(RotateArgs a, int vectors, int slots, int first_token) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int N = 16 / sizeof(T);
    constexpr int kPairs = kHalf ? N : N / 2;
    const unsigned idx = blockIdx.x * 256u + threadIdx.x;
    const int v = static_cast<int>(idx % vectors);
    const unsigned rest = idx / vectors;
    const int slot = static_cast<int>(rest % slots);
    const long long i = first_token + static_cast<long long>(rest / slots);
    if (i >= a.num_tokens) return;
    const int heads = a.q.num_heads + a.k.num_heads;
    const int h0 = slot * kRows;
    const int half = a.rotary / 2;
    const int turns = kHalf ? half / N : a.rotary / N;  // vector positions that rotate
    const bool pass = v >= turns;
    // the rows' loads do not wait for the position's
    uint4 x[kRows], y[kHalf ? kRows : 1];
    const int at = pass ? (a.rotary + (v - turns) * N) * static_cast<int>(sizeof(T)) : v * 16;
    const int mate = at + half * static_cast<int>(sizeof(T));
    const int p = a.positions[i];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (h0 + r < heads) {
            const RotateRow row = rotate_row<T>(a, i, h0 + r);
            x[r] = *reinterpret_cast<const uint4*>(row.in + at);
            if constexpr (kHalf)
                if (!pass) y[r] = *reinterpret_cast<const uint4*>(row.in + mate);
        }
    if (p < 0) return;
    if (p >= a.max_pos) {
        if (v == 0 && slot == 0) flag_error(a.err, PKV_DEVERR_POSITION);
        return;
    }
    if (pass) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (h0 + r < heads) *reinterpret_cast<uint4*>(rotate_row<T>(a, i, h0 + r).out + at) = x[r];
        return;
    }
    float c[kPairs], s[kPairs];
    const float4* cs = reinterpret_cast<const float4*>(a.cos_sin + (static_cast<size_t>(p) * half + v * kPairs) * 2);
#pragma unroll
    for (int j = 0; j < kPairs; j += 2) {
        const float4 t = cs[j / 2];
        c[j] = t.x;
        s[j] = a.inverse ? -t.y : t.y;
        c[j + 1] = t.z;
        s[j + 1] = a.inverse ? -t.w : t.w;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (h0 + r < heads) {
            const RotateRow row = rotate_row<T>(a, i, h0 + r);
            float f[N];
            unpack<T>(x[r], f);
            if constexpr (kHalf) {
                float g[N];
                unpack<T>(y[r], g);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float2 z = turn(f[j], g[j], c[j], s[j]);
                    f[j] = z.x;
                    g[j] = z.y;
                }
                *reinterpret_cast<uint4*>(row.out + mate) = pack<T>(g);
            } else {
#pragma unroll
                for (int j = 0; j < N; j += 2) {
                    const float2 z = turn(f[j], f[j + 1], c[j / 2], s[j / 2]);
                    f[j] = z.x;
                    f[j + 1] = z.y;
                }
            }
            *reinterpret_cast<uint4*>(row.out + at) = pack<T>(f);
        }
}

// Rows that no 16-byte vector fits (their address, stride, rotary or head dims):
// one thread per (token, head, pair or passing element).
template <typename T>
__global__ void __launch_bounds__(256) rope_scalar_kernel(RotateArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int half = a.rotary / 2;
    const int items = a.d - half;  // pairs, then the dims that pass
    const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int it = static_cast<int>(idx % items);
    const long long row = idx / items;
    const int heads = a.q.num_heads + a.k.num_heads;
    const long long i = row / heads;
    if (i >= a.num_tokens) return;
    const int p = a.positions[i];
    if (p < 0) return;
    if (p >= a.max_pos) {
        if (it == 0) flag_error(a.err, PKV_DEVERR_POSITION);
        return;
    }
    const RotateRow r = rotate_row<T>(a, i, static_cast<int>(row % heads));
    const T* in = reinterpret_cast<const T*>(r.in);
    T* out = reinterpret_cast<T*>(r.out);
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
// D/8 lanes per row, 8 dims each; rows are the Hq query heads, the Hkv K heads
// and the Hkv V heads of a token, kRows consecutive ones per thread.

// The block and slot of position p of sequence s: false for padding and for a bad position or
// block id (flagged by `report`).
__device__ __forceinline__ bool quant_slot(const QuantArgs& a, int s, int p, bool report, int* blk, int* row) {
    if (s < 0) return false;
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

// 8 dims of a K or V row (dims 8 lane .. 8 lane + 7 of the row's lanes) into its record.
template <int D, bool kFp4>
__device__ __forceinline__ void store_row(uint8_t* rec, int row, int lane, const float (&v)[8], float g, bool ok) {
    using R = QuantRecord<D, kFp4>;
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite_magnitude(v[e]));
    if constexpr (kFp4) {
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        const uint32_t sc = fp4_scale_code(amax, g);
        const float t = __fmul_rn(e4m3_float(sc), g);
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; e += 2) w |= fp4_pair(fp4_quotient(v[e], t), fp4_quotient(v[e + 1], t)) << (4 * e);
        if (ok) {
            *reinterpret_cast<uint32_t*>(rec + quant_byte<R::kRowBytes>(row, 4 * lane)) = w;
            if (!(lane & 1)) rec[R::kScales + row * R::kScaleBytes + lane / 2] = static_cast<uint8_t>(sc);
        }
    } else {
#pragma unroll
        for (int o = 1; o < D / 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const float sc = __fdiv_rn(amax, 127.f);
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e / 4] |= int8_code(v[e], sc) << (8 * (e % 4));
        if (ok) {
            *reinterpret_cast<uint2*>(rec + quant_byte<R::kRowBytes>(row, 8 * lane)) = make_uint2(w[0], w[1]);
            if (lane == 0) *reinterpret_cast<float*>(rec + R::kScales + row * 4) = sc;
        }
    }
}

// How a row's pairs are found: any rotary dim element by element (or none), or
// every lane's 8 dims inside the rotary dims or outside them, their partners in one
// vector (half-split, r a multiple of 16) or in the lane (interleaved, r of 8).
enum Pairs { kAnyPairs, kHalfPairs, kLanePairs };

template <int D, bool kFp4, int kRows, int kPairs>
__global__ void __launch_bounds__(256) quant_append_kernel(QuantArgs a, int slots) {
    pdl_wait();
    pdl_launch_dependents();
    using R = QuantRecord<D, kFp4>;
    constexpr int kLanes = D / 8;
    const int lane = threadIdx.x % kLanes;
    const long long group = static_cast<long long>(blockIdx.x) * (256 / kLanes) + threadIdx.x / kLanes;
    const long long i = group / slots;
    const int r0 = static_cast<int>(group % slots) * kRows;
    const int hq = a.q ? a.hq : 0;
    const int turned = hq + a.hkv;  // rows that rotate
    const int rows = turned + a.hkv;
    const int d0 = 8 * lane;
    const int half = a.rotary / 2;
    const bool rope = a.cos_sin != nullptr && d0 < a.rotary;
    const bool second = kPairs == kHalfPairs && d0 >= half;
    auto source = [&](int r) {
        return r < hq ? static_cast<const __nv_bfloat16*>(a.q) + i * a.q_stride + static_cast<size_t>(r) * D
               : r < turned ? static_cast<const __nv_bfloat16*>(a.k_new) + i * a.new_stride + static_cast<size_t>(r - hq) * D
                            : static_cast<const __nv_bfloat16*>(a.v_new) + i * a.new_stride + static_cast<size_t>(r - turned) * D;
    };
    // the rows' loads do not wait for the token's slot.  Every lane stays to the
    // end: rows share shuffles with their warp.
    uint4 x[kRows], y[kPairs == kHalfPairs ? kRows : 1];
    const bool in = i < a.num_tokens;
    int s = -1, p = 0;
    if (in) {
        s = a.token_to_seq[i];
        p = a.positions[i];
    }
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        x[n] = make_uint4(0u, 0u, 0u, 0u);
        if (in && r0 + n < rows) {
            const __nv_bfloat16* src = source(r0 + n);
            x[n] = *reinterpret_cast<const uint4*>(src + d0);
            if constexpr (kPairs == kHalfPairs)
                if (rope && r0 + n < turned) y[n] = *reinterpret_cast<const uint4*>(src + (second ? d0 - half : d0 + half));
        }
    }
    int blk = 0, row = 0;
    const bool ok = in && quant_slot(a, s, p, lane == 0 && r0 == 0, &blk, &row);
    // (cos, sin) of this lane's dims
    constexpr int kCs = kPairs == kLanePairs ? 4 : 8;
    float c[kCs], sn[kCs];
    if (ok && rope && r0 < turned) {
        const float* cs = a.cos_sin + static_cast<size_t>(p) * a.rotary;
        if constexpr (kPairs == kAnyPairs) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = d0 + e;
                if (d >= a.rotary) continue;
                const float2 t = *reinterpret_cast<const float2*>(cs + 2 * (a.interleaved ? d >> 1 : d < half ? d : d - half));
                c[e] = t.x;
                sn[e] = t.y;
            }
        } else {
            const float4* t4 = reinterpret_cast<const float4*>(cs + (kPairs == kLanePairs ? d0 : 2 * (second ? d0 - half : d0)));
#pragma unroll
            for (int e = 0; e < kCs; e += 2) {
                const float4 t = t4[e / 2];
                c[e] = t.x;
                sn[e] = t.y;
                c[e + 1] = t.z;
                sn[e + 1] = t.w;
            }
        }
        if (a.inverse) {
#pragma unroll
            for (int e = 0; e < kCs; ++e) sn[e] = -sn[e];
        }
    }
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        const int r = r0 + n;
        const bool live = ok && r < rows;
        float v[8];
        unpack<__nv_bfloat16>(x[n], v);
        if (live && rope && r < turned) {
            if constexpr (kPairs == kLanePairs) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 z = turn(v[e], v[e + 1], c[e / 2], sn[e / 2]);
                    v[e] = z.x;
                    v[e + 1] = z.y;
                }
            } else if constexpr (kPairs == kHalfPairs) {
                float m[8];
                unpack<__nv_bfloat16>(y[n], m);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = second ? turn(m[e], v[e], c[e], sn[e]).y : turn(v[e], m[e], c[e], sn[e]).x;
            } else {
                const __nv_bfloat16* src = source(r);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int d = d0 + e;
                    if (d >= a.rotary) continue;
                    const bool b = a.interleaved ? d & 1 : d >= half;
                    const float m = __bfloat162float(src[a.interleaved ? d ^ 1 : b ? d - half : d + half]);
                    v[e] = b ? turn(m, v[e], c[e], sn[e]).y : turn(v[e], m, c[e], sn[e]).x;
                }
            }
        }
        __syncwarp();  // q in place: the row's lanes have read their pairs
        if (live && r < hq) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.q_out) + i * a.q_out_stride + static_cast<size_t>(r) * D +
                                      d0) = pack<__nv_bfloat16>(v);
        }
        // a warp's rows may be of different kinds: the shuffles below are for all
        // of them, the stores for K and V rows
        const bool kv = live && r >= hq;
        if (__any_sync(0xFFFFFFFFu, kv)) {
            const bool is_k = r < turned;
            const int h = is_k ? r - hq : r - turned;
            uint8_t* rec = nullptr;
            float g = 1.f;
            if (kv) {
                rec = static_cast<uint8_t*>(is_k ? a.k_pool : a.v_pool) + (static_cast<size_t>(blk) * a.hkv + h) * R::kBytes;
                if constexpr (kFp4) g = (is_k ? a.k_scale : a.v_scale)[h];
            }
            store_row<D, kFp4>(rec, row, lane, v, g, kv);
        }
    }
}

// ----------------------------------------------------------------- read --

// 8 values of a record's row (dims 8 lane ..), each rounded to fp32 once.
template <int D, bool kFp4>
struct RowPart {
    uint2 codes;  // 4-bit: codes.x
    float scale;
};

template <int D, bool kFp4>
__device__ __forceinline__ RowPart<D, kFp4> fetch_row(const uint8_t* rec, int row, int lane) {
    using R = QuantRecord<D, kFp4>;
    RowPart<D, kFp4> p;
    if constexpr (kFp4) {
        p.codes.x = *reinterpret_cast<const uint32_t*>(rec + quant_byte<R::kRowBytes>(row, 4 * lane));
        p.scale = __uint_as_float(rec[R::kScales + row * R::kScaleBytes + lane / 2]);  // its code, widened below
    } else {
        p.codes = *reinterpret_cast<const uint2*>(rec + quant_byte<R::kRowBytes>(row, 8 * lane));
        p.scale = *reinterpret_cast<const float*>(rec + R::kScales + row * 4);
    }
    return p;
}

template <int D, bool kFp4>
__device__ __forceinline__ void widen_row(const RowPart<D, kFp4>& p, float g, float (&v)[8]) {
    if constexpr (kFp4) {
        const float e = e4m3_float(__float_as_uint(p.scale));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t f = fp4x2_to_f16x2((p.codes.x >> (8 * i)) & 0xFFu);
            const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&f));
            v[2 * i] = __fmul_rn(z.x * e, g);
            v[2 * i + 1] = __fmul_rn(z.y * e, g);
        }
    } else {
        (void)g;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t u = ((i < 4 ? p.codes.x : p.codes.y) >> (8 * (i % 4))) & 0xFFu;
            v[i] = __fmul_rn(static_cast<float>(u) - 128.f, p.scale);
        }
    }
}

// D/8 lanes per (token, head), K and V of it in one thread.
template <int D, bool kFp4>
__global__ void __launch_bounds__(256) quant_read_kernel(QuantArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kLanes = D / 8;
    const int lane = threadIdx.x % kLanes;
    const long long group = static_cast<long long>(blockIdx.x) * (256 / kLanes) + threadIdx.x / kLanes;
    const long long i = group / a.hkv;
    const int h = static_cast<int>(group % a.hkv);
    if (i >= a.num_tokens) return;
    int blk, row;
    if (!quant_slot(a, a.token_to_seq[i], a.positions[i], lane == 0 && h == 0, &blk, &row)) return;
    const size_t at = (static_cast<size_t>(blk) * a.hkv + h) * QuantRecord<D, kFp4>::kBytes;
    RowPart<D, kFp4> part[2];
#pragma unroll
    for (int pool = 0; pool < 2; ++pool)
        if (pool ? a.v_out : a.k_out)
            part[pool] = fetch_row<D, kFp4>(static_cast<const uint8_t*>(pool ? a.v_pool : a.k_pool) + at, row, lane);
    const size_t to = (static_cast<size_t>(i) * a.hkv + h) * D + 8 * lane;
#pragma unroll
    for (int pool = 0; pool < 2; ++pool) {
        void* dst = pool ? a.v_out : a.k_out;
        if (!dst) continue;
        float v[8];
        widen_row<D, kFp4>(part[pool], kFp4 ? (pool ? a.v_scale : a.k_scale)[h] : 1.f, v);
        if (a.out_f32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(dst) + to);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst) + to) = pack<__nv_bfloat16>(v);
        }
    }
}

// A CTA per (pair, kHeads heads): thread (row, lane) widens 8 dims of each of
// their records, K and V.
template <int D, bool kFp4, int kHeads>
__global__ void __launch_bounds__(2 * D) quant_load_kernel(QuantArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kLanes = D / 8;
    const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
    const int src = a.src_blocks[blockIdx.x], dst = a.dst_blocks[blockIdx.x];
    if (src < 0 || src >= a.num_blocks || dst < 0 || dst >= a.dst_num_blocks) {
        if (threadIdx.x == 0) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
        return;
    }
    const int h0 = blockIdx.y * kHeads;
    RowPart<D, kFp4> part[2][kHeads];
#pragma unroll
    for (int n = 0; n < kHeads; ++n)
#pragma unroll
        for (int pool = 0; pool < 2; ++pool)
            if (h0 + n < a.hkv)
                part[pool][n] = fetch_row<D, kFp4>(static_cast<const uint8_t*>(pool ? a.v_pool : a.k_pool) +
                                                       (static_cast<size_t>(src) * a.hkv + h0 + n) * QuantRecord<D, kFp4>::kBytes,
                                                   row, lane);
#pragma unroll
    for (int n = 0; n < kHeads; ++n)
#pragma unroll
        for (int pool = 0; pool < 2; ++pool)
            if (h0 + n < a.hkv) {
                float v[8];
                widen_row<D, kFp4>(part[pool][n], kFp4 ? (pool ? a.v_scale : a.k_scale)[h0 + n] : 1.f, v);
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(pool ? a.v_out : a.k_out) +
                                     ((static_cast<size_t>(dst) * a.hkv + h0 + n) * kBlockSize + row) * D + 8 * lane;
                *reinterpret_cast<uint4*>(out) = pack<__nv_bfloat16>(v);
            }
}

// ------------------------------------------------------------- launches --

cudaError_t grid_of(long long threads, dim3* grid) {
    const long long blocks = (threads + 255) / 256;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    *grid = dim3(static_cast<unsigned>(blocks));
    return cudaSuccess;
}

constexpr long long kBusyThreads = 152LL * 512;  // 16 warps an SM: enough to give a thread more rows

template <template <int, bool> class F>
cudaError_t by_format(const QuantArgs& a) {
    if (a.d == 64) return a.fp4 ? F<64, true>::go(a) : F<64, false>::go(a);
    return a.fp4 ? F<128, true>::go(a) : F<128, false>::go(a);
}

template <int D, bool kFp4>
struct AppendLaunch {
    template <int kRows, int kPairs>
    static cudaError_t rows(const QuantArgs& a, int rows) {
        const int slots = (rows + kRows - 1) / kRows;
        dim3 grid;
        const cudaError_t e = grid_of(static_cast<long long>(a.num_tokens) * slots * (D / 8), &grid);
        return e != cudaSuccess ? e
                                : launch_pdl(quant_append_kernel<D, kFp4, kRows, kPairs>, grid, dim3(256), 0, a.stream, a, slots);
    }
    template <int kPairs>
    static cudaError_t pairs(const QuantArgs& a) {
        const int n = 2 * a.hkv + (a.q ? a.hq : 0);
        return static_cast<long long>(a.num_tokens) * n * (D / 8) >= 4 * kBusyThreads ? rows<2, kPairs>(a, n) : rows<1, kPairs>(a, n);
    }
    static cudaError_t go(const QuantArgs& a) {
        if (a.cos_sin && reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0) {
            if (!a.interleaved && a.rotary % 16 == 0) return pairs<kHalfPairs>(a);
            if (a.interleaved && a.rotary % 8 == 0) return pairs<kLanePairs>(a);
        }
        return pairs<kAnyPairs>(a);
    }
};
template <int D, bool kFp4>
struct ReadLaunch {
    static cudaError_t go(const QuantArgs& a) {
        dim3 grid;
        const cudaError_t e = grid_of(static_cast<long long>(a.num_tokens) * a.hkv * (D / 8), &grid);
        return e != cudaSuccess ? e : launch_pdl(quant_read_kernel<D, kFp4>, grid, dim3(256), 0, a.stream, a);
    }
};
template <int D, bool kFp4>
struct LoadLaunch {
    static cudaError_t go(const QuantArgs& a) {
        if (static_cast<long long>(a.num_tokens) * a.hkv * 2 * D >= 16 * kBusyThreads)
            return launch_pdl(quant_load_kernel<D, kFp4, 4>, dim3(a.num_tokens, (a.hkv + 3) / 4), dim3(2 * D), 0, a.stream, a);
        return launch_pdl(quant_load_kernel<D, kFp4, 1>, dim3(a.num_tokens, a.hkv), dim3(2 * D), 0, a.stream, a);
    }
};

template <typename T>
struct RotateLaunch {
    static bool vectors_fit(const RotateArgs& a) {
        constexpr int N = 16 / sizeof(T);
        auto rows = [](const RotateRows& r) {
            return r.num_heads == 0 ||
                   ((reinterpret_cast<uintptr_t>(r.in) | reinterpret_cast<uintptr_t>(r.out)) % 16 == 0 &&
                    (r.in_token | r.in_head | r.out_token | r.out_head) % N == 0);
        };
        return a.d % N == 0 && a.rotary % (a.interleaved ? N : 2 * N) == 0 &&
               reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0 && rows(a.q) && rows(a.k);
    }
    template <bool kHalf, int kRows>
    static cudaError_t vectors(const RotateArgs& a, int count, cudaStream_t stream) {
        const int slots = (a.q.num_heads + a.k.num_heads + kRows - 1) / kRows;
        const long long per_token = static_cast<long long>(count) * slots;
        const long long most = (0xFFFFFFFFLL - 256) / per_token;  // thread indexes are 32 bits wide
        for (long long i = 0; i < a.num_tokens; i += most) {
            const long long n = a.num_tokens - i < most ? a.num_tokens - i : most;
            const cudaError_t e = launch_pdl(rope_vector_kernel<T, kHalf, kRows>, dim3(static_cast<unsigned>((n * per_token + 255) / 256)),
                                             dim3(256), 0, stream, a, count, slots, static_cast<int>(i));
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    template <bool kHalf>
    static cudaError_t by_rows(const RotateArgs& a, cudaStream_t stream) {
        constexpr int N = 16 / sizeof(T);
        // in place nothing passes (with one of q and k in place, its passing dims
        // are written back as they are: the same bytes, by the thread that read them)
        const bool in_place = a.q.in == a.q.out && (a.k.num_heads == 0 || a.k.in == a.k.out);
        const int count = (kHalf ? a.rotary / 2 : a.rotary) / N + (in_place ? 0 : (a.d - a.rotary) / N);
        const long long one = static_cast<long long>(a.num_tokens) * (a.q.num_heads + a.k.num_heads) * count;
        if (one >= 4 * kBusyThreads) return vectors<kHalf, kHalf ? 4 : 8>(a, count, stream);
        return vectors<kHalf, 1>(a, count, stream);
    }
    static cudaError_t go(const RotateArgs& a, cudaStream_t stream) {
        if (vectors_fit(a)) return a.interleaved ? by_rows<false>(a, stream) : by_rows<true>(a, stream);
        dim3 grid;
        const cudaError_t e = grid_of(static_cast<long long>(a.num_tokens) * (a.q.num_heads + a.k.num_heads) *
                                          (a.d - a.rotary / 2), &grid);
        return e != cudaSuccess ? e : launch_pdl(rope_scalar_kernel<T>, grid, dim3(256), 0, stream, a);
    }
};

}  // namespace

int quant_record_bytes(int d, int fp4) {
    if (d == 64) return fp4 ? QuantRecord<64, true>::kBytes : QuantRecord<64, false>::kBytes;
    return fp4 ? QuantRecord<128, true>::kBytes : QuantRecord<128, false>::kBytes;
}

cudaError_t launch_rope_rotate(const RotateArgs& a, cudaStream_t stream) {
    switch (a.dtype) {
        case PKV_BF16: return RotateLaunch<__nv_bfloat16>::go(a, stream);
        case PKV_F16: return RotateLaunch<__half>::go(a, stream);
        default: return RotateLaunch<float>::go(a, stream);
    }
}

cudaError_t launch_quant_append(const QuantArgs& a) { return by_format<AppendLaunch>(a); }
cudaError_t launch_quant_read(const QuantArgs& a) { return by_format<ReadLaunch>(a); }
cudaError_t launch_quant_load(const QuantArgs& a) { return by_format<LoadLaunch>(a); }

}  // namespace pkv
