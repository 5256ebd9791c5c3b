// rope_quant.cu -- rotary positions in both pair layouts, and the quantised
// pools' append, row read and block widening (formats: include/pkv.h).
//
// All four move bytes, and a call is short: one to three waves of blocks whose loads
// depend on one another twice (the position, then its table entry or block).  So a lane
// handles 16 bytes of 16-bit values (8 dims) at a time, a warp's loads and stores of a row
// being whole lines; the rows are loaded before the position is waited for; where there
// are many rows a thread of the rotation takes four, whose (cos, sin) it reads once; and
// blocks are small, so that the last wave is.
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace pkv {

namespace {

constexpr int kRopeThreads = 64, kAppendThreads = 128;

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

// Whether position p of sequence s has a table entry.
__device__ __forceinline__ bool token_in_table(int s, int p, int num_seqs, int mbps, int ring) {
    const int tb = ring > 0 ? (p / kBlockSize) % ring : p / kBlockSize;
    return s >= 0 && s < num_seqs && p >= 0 && tb < mbps;
}

// ------------------------------------------------------------- rotation --
//
// Rows by strides.  A thread takes one vector position of kRows heads of a token, all of
// q or all of k: with half-split pairs the vectors at j and j + r/2, with interleaved
// pairs one vector; positions past the rotary dims copy a vector (out of place only).
// It moves each byte once, so HBM bounds it; what it fights is the address arithmetic (one
// base per thread, then the head stride) and latency (kRows vectors in flight before
// anything waits, the position among them).  4096 tokens of 32 + 8 heads of 128, in place in
// a packed buffer (84 MB), from a replayed graph: 15.3 us, 5.6 TB/s; 16.0 in blocks of 256
// threads, 17.8 with a head a thread, 16.5 with two.

template <typename T, bool kHalf, int kRows>
__device__ __forceinline__ void rotate_vectors(const RotateArgs& a, unsigned idx, unsigned vectors, unsigned q_slots,
                                               unsigned slots, int first_token) {
    constexpr int N = 16 / sizeof(T);
    constexpr int kPairs = kHalf ? N : N / 2;
    const unsigned rest = idx / vectors, v = idx - rest * vectors;
    const unsigned token = rest / slots;
    unsigned slot = rest - token * slots;
    const long long i = first_token + static_cast<long long>(token);
    if (i >= a.num_tokens) return;
    const bool is_k = slot >= q_slots;
    if (is_k) slot -= q_slots;
    const int h0 = static_cast<int>(slot) * kRows;
    const int rows = min(kRows, (is_k ? a.k.num_heads : a.q.num_heads) - h0);
    const int64_t in_head = is_k ? a.k.in_head : a.q.in_head, out_head = is_k ? a.k.out_head : a.q.out_head;
    const int half = a.rotary / 2;
    const unsigned turns = static_cast<unsigned>(kHalf ? half : a.rotary) / N;  // vector positions that rotate
    const bool pass = v >= turns;
    const int at = pass ? a.rotary + static_cast<int>(v - turns) * N : static_cast<int>(v) * N;
    const T* in = static_cast<const T*>(is_k ? a.k.in : a.q.in) + i * (is_k ? a.k.in_token : a.q.in_token) + h0 * in_head + at;
    T* out = static_cast<T*>(is_k ? a.k.out : a.q.out) + i * (is_k ? a.k.out_token : a.q.out_token) + h0 * out_head + at;
    // the rows' loads do not wait for the position's
    uint4 x[kRows], y[kHalf ? kRows : 1];
    const int p = a.positions[i];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (r < rows) {
            x[r] = *reinterpret_cast<const uint4*>(in + r * in_head);
            if constexpr (kHalf)
                if (!pass) y[r] = *reinterpret_cast<const uint4*>(in + r * in_head + half);
        }
    if (p < 0) return;
    if (p >= a.max_pos) {
        if (v == 0 && h0 == 0) flag_error(a.err, PKV_DEVERR_POSITION);
        return;
    }
    if (a.token_to_seq && !token_in_table(a.token_to_seq[i], p, a.num_seqs, a.mbps, a.ring)) return;
    if (pass) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (r < rows) *reinterpret_cast<uint4*>(out + r * out_head) = x[r];
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
        if (r < rows) {
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
                *reinterpret_cast<uint4*>(out + r * out_head + half) = pack<T>(g);
            } else {
#pragma unroll
                for (int j = 0; j < N; j += 2) {
                    const float2 z = turn(f[j], f[j + 1], c[j / 2], s[j / 2]);
                    f[j] = z.x;
                    f[j + 1] = z.y;
                }
            }
            *reinterpret_cast<uint4*>(out + r * out_head) = pack<T>(f);
        }
}

template <typename T, bool kHalf, int kRows>
__global__ void __launch_bounds__(kRopeThreads, 16) rope_vector_kernel(const __grid_constant__ RotateArgs a, unsigned vectors,
                                                          unsigned q_slots, unsigned slots, int first_token) {
    pdl_wait();
    pdl_launch_dependents();
    rotate_vectors<T, kHalf, kRows>(a, blockIdx.x * kRopeThreads + threadIdx.x, vectors, q_slots, slots, first_token);
}

// The warps of rotate_partial: those that turn, then those that copy.
struct PartialWarps {
    unsigned lanes;  // vectors of a row that hold rotary dims
    unsigned turning, all;
};

// Rows of vectors whose rotary dims are not: the first `turning` warps turn the vectors
// that hold rotary dims, `lanes` a row, a row's lanes in one warp (32 / lanes units of kRows
// heads), each looking its elements' partners up in the row -- with interleaved pairs they
// are its own -- before any lane of the warp stores, so that in place is safe.  The other
// warps copy the vectors that pass whole (out of place only).
// 9265 tokens of 8 + 4 heads of 64, 18 dims turning, out of place (28 MB, 4.3 us of HBM): 6.3 us
// interleaved; half-split 9.2, bound by the lookups of partners, 12.0 with the passing
// vectors' lanes in the turning warps, 12.9 with partners from shuffles, 36.6 with a thread
// per pair and per passing element.
template <typename T, int kRows>
__device__ __forceinline__ void rotate_partial(const RotateArgs& a, unsigned warp, const PartialWarps& w, unsigned q_slots,
                                               unsigned slots, int first_token) {
    constexpr int N = 16 / sizeof(T);
    if (warp >= w.all) return;
    const unsigned lane = threadIdx.x % 32u, lanes = w.lanes;
    const bool turns = warp < w.turning;
    unsigned rest, v;  // the unit, and the vector of its rows
    bool live = true;
    if (turns) {
        const unsigned units = 32u / lanes, unit = lane / lanes;
        live = unit < units;
        rest = warp * units + unit;
        v = lane - unit * lanes;
    } else {
        const unsigned passing = static_cast<unsigned>(a.d) / N - lanes, idx = (warp - w.turning) * 32u + lane;
        rest = idx / passing;
        v = lanes + idx - rest * passing;
    }
    const unsigned token = rest / slots;
    unsigned slot = rest - token * slots;
    const long long i = first_token + static_cast<long long>(token);
    const bool is_k = slot >= q_slots;
    if (is_k) slot -= q_slots;
    const int h0 = static_cast<int>(slot) * kRows, d0 = static_cast<int>(v) * N;
    const int rows = live && i < a.num_tokens ? min(kRows, (is_k ? a.k.num_heads : a.q.num_heads) - h0) : 0;
    const int64_t in_head = is_k ? a.k.in_head : a.q.in_head, out_head = is_k ? a.k.out_head : a.q.out_head;
    const T* in = static_cast<const T*>(is_k ? a.k.in : a.q.in) + i * (is_k ? a.k.in_token : a.q.in_token) + h0 * in_head;
    uint4 x[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (r < rows) x[r] = *reinterpret_cast<const uint4*>(in + r * in_head + d0);
    int p = -1;
    if (rows > 0) p = a.positions[i];
    bool ok = p >= 0;
    if (ok && p >= a.max_pos) {
        if (d0 == 0 && h0 == 0) flag_error(a.err, PKV_DEVERR_POSITION);
        ok = false;
    }
    if (ok && a.token_to_seq) ok = token_in_table(a.token_to_seq[i], p, a.num_seqs, a.mbps, a.ring);
    if (turns) {
        if (ok) {
            const int half = a.rotary / 2;
            const float2* cs = reinterpret_cast<const float2*>(a.cos_sin) + static_cast<size_t>(p) * half;
            float2 t[N];
            T m[kRows][N];  // partners
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int n = d0 + e;
                if (n >= a.rotary) continue;
                if (a.interleaved) {
                    if (e % 2 == 0) t[e] = cs[n / 2];
                    continue;
                }
                t[e] = cs[n < half ? n : n - half];
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    if (r < rows) m[r][e] = in[r * in_head + (n < half ? n + half : n - half)];
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (r >= rows) break;
                T* f = reinterpret_cast<T*>(&x[r]);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const int n = d0 + e;
                    if (n >= a.rotary) continue;
                    if (a.interleaved) {
                        if (e % 2) continue;
                        const float2 z = turn(to_f32(f[e]), to_f32(f[e + 1]), t[e].x, a.inverse ? -t[e].y : t[e].y);
                        f[e] = from_f32<T>(z.x);
                        f[e + 1] = from_f32<T>(z.y);
                        continue;
                    }
                    // the first of a pair: own c - other s; the second: own c + other s
                    const float own = __fmul_rn(to_f32(f[e]), t[e].x), other = __fmul_rn(to_f32(m[r][e]), t[e].y);
                    f[e] = from_f32<T>(__fadd_rn(own, (n < half) != static_cast<bool>(a.inverse) ? -other : other));
                }
            }
        }
        __syncwarp();
    }
    if (!ok) return;
    T* out = static_cast<T*>(is_k ? a.k.out : a.q.out) + i * (is_k ? a.k.out_token : a.q.out_token) + h0 * out_head + d0;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (r < rows) *reinterpret_cast<uint4*>(out + r * out_head) = x[r];
}

// Of n elements a vector, for `units` groups of rows (the caller bounds them).
PartialWarps partial_warps(const RotateArgs& a, int n, bool in_place, long long units) {
    const long long lanes = (a.rotary + n - 1) / n, per_warp = 32 / lanes, passing = in_place ? 0 : a.d / n - lanes;
    const long long turning = (units + per_warp - 1) / per_warp;
    return PartialWarps{static_cast<unsigned>(lanes), static_cast<unsigned>(turning),
                        static_cast<unsigned>(turning + (units * passing + 31) / 32)};
}

template <typename T, int kRows>
__global__ void __launch_bounds__(kRopeThreads) rope_partial_kernel(const __grid_constant__ RotateArgs a, const PartialWarps w,
                                                                    unsigned q_slots, unsigned slots, int first_token) {
    pdl_wait();
    pdl_launch_dependents();
    rotate_partial<T, kRows>(a, (blockIdx.x * kRopeThreads + threadIdx.x) / 32u, w, q_slots, slots, first_token);
}

// Rows that start on no 16-byte boundary, are not whole vectors or are longer than a warp's:
// a thread takes kPairRun pairs of a row element by element, or 16 bytes of the dims that
// pass (out of place only), as one vector where `vec` says that rows allow it.
constexpr int kPairRun = 4;

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(const __grid_constant__ RotateArgs a, unsigned pair_items,
                                                                unsigned items, bool vec, int first_token) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int N = 16 / sizeof(T);
    const int half = a.rotary / 2;
    const unsigned idx = blockIdx.x * kRopeThreads + threadIdx.x, heads = a.q.num_heads + a.k.num_heads;
    const unsigned row = idx / items, it = idx - row * items, token = row / heads;
    int h = static_cast<int>(row - token * heads);
    const long long i = first_token + static_cast<long long>(token);
    if (i >= a.num_tokens) return;
    const int p = a.positions[i];
    if (p < 0) return;
    if (p >= a.max_pos) {
        if (it == 0 && h == 0) flag_error(a.err, PKV_DEVERR_POSITION);
        return;
    }
    const RotateRows& r = h >= a.q.num_heads ? a.k : a.q;
    if (h >= a.q.num_heads) h -= a.q.num_heads;
    const T* in = static_cast<const T*>(r.in) + i * r.in_token + h * r.in_head;
    T* out = static_cast<T*>(r.out) + i * r.out_token + h * r.out_head;
    if (it < pair_items) {
        const int j0 = static_cast<int>(it) * kPairRun, n = min(kPairRun, half - j0);
        const float2* cs = reinterpret_cast<const float2*>(a.cos_sin) + static_cast<size_t>(p) * half + j0;
        const int e0 = a.interleaved ? 2 * j0 : j0, step = a.interleaved ? 2 : 1, away = a.interleaved ? 1 : half;
        T x[kPairRun], y[kPairRun];
        float2 t[kPairRun];
#pragma unroll
        for (int u = 0; u < kPairRun; ++u)
            if (u < n) {
                x[u] = in[e0 + u * step];
                y[u] = in[e0 + u * step + away];
                t[u] = cs[u];
            }
#pragma unroll
        for (int u = 0; u < kPairRun; ++u)
            if (u < n) {
                const float2 z = turn(to_f32(x[u]), to_f32(y[u]), t[u].x, a.inverse ? -t[u].y : t[u].y);
                out[e0 + u * step] = from_f32<T>(z.x);
                out[e0 + u * step + away] = from_f32<T>(z.y);
            }
        return;
    }
    const int d0 = (a.rotary / N + static_cast<int>(it - pair_items)) * N;
    if (vec && d0 >= a.rotary) {
        *reinterpret_cast<uint4*>(out + d0) = *reinterpret_cast<const uint4*>(in + d0);
        return;
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (d0 + e >= a.rotary && d0 + e < a.d) out[d0 + e] = in[d0 + e];
}

// --------------------------------------------------------------- append --
//
// D/16 lanes per row, two vectors of 8 dims each: a rotation's pair of vectors where the
// pairs are half-split, so that every byte and every (cos, sin) is read once.
//
// Latency bounds it: a row waits for its token's position, then the block id, then goes
// through some 430 instructions per warp and 512 values that start from its largest
// magnitude.  At 43 % of an SM's warps 4.7 wait for a load at any issue, while the issue
// slots are 48 % busy, the ALU 44 %, DRAM 34 %.  K and V of 4096 tokens of 8 heads of 128
// (21 MB) take 8.8 us in a replayed graph where HBM would take 3.2, and with 32 rotated q
// heads (88 MB) 20 where it would take 13.0.  32 dims a lane, which halves the
// instructions, were tried when those took 9.8 and 20.4: 8.6 and 20.3, but K and V of 256
// tokens 3.1 us instead of 2.6, and 999 tokens of 64 + 8 heads of 64 5.8 instead of 4.3.

// The sequence and position of a token: false for padding and, flagged by `report`,
// for a bad one.
__device__ __forceinline__ bool quant_token(const QuantArgs& a, int s, int p, bool report) {
    if (s < 0) return false;
    if (token_in_table(s, p, a.num_seqs, a.mbps, a.ring) && (a.cos_sin == nullptr || p < a.max_pos)) return true;
    if (report) flag_error(a.err, PKV_DEVERR_POSITION);
    return false;
}

// The block id of a good token, and whether it is one.
__device__ __forceinline__ int quant_block(const QuantArgs& a, int s, int p) {
    const int tb = a.ring > 0 ? (p / kBlockSize) % a.ring : p / kBlockSize;
    return a.block_tables[static_cast<size_t>(s) * a.mbps + tb];
}
__device__ __forceinline__ bool good_block(const QuantArgs& a, int blk, bool report) {
    if (blk >= 0 && blk < a.num_blocks) return true;
    if (report) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
    return false;
}

// A lane's two vectors of a K or V row, dims 8 c0 .. and 8 c1 .., into its record.  split:
// the other half of each vector's 16 dims is in lane ^ 1; else c1 = c0 + 1 and they are
// the lane's own.
template <int D, bool kFp4>
__device__ __forceinline__ void store_row(uint8_t* rec, int row, int lane, int c0, int c1, bool split, const float (&v0)[8],
                                          const float (&v1)[8], float g, bool ok) {
    using R = QuantRecord<D, kFp4>;
    float m0 = 0.f, m1 = 0.f;  // over all but NaN
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        m0 = fmax3(m0, fabsf(v0[e]), fabsf(v0[e + 1]));
        m1 = fmax3(m1, fabsf(v1[e]), fabsf(v1[e + 1]));
    }
    if (__any_sync(0xFFFFFFFFu, fmaxf(m0, m1) == INFINITY)) {
        m0 = m1 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            m0 = fmaxf(m0, finite_magnitude(v0[e]));
            m1 = fmaxf(m1, finite_magnitude(v1[e]));
        }
    }
    float y0[8], y1[8];
    if constexpr (kFp4) {
        // a lane finds one scale: of its own 16 dims, or where they are split, an even lane that
        // of both c0 vectors and an odd one that of both c1
        const bool odd = lane & 1;
        const float theirs = __shfl_xor_sync(0xFFFFFFFFu, odd ? m0 : m1, 1);
        const uint32_t code = fp4_scale_code(split ? fmaxf(odd ? m1 : m0, theirs) : fmaxf(m0, m1), g);
        const float t = __fmul_rn(e4m3_float(code), g), r = divisor_reciprocal(t);
        const float other_t = __shfl_xor_sync(0xFFFFFFFFu, t, 1), other_r = __shfl_xor_sync(0xFFFFFFFFu, r, 1);
        quotients(v0, split && odd ? other_t : t, split && odd ? other_r : r, y0);
        quotients(v1, split && !odd ? other_t : t, split && !odd ? other_r : r, y1);
        uint32_t w0 = 0, w1 = 0;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            w0 |= fp4_pair(y0[e], y0[e + 1]) << (4 * e);
            w1 |= fp4_pair(y1[e], y1[e + 1]) << (4 * e);
        }
        if (ok) {
            *reinterpret_cast<uint32_t*>(rec + quant_byte<R::kRowBytes>(row, 4 * c0)) = w0;
            *reinterpret_cast<uint32_t*>(rec + quant_byte<R::kRowBytes>(row, 4 * c1)) = w1;
            rec[R::kScales + row * R::kScaleBytes + (split && odd ? c1 : c0) / 2] = static_cast<uint8_t>(code);
        }
    } else {
        float amax = fmaxf(m0, m1);
#pragma unroll
        for (int o = 1; o < D / 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const float sc = __fdiv_rn(amax, 127.f), r = divisor_reciprocal(sc);
        quotients(v0, sc, r, y0);
        quotients(v1, sc, r, y1);
        if (ok) {
            *reinterpret_cast<uint2*>(rec + quant_byte<R::kRowBytes>(row, 8 * c0)) = int8_codes(y0);
            *reinterpret_cast<uint2*>(rec + quant_byte<R::kRowBytes>(row, 8 * c1)) = int8_codes(y1);
            if (lane == 0) *reinterpret_cast<float*>(rec + R::kScales + row * 4) = sc;
        }
    }
}

// How a row's pairs are found: any rotary dim (or none) element by element; half-split
// with r a multiple of 32, a lane holding both vectors of its pairs; interleaved with r a
// multiple of 16, a lane's 16 dims all inside the rotary dims or all outside.
enum Pairs { kAnyPairs, kHalfPairs, kLanePairs };

template <int D, bool kFp4, int kPairs, int kThreads>
__device__ __forceinline__ void append_rows(const QuantArgs& a, unsigned block, int first_token) {
    using R = QuantRecord<D, kFp4>;
    constexpr int kLanes = D / 16;
    const int lane = threadIdx.x % kLanes;
    const unsigned group = block * (kThreads / kLanes) + threadIdx.x / kLanes, slots = 2u * static_cast<unsigned>(a.hkv);
    const unsigned token = group / slots, slot = group - token * slots;
    const long long i = first_token + static_cast<long long>(token);
    const bool is_v = slot >= static_cast<unsigned>(a.hkv), report = lane == 0 && slot == 0;
    const int h = static_cast<int>(is_v ? slot - a.hkv : slot);
    const int half = a.rotary / 2;
    // the lane's vectors
    const int turning = a.rotary / 16;  // lanes that rotate (vector paths)
    const bool split = kPairs == kHalfPairs && !is_v && lane < turning;
    const int c0 = split ? lane : 2 * lane, c1 = split ? lane + turning : c0 + 1;
    const bool rope = a.cos_sin != nullptr && !is_v && (kPairs == kAnyPairs ? 8 * c0 < a.rotary : lane < turning);
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? a.v_new : a.k_new) + i * a.new_stride + h * D;
    // the row's loads do not wait for the token's position, nor the rotation for its
    // block.  Every lane stays to the end: rows share shuffles with their warp.
    uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
    const bool in = i < a.num_tokens;
    int s = -1, p = 0;
    float g = 1.f;  // 4-bit: the head's scale
    if (in) {
        s = a.token_to_seq[i];
        p = a.positions[i];
        x0 = *reinterpret_cast<const uint4*>(src + 8 * c0);
        x1 = *reinterpret_cast<const uint4*>(src + 8 * c1);
        if (kFp4) g = (is_v ? a.v_scale : a.k_scale)[h];
    }
    const bool ok = in && quant_token(a, s, p, report);
    int blk = 0;  // looked at after the rotation, whose loads are then in flight beside it
    if (ok) blk = quant_block(a, s, p);
    // (cos, sin) of the lane's pairs: 8 on the vector paths (of c0 with c1, or of the 16
    // dims), else one per dim
    constexpr int kCs = kPairs == kAnyPairs ? 16 : 8;
    float c[kCs], sn[kCs];
    if (ok && rope) {
        const float* cs = a.cos_sin + static_cast<size_t>(p) * a.rotary;
        if constexpr (kPairs == kAnyPairs) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int d = 8 * c0 + e;
                if (d >= a.rotary) continue;
                if (a.interleaved && e % 2) continue;  // its pair's
                const float2 t = *reinterpret_cast<const float2*>(cs + 2 * (a.interleaved ? d >> 1 : d < half ? d : d - half));
                c[e] = t.x;
                sn[e] = t.y;
            }
        } else {
            const float4* t4 = reinterpret_cast<const float4*>(cs + 16 * lane);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
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
    float v0[8], v1[8];
    unpack<__nv_bfloat16>(x0, v0);
    unpack<__nv_bfloat16>(x1, v1);
    if (ok && rope) {
        if constexpr (kPairs == kHalfPairs) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 z = turn(v0[e], v1[e], c[e], sn[e]);
                v0[e] = z.x;
                v1[e] = z.y;
            }
        } else if constexpr (kPairs == kLanePairs) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 z0 = turn(v0[e], v0[e + 1], c[e / 2], sn[e / 2]);
                const float2 z1 = turn(v1[e], v1[e + 1], c[4 + e / 2], sn[4 + e / 2]);
                v0[e] = z0.x;
                v0[e + 1] = z0.y;
                v1[e] = z1.x;
                v1[e + 1] = z1.y;
            }
        } else if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                if (8 * c0 + e >= a.rotary) continue;
                float* v = e < 8 ? v0 + e : v1 + (e - 8);
                const float2 z = turn(v[0], v[1], c[e], sn[e]);
                v[0] = z.x;
                v[1] = z.y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int d = 8 * c0 + e;
                if (d >= a.rotary) continue;
                const float m = __bfloat162float(src[d >= half ? d - half : d + half]);
                float& v = e < 8 ? v0[e] : v1[e - 8];
                v = d >= half ? turn(m, v, c[e], sn[e]).y : turn(v, m, c[e], sn[e]).x;
            }
        }
    }
    const bool stored = ok && good_block(a, blk, report);
    uint8_t* rec = static_cast<uint8_t*>(is_v ? a.v_pool : a.k_pool) + (static_cast<size_t>(blk) * a.hkv + h) * R::kBytes;
    if (__any_sync(0xFFFFFFFFu, stored)) store_row<D, kFp4>(rec, p % kBlockSize, lane, c0, c1, split, v0, v1, g, stored);
}

template <int D, bool kFp4, int kPairs>
__global__ void __launch_bounds__(kAppendThreads) quant_append_kernel(const __grid_constant__ QuantArgs a, int first_token) {
    pdl_wait();  // dependents start as its CTAs leave: triggered here they took the slots of its last waves
    append_rows<D, kFp4, kPairs, kAppendThreads>(a, blockIdx.x, first_token);
}

// With q: blocks that rotate it as the rotation's kernels do (four heads a thread, bound
// by HBM) beside blocks that quantise K and V (bound by their waits).  While the whole
// call is a few waves, K and V go first, whose chain of loads and work is the longer; beyond,
// the two kinds alternate evenly, so that each SM runs both (4-bit, 32 + 8 heads of 128, K and
// V first against alternating: 1024 tokens 5.5 and 5.7 us, 4096 tokens 19.8 and 19.9, 16384
// tokens 71.0 and 67.4; 64 + 8 heads of 64: 1024 tokens 4.1 and 4.8).  Heads of q as rows
// beside those of K and V took 2.4 instead of 2.2 us for 16 tokens, 3.1 instead of 2.75 for 256, 6.7
// instead of 5.5 for 1024, 23.6 instead of 19.9 for 4096.  Where q's pairs are looked up a thread
// takes two heads (18 of 128 dims, 16 + 4 heads, 4096 tokens: 17.1 us, 24.8 with four heads, whose
// registers spill, 20.8 with one).
constexpr int kPartialHeads = 2;

struct MixPlan {
    unsigned vectors;  // of a q row that a thread of rotate_vectors takes one of, or 0
    PartialWarps w;    // and rotate_partial's
    unsigned q_slots, q_blocks, blocks;
    bool kv_first;
};

template <int D, bool kFp4, int kPairs>
__global__ void __launch_bounds__(kRopeThreads, 16) quant_append_q_kernel(const __grid_constant__ QuantArgs a,
                                                                              const __grid_constant__ RotateArgs r, MixPlan m,
                                                                              int first_token) {
    pdl_wait();
    const unsigned kv_blocks = m.blocks - m.q_blocks;
    // q blocks among the first blockIdx.x, and among one more
    unsigned before, after;
    if (m.kv_first) {
        before = blockIdx.x < kv_blocks ? 0 : blockIdx.x - kv_blocks;
        after = blockIdx.x < kv_blocks ? 0 : before + 1;
    } else {
        before = static_cast<unsigned>(static_cast<uint64_t>(blockIdx.x) * m.q_blocks / m.blocks);
        after = static_cast<unsigned>((static_cast<uint64_t>(blockIdx.x) + 1) * m.q_blocks / m.blocks);
    }
    if (after > before) {
        const unsigned thread = before * kRopeThreads + threadIdx.x;
        if (kPairs == kAnyPairs && m.vectors == 0)
            rotate_partial<__nv_bfloat16, kPartialHeads>(r, thread / 32u, m.w, m.q_slots, m.q_slots, first_token);
        else
            rotate_vectors<__nv_bfloat16, kPairs != kLanePairs, 4>(r, thread, m.vectors, m.q_slots, m.q_slots, first_token);
    } else {
        append_rows<D, kFp4, kPairs, kRopeThreads>(a, blockIdx.x - before, first_token);
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

// D/8 lanes per token and kRows heads, K and V of them in one thread: four heads where there
// are many rows, for fewer waves of the chain position, block id, row (4096 tokens of 8
// heads of 128, 4-bit: 6.0 us with one, 5.3 with two, 4.8 with four; 16384 tokens 24.4,
// 20.7, 18.8; below the bound, 4096 tokens of 8 heads of 64: 6.2 with one, 6.7 with two).
// Blocks of 128 threads took the 4.8 to 4.45, and left the calls with one head a thread.
constexpr int read_threads(int rows) { return rows > 1 ? 128 : 256; }

template <int D, bool kFp4, int kRows>
__global__ void __launch_bounds__(read_threads(kRows)) quant_read_kernel(const __grid_constant__ QuantArgs a, unsigned slots) {
    pdl_wait();
    constexpr int kLanes = D / 8;
    const int lane = threadIdx.x % kLanes;
    const long long group = static_cast<long long>(blockIdx.x) * (read_threads(kRows) / kLanes) + threadIdx.x / kLanes;
    // groups past 32 bits divide as 64-bit numbers
    const long long i = group <= 0xFFFFFFFFLL ? static_cast<unsigned>(group) / slots : group / slots;
    const int h0 = static_cast<int>(group - i * slots) * kRows;
    if (i >= a.num_tokens) return;
    const int s = a.token_to_seq[i], p = a.positions[i], row = p % kBlockSize;
    const bool report = lane == 0 && h0 == 0;
    if (!quant_token(a, s, p, report)) return;
    const int blk = quant_block(a, s, p);
    if (!good_block(a, blk, report)) return;
    const size_t at = (static_cast<size_t>(blk) * a.hkv + h0) * QuantRecord<D, kFp4>::kBytes;
    RowPart<D, kFp4> part[2][kRows];
#pragma unroll
    for (int n = 0; n < kRows; ++n)
#pragma unroll
        for (int pool = 0; pool < 2; ++pool)
            if ((pool ? a.v_out : a.k_out) && h0 + n < a.hkv)
                part[pool][n] = fetch_row<D, kFp4>(static_cast<const uint8_t*>(pool ? a.v_pool : a.k_pool) + at +
                                                       n * QuantRecord<D, kFp4>::kBytes, row, lane);
    const size_t to = (static_cast<size_t>(i) * a.hkv + h0) * D + 8 * lane;
#pragma unroll
    for (int n = 0; n < kRows; ++n)
#pragma unroll
        for (int pool = 0; pool < 2; ++pool) {
            void* dst = pool ? a.v_out : a.k_out;
            if (!dst || h0 + n >= a.hkv) continue;
            float v[8];
            widen_row<D, kFp4>(part[pool][n], kFp4 ? (pool ? a.v_scale : a.k_scale)[h0 + n] : 1.f, v);
            if (a.out_f32) {
                float4* o = reinterpret_cast<float4*>(static_cast<float*>(dst) + to + n * D);
                o[0] = make_float4(v[0], v[1], v[2], v[3]);
                o[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst) + to + n * D) = pack<__nv_bfloat16>(v);
            }
        }
}

// A CTA per (pair, kHeads heads): thread (row, lane) widens 8 dims of each of
// their records, K and V.
template <int D, bool kFp4, int kHeads>
__global__ void __launch_bounds__(2 * D) quant_load_kernel(const __grid_constant__ QuantArgs a) {
    pdl_wait();
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

constexpr long long kFewWaves = 1 << 25;         // an append's elements of q, K and V
constexpr long long kBusyThreads = 152LL * 512;  // 16 warps an SM: enough to give a thread more rows

// Launches over as many tokens as 32-bit thread indexes reach: launch(args, first token, tokens),
// with args that end at the launch's last token, so that none is taken twice.
template <typename Args, typename F>
cudaError_t token_runs(const Args& a, long long threads_per_token, F launch) {
    const long long most = (1LL << 31) / threads_per_token;
    if (most == 0) return cudaErrorInvalidValue;
    for (long long i = 0; i < a.num_tokens; i += most) {
        const long long n = a.num_tokens - i < most ? a.num_tokens - i : most;
        Args run = a;
        run.num_tokens = static_cast<int32_t>(i + n);
        const cudaError_t e = launch(run, static_cast<int>(i), n);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

dim3 blocks_of(long long threads, int per_block) { return dim3(static_cast<unsigned>((threads + per_block - 1) / per_block)); }

template <template <int, bool> class F>
cudaError_t by_format(const QuantArgs& a) {
    if (a.d == 64) return a.fp4 ? F<64, true>::go(a) : F<64, false>::go(a);
    return a.fp4 ? F<128, true>::go(a) : F<128, false>::go(a);
}

template <int D, bool kFp4>
struct AppendLaunch {
    template <int kPairs>
    static cudaError_t pairs(const QuantArgs& a) {
        const long long kv_threads = 2LL * a.hkv * (D / 16);
        if (a.q) return with_q<kPairs>(a, kv_threads);
        return token_runs(a, kv_threads, [&](const QuantArgs& run, int first, long long n) {
            return launch_pdl(quant_append_kernel<D, kFp4, kPairs>, blocks_of(n * kv_threads, kAppendThreads), dim3(kAppendThreads), 0,
                              a.stream, run, first);
        });
    }
    template <int kPairs>
    static cudaError_t with_q(const QuantArgs& a, long long kv_threads) {
        RotateArgs r{};
        r.q = RotateRows{a.q, a.q_out, a.q_stride, D, a.q_out_stride, D, a.hq};
        r.cos_sin = a.cos_sin;
        r.positions = a.positions;
        r.num_tokens = a.num_tokens;
        r.d = D;
        r.rotary = a.rotary;
        r.interleaved = a.interleaved;
        r.inverse = a.inverse;
        r.max_pos = a.max_pos;
        r.dtype = PKV_BF16;
        r.token_to_seq = a.token_to_seq;
        r.num_seqs = a.num_seqs;
        r.mbps = a.mbps;
        r.ring = a.ring;
        // q's pairs: as vectors, half-split with r a multiple of 16 too, or looked up in the row
        const bool whole = kPairs != kAnyPairs ||
                           (!a.interleaved && a.rotary % 16 == 0 && reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0);
        const bool in_place = a.q == a.q_out;
        const long long q_slots = whole ? (a.hq + 3) / 4 : (a.hq + kPartialHeads - 1) / kPartialHeads;
        const long long vectors = (kPairs != kLanePairs ? a.rotary / 2 : a.rotary) / 8 + (in_place ? 0 : (D - a.rotary) / 8);
        return token_runs(a, kv_threads + q_slots * (D / 8 + 32), [&](const QuantArgs& run, int first, long long n) {
            r.num_tokens = run.num_tokens;
            MixPlan m{};
            m.q_slots = static_cast<unsigned>(q_slots);
            long long q_threads = n * q_slots * vectors;
            if (whole) {
                m.vectors = static_cast<unsigned>(vectors);
            } else {
                m.w = partial_warps(r, 8, in_place, n * q_slots);
                q_threads = 32LL * m.w.all;
            }
            m.q_blocks = blocks_of(q_threads, kRopeThreads).x;
            m.blocks = m.q_blocks + blocks_of(n * kv_threads, kRopeThreads).x;
            m.kv_first = n * (2LL * a.hkv + a.hq) * D < kFewWaves;
            return launch_pdl(quant_append_q_kernel<D, kFp4, kPairs>, dim3(m.blocks), dim3(kRopeThreads), 0, a.stream, run, r, m, first);
        });
    }
    static cudaError_t go(const QuantArgs& a) {
        if (a.cos_sin && reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0) {
            if (!a.interleaved && a.rotary % 32 == 0) return pairs<kHalfPairs>(a);
            if (a.interleaved && a.rotary % 16 == 0) return pairs<kLanePairs>(a);
        }
        return pairs<kAnyPairs>(a);
    }
};
template <int D, bool kFp4>
struct ReadLaunch {
    template <int kRows>
    static cudaError_t rows(const QuantArgs& a) {
        const unsigned slots = static_cast<unsigned>((a.hkv + kRows - 1) / kRows);
        constexpr int kThreads = read_threads(kRows);
        const long long blocks = (static_cast<long long>(a.num_tokens) * slots * (D / 8) + kThreads - 1) / kThreads;
        if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
        return launch_pdl(quant_read_kernel<D, kFp4, kRows>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, a.stream, a, slots);
    }
    static cudaError_t go(const QuantArgs& a) {
        if (static_cast<long long>(a.num_tokens) * a.hkv * (D / 8) >= 4 * kBusyThreads) return rows<4>(a);
        return rows<1>(a);
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
    static constexpr int N = 16 / sizeof(T);
    // every row starts on a 16-byte boundary and is whole vectors
    static bool rows_fit(const RotateArgs& a) {
        auto rows = [](const RotateRows& r) {
            return r.num_heads == 0 ||
                   ((reinterpret_cast<uintptr_t>(r.in) | reinterpret_cast<uintptr_t>(r.out)) % 16 == 0 &&
                    (r.in_token | r.in_head | r.out_token | r.out_head) % N == 0);
        };
        return a.d % N == 0 && rows(a.q) && rows(a.k);
    }
    // in place nothing passes (with one of q and k in place, its passing dims are
    // written back as they are: the same bytes, by the thread that read them)
    static bool in_place(const RotateArgs& a) { return a.q.in == a.q.out && (a.k.num_heads == 0 || a.k.in == a.k.out); }
    template <bool kHalf, int kRows>
    static cudaError_t vectors(const RotateArgs& a, int count, cudaStream_t stream) {
        const unsigned q_slots = (a.q.num_heads + kRows - 1) / kRows, slots = q_slots + (a.k.num_heads + kRows - 1) / kRows;
        const long long per_token = static_cast<long long>(count) * slots;
        return token_runs(a, per_token, [&](const RotateArgs& run, int first, long long n) {
            return launch_pdl(rope_vector_kernel<T, kHalf, kRows>, blocks_of(n * per_token, kRopeThreads), dim3(kRopeThreads), 0, stream,
                              run, static_cast<unsigned>(count), q_slots, slots, first);
        });
    }
    template <bool kHalf>
    static cudaError_t by_rows(const RotateArgs& a, cudaStream_t stream) {
        const int count = (kHalf ? a.rotary / 2 : a.rotary) / N + (in_place(a) ? 0 : (a.d - a.rotary) / N);
        const long long one = static_cast<long long>(a.num_tokens) * (a.q.num_heads + a.k.num_heads) * count;
        if (one >= 4 * kBusyThreads) return vectors<kHalf, 4>(a, count, stream);
        return vectors<kHalf, 1>(a, count, stream);
    }
    template <int kRows>
    static cudaError_t partial(const RotateArgs& a, cudaStream_t stream) {
        const unsigned q_slots = (a.q.num_heads + kRows - 1) / kRows, slots = q_slots + (a.k.num_heads + kRows - 1) / kRows;
        return token_runs(a, static_cast<long long>(slots) * (a.d / N + 32), [&](const RotateArgs& run, int first, long long n) {
            const PartialWarps w = partial_warps(a, N, in_place(a), n * slots);
            return launch_pdl(rope_partial_kernel<T, kRows>, blocks_of(32LL * w.all, kRopeThreads), dim3(kRopeThreads), 0, stream, run, w,
                              q_slots, slots, first);
        });
    }
    static cudaError_t any(const RotateArgs& a, bool vec, cudaStream_t stream) {
        const unsigned pair_items = static_cast<unsigned>((a.rotary / 2 + kPairRun - 1) / kPairRun);
        const unsigned items = pair_items + (in_place(a) || a.rotary == a.d ? 0u : static_cast<unsigned>((a.d + N - 1) / N - a.rotary / N));
        const long long per_token = static_cast<long long>(items) * (a.q.num_heads + a.k.num_heads);
        return token_runs(a, per_token, [&](const RotateArgs& run, int first, long long n) {
            return launch_pdl(rope_any_kernel<T>, blocks_of(n * per_token, kRopeThreads), dim3(kRopeThreads), 0, stream, run, pair_items,
                              items, vec, first);
        });
    }
    static cudaError_t go(const RotateArgs& a, cudaStream_t stream) {
        const bool vec = rows_fit(a);
        if (vec && a.rotary % (a.interleaved ? N : 2 * N) == 0 && reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0)
            return a.interleaved ? by_rows<false>(a, stream) : by_rows<true>(a, stream);
        if (vec && (a.rotary + N - 1) / N <= 32) {
            const long long one = static_cast<long long>(a.num_tokens) * (a.q.num_heads + a.k.num_heads) *
                                  (in_place(a) ? (a.rotary + N - 1) / N : a.d / N);
            return one >= 4 * kBusyThreads ? partial<4>(a, stream) : partial<1>(a, stream);
        }
        return any(a, vec, stream);
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
