// quant_decode.cu -- split-KV GQA decode attention over the quantised pools.
//
//   o = softmax(sm_scale * q k^T) v over the visible keys, k and v the records'
//   values (int8 code * row scale; e2m1 * 16-dim scale * head scale); a sink
//   logit joins the normaliser with a zero value.
//
// Work decomposition.  The visible blocks of every (sequence, KV head) are cut
// into chunks (the planner in api.cu); a CTA owns one chunk and its 4 warps
// take the chunk's blocks round-robin, NB at a time, each with its own ring of
// asynchronous copies (a K record and a V record per block, 16 bytes a lane; a record
// holds codes and scales side by side, already in the bank-conflict-free order).
// The warps' states meet in shared memory.  The chunks of a sequence merge in a
// thread-block cluster where the whole grid is resident, else by a second launch over
// the fp32 states they leave in the workspace: a last-chunk ticket in this kernel cost
// 3 to 6 us of fence, atomic and serial merge (2 pairs of 2048 blocks 12.8 us, 7.9 with
// the second launch; 960 pairs 434 us, 424), and its registers slowed the main loop 3 %.
//
// The MMAs run transposed: S^T = K Q^T and O^T += V^T P^T (m16n8k16, f16 ->
// fp32), so the 16 tokens of a block (S^T) and the head's dims (O^T) fill the
// m16 side and up to 8 query heads the n8 side: a group of at most 8 heads
// pads nothing, and a lane's softmax state is that of its two heads.  Both
// products allow any order of their summed index, which is used to read codes
// as they lie:
//   S^T: lane (g, t) reads dims [t D/4, (t+1) D/4) of two tokens' rows, k-step j
//        taking dims t D/4 + 4j .. + 3; q takes the same order;
//   O^T: lane (g, t) reads dims [g D/8, (g+1) D/8) of four tokens' rows, m-tile i
//        taking dims g D/8 + 2i (row g) and + 1 (row g + 8); token slot k of a
//        block is row slot_row(k), for S^T and O^T alike.
// P^T in the second product's operand layout is the first's result transposed
// per 8x8: one movmatrix each.
//
// Operands are exact: codes are integers below 128, or e2m1 times e4m3 (6 significant
// bits, at least 2^-10), q is scaled by a power of two into f16's range: one for the
// group's heads, or where they lie more than 2^10 apart one for each (a common one rounds
// a head away beside one of 2^40 times its size).  The int8 row scale of K multiplies the
// logit, that of V the weight, and a power of two for each head brings their product into
// f16's range: it follows the largest product, not the largest scale, so that a row of
// little weight takes no bits from the others.  What goes into the MMA is rounded to f16
// (by 2^-11 of it or 2^-25 of the largest weight, int8: 2^-29 of the largest product);
// the statistics, l and O are fp32.
//
// What bounds it.  Per token and KV head it reads 2 (D + 4) bytes (int8) or 2 (D/2 + D/16)
// (4-bit) for 4 D G flops: HBM by the roofline.  int8 gets there (76 sequences x 8 KV heads
// of 512 blocks, one steady wave: 6.18 TB/s at D = 128, 6.02 at 64; its copies alone 6.58
// and 6.50).  A 4-bit block of D = 128 is 2304 bytes and costs a warp about 265 instructions
// beside 16 MMAs, which hold the issue port for 8 cycles each (an MMA with 4 independent
// FMAs measured 11.7 cycles, alone 8.0): some 390 issue cycles where HBM delivers a block
// every 404.  So one steady wave runs at 6.24 TB/s and its copies alone at 6.89; at D = 64,
// half the bytes for more than half the instructions, at 5.07 and 6.18.  Tried and dropped:
// one bulk copy per record (5.49 TB/s where this was 6.01: a copy's issue costs a warp more
// than 5 per-lane ones), one block per pass (5.60), 5 or 6 CTAs per SM (5.49, 4.07: the port,
// not latency, is short), 8-warp CTAs (long batch 462 us, 426 with 4 warps).
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

template <int D, bool kFp4, int NT>
struct Cfg {
    using R = QuantRecord<D, kFp4>;
    static constexpr int kTile = (R::kBytes + 127) / 128 * 128;  // a record in shared memory
    static constexpr int kBlock = 2 * kTile;                     // K + V
    // blocks of one loop pass: two share its softmax vote and loop overhead
    static constexpr int NB = !kFp4 && D == 128 ? 1 : 2;
    static constexpr int kStage = NB * kBlock;
    static constexpr int kStages = kFp4 ? (D == 128 ? 3 : 4) : 3;
    static constexpr int kFull = R::kBytes / 512;                // 16-byte copies of a whole warp per record
    static constexpr int kTail = R::kBytes % 512 / 16;           // lanes of the rest: K's, then V's
    static_assert(R::kBytes % 16 == 0 && 2 * kTail <= 32, "one copy brings both tails");
    static constexpr int kHeads = 8 * NT;
    static constexpr int kCombStride = D + 4;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kComb = kWarps * kHeads * kCombStride * 4;
    static constexpr int kSmem = (kRing > kComb ? kRing : kComb) + 128;
    // registers: NT * D / 4 accumulators and NT * D / 8 of q
    static constexpr int kCtas = NT * D > 128 ? 3 : 4;
};

// The row of a block that token slot k (0..7; slot k + 8 is row + 8) stands for:
// pairs swapped where that spreads the rows one load touches over all banks.
template <int kRowBytes>
__device__ __forceinline__ constexpr int slot_row(int k) {
    return kRowBytes == 128 ? k : kRowBytes == 64 ? k ^ ((k >> 1) & 1) : k ^ ((k >> 2) & 1);
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t hsub2_bits(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Four bytes of e2m1 pairs -> four f16x2 words.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&d)[4]) {
    asm("{\n\t.reg .b8 a, b, c, e;\n\tmov.b32 {a, b, c, e}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, e;\n\t}"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(w));
}

// Two e4m3 scales (the low and high byte) -> f16x2.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t pair) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(pair)));
    return d;
}

// Codes + 128 in bytes 0, 1 (or 2, 3) of w -> their f16 values: 0x6400 | u is
// 1024 + u, less 1152 (both exact).
template <bool kHigh>
__device__ __forceinline__ uint32_t int8x2(uint32_t w) {
    return hsub2_bits(__byte_perm(w, 0x64646464u, kHigh ? 0x4342 : 0x4140), 0x64806480u);
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most N of this thread's latest groups are still in flight.
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's running state: lane (g, t) holds heads 2t, 2t + 1 (+ 8 nt) as a pair.
template <int D, int NT>
struct State {
    float mu[NT][2];    // what is subtracted from the logits (exp2 domain), -inf before any key
    uint64_t l[NT];     // this lane's share of sum 2^(x - mu), both heads
    float o[NT][D / 16][4];
    float vf[NT][2];    // int8: the powers of two on weight x V row scale, inf before any key
};

constexpr float kGrow = 8.f;    // logits may exceed mu by this before it moves (2^8 fits f16)
constexpr float kVGrow = 32768.f;  // int8: weight x V row scale x vf may reach this (it fits f16)
// From logits of this size on every pass rounds them before mu leaves them: fused, the largest
// would keep what mu's rounding took, up to 2^8 of a logit of 2^32, a weight of 2^256.
constexpr float kFar = 16777216.f;

// S^T = K Q^T of one block: 16 token slots x 8 NT heads.
template <int D, bool kFp4, int NT>
__device__ __forceinline__ void scores(float (&s)[NT][4], const uint32_t (&qb)[NT][D / 16][2], const uint8_t* kt, int row,
                                       int t) {
    using R = QuantRecord<D, kFp4>;
    constexpr int RB = R::kRowBytes;
    uint32_t kw[2][RB / 16];  // this lane's RB/4 bytes of rows row and row + 8
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint8_t* base = kt + half * 8 * RB;
        if constexpr (RB == 128) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
                *reinterpret_cast<uint4*>(&kw[half][4 * c]) =
                    *reinterpret_cast<const uint4*>(base + quant_chunk<RB>(row, 2 * t + c));
        } else if constexpr (RB == 64) {
            *reinterpret_cast<uint4*>(&kw[half][0]) = *reinterpret_cast<const uint4*>(base + quant_chunk<RB>(row, t));
        } else {
            *reinterpret_cast<uint2*>(&kw[half][0]) =
                *reinterpret_cast<const uint2*>(base + quant_chunk<RB>(row, t >> 1) + 8 * (t & 1));
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    if constexpr (kFp4) {
        uint32_t sc[2][D / 64];  // f16x2, both halves the scale of 16 dims
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint8_t* p = kt + R::kScales + (row + 8 * half) * R::kScaleBytes + t * (D / 64);
            if constexpr (D == 128) {
                const uint32_t v = e4m3x2(*reinterpret_cast<const uint16_t*>(p));
                sc[half][0] = __byte_perm(v, v, 0x1010);
                sc[half][1] = __byte_perm(v, v, 0x3232);
            } else {
                const uint32_t v = e4m3x2(*p);
                sc[half][0] = __byte_perm(v, v, 0x1010);
            }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {  // a word: 8 dims, two k-steps
            uint32_t r0[4], r1[4];
            e2m1x8(kw[0][w], r0);
            e2m1x8(kw[1][w], r1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r0[i] = hmul2_bits(r0[i], sc[0][w / 2]);
                r1[i] = hmul2_bits(r1[i], sc[1][w / 2]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t a[4] = {r0[2 * j], r1[2 * j], r0[2 * j + 1], r1[2 * j + 1]};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_16816<true>(s[n], a, qb[n][2 * w + j][0], qb[n][2 * w + j][1]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const uint32_t a[4] = {int8x2<false>(kw[0][j]), int8x2<false>(kw[1][j]), int8x2<true>(kw[0][j]),
                                   int8x2<true>(kw[1][j])};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816<true>(s[n], a, qb[n][j][0], qb[n][j][1]);
        }
    }
}

// O^T += V^T P^T of one block: D dims x 8 NT heads.  vs2: f16x2 scales (4-bit) of
// rows (ta, tb) and (ta + 8, tb + 8).
template <int D, bool kFp4, int NT>
__device__ __forceinline__ void accumulate(float (&o)[NT][D / 16][4], const uint32_t (&pb)[NT][2], const uint8_t* vt, int g,
                                           int ta, int tb, const uint32_t (&vs2)[2]) {
    using R = QuantRecord<D, kFp4>;
    constexpr int RB = R::kRowBytes;
    constexpr int VB = RB / 8;  // this lane's bytes of a token's row
    constexpr int VW = VB / 4;
    uint32_t vw[4][VW];  // rows ta, tb, ta + 8, tb + 8
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t* q = vt + (i & 2 ? 8 * RB : 0) + quant_chunk<RB>(i & 1 ? tb : ta, g * VB / 16) + (g * VB) % 16;
        if constexpr (VB == 16) {
            *reinterpret_cast<uint4*>(vw[i]) = *reinterpret_cast<const uint4*>(q);
        } else if constexpr (VB == 8) {
            *reinterpret_cast<uint2*>(vw[i]) = *reinterpret_cast<const uint2*>(q);
        } else {
            vw[i][0] = *reinterpret_cast<const uint32_t*>(q);
        }
    }
    if constexpr (kFp4) {
#pragma unroll
        for (int w = 0; w < VW; ++w) {  // a word: 8 dims, four m-tiles
            uint32_t even[2][4], odd[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x = vw[2 * h][w], y = vw[2 * h + 1][w];
                e2m1x8((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), even[h]);
                e2m1x8(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), odd[h]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a[4] = {hmul2_bits(even[0][i], vs2[0]), hmul2_bits(odd[0][i], vs2[0]),
                                       hmul2_bits(even[1][i], vs2[1]), hmul2_bits(odd[1][i], vs2[1])};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_16816<true>(o[n][4 * w + i], a, pb[n][0], pb[n][1]);
            }
        }
    } else {
        (void)vs2;
#pragma unroll
        for (int w = 0; w < VW; ++w) {  // a word: 4 dims, two m-tiles
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t lo2 = __byte_perm(vw[0][w], vw[1][w], i ? 0x7362 : 0x5140);
                const uint32_t hi2 = __byte_perm(vw[2][w], vw[3][w], i ? 0x7362 : 0x5140);
                const uint32_t a[4] = {int8x2<false>(lo2), int8x2<true>(lo2), int8x2<false>(hi2), int8x2<true>(hi2)};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_16816<true>(o[n][2 * w + i], a, pb[n][0], pb[n][1]);
            }
        }
    }
}

// NB consecutive blocks, K and V records of block i at stage + i * kBlock: tok_base is
// the first one's first position, keys in [lo, hi) take part.  kEdge: some of the blocks'
// tokens may lie outside (masking them as they come cost 24 instructions a block in the
// passes that have none), the group's heads have scales of their own (a pair of them in
// registers, in every pass, cost the 4-bit kernel of D = 128 1.7 %; with heads 2^12 apart
// it takes 96.8 us where it takes 89.4 with heads alike, 57 sequences x 8 KV heads of 512
// blocks), or, 4-bit, the logits may reach kFar.  sl: what the logits are scaled by;
// kEdge: head_sl[h] those of head h.
template <int D, bool kFp4, int NT, bool kEdge>
__device__ __forceinline__ void attend(State<D, NT>& st, const uint32_t (&qb)[NT][D / 16][2], const uint8_t* stage,
                                       int lane, uint32_t tok_base, uint32_t lo, uint32_t hi,
                                       const float* head_sl, float sl) {
    using C = Cfg<D, kFp4, NT>;
    using R = QuantRecord<D, kFp4>;
    constexpr int RB = R::kRowBytes, NB = C::NB;
    const int g = lane >> 2, t = lane & 3;
    const int row = slot_row<RB>(g);                                    // S^T's rows: row, row + 8
    const int ta = slot_row<RB>(2 * t), tb = slot_row<RB>(2 * t + 1);  // O^T's token slots: rows ta, tb (+ 8)
    auto visible = [&](int b, int r) { return tok_base - lo + static_cast<uint32_t>(b * kBlockSize + r) < hi - lo; };

    float s[NB][NT][4];
    float ks[NB][2];      // int8: the rows' K scales
    float vs[NB][2];      // int8: the rows' V scales
    uint32_t vs2[NB][2];  // 4-bit: V's f16x2 scales of rows (ta, tb) and (ta + 8, tb + 8)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint8_t* kt = stage + b * C::kBlock;
        const uint8_t* vt = kt + C::kTile;
        scores<D, kFp4, NT>(s[b], qb, kt, row, t);
        vs2[b][0] = vs2[b][1] = 0u;
        if constexpr (kFp4) {
            const uint8_t* p = vt + R::kScales + (D == 128 ? g : g >> 1);
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = p[((i & 1 ? tb : ta) + (i & 2 ? 8 : 0)) * R::kScaleBytes];
            if constexpr (kEdge) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!visible(b, (i & 1 ? tb : ta) + (i & 2 ? 8 : 0))) c[i] = 0;
            }
            vs2[b][0] = e4m3x2(__byte_perm(c[0], c[1], 0x0040));
            vs2[b][1] = e4m3x2(__byte_perm(c[2], c[3], 0x0040));
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ks[b][h] = *reinterpret_cast<const float*>(kt + R::kScales + (row + 8 * h) * 4);
                vs[b][h] = *reinterpret_cast<const float*>(vt + R::kScales + (row + 8 * h) * 4);
            }
        }
        if constexpr (kEdge) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (!visible(b, row + 8 * h)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) s[b][n][2 * h] = s[b][n][2 * h + 1] = -INFINITY;
                    ks[b][h] = 1.f;  // > 0: the product stays -inf
                    vs[b][h] = 0.f;
                }
        }
    }

    // ---- softmax: p = 2^(s kf - mu), mu moving only when a logit exceeds it by 2^8
    auto kf = [&](int b, int n, int h) {
        if constexpr (kEdge) {
            const uint64_t two = *reinterpret_cast<const uint64_t*>(head_sl + 2 * t + 8 * n);
            return kFp4 ? two : mul_f32x2(pack_f32x2(ks[b][h], ks[b][h]), two);
        }
        const float f = kFp4 ? sl : ks[b][h] * sl;
        return pack_f32x2(f, f);
    };
    constexpr bool kMayBeFar = kEdge || !kFp4;
    uint64_t p[NB][NT][2];  // row, row + 8: a pair of heads each
    auto logits = [&]() {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    p[b][n][h] = fma_f32x2(pack_f32x2(s[b][n][2 * h], s[b][n][2 * h + 1]), kf(b, n, h),
                                           pack_f32x2(-st.mu[n][0], -st.mu[n][1]));
    };
    auto logit = [&](int b, int n, int i) {  // rounded
        float k[2];
        unpack_f32x2(kf(b, n, i / 2), k[0], k[1]);
        return __fmul_rn(s[b][n][i], k[i % 2]);
    };
    logits();
    float top = -INFINITY;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x, y;
                unpack_f32x2(p[b][n][h], x, y);
                top = fmax3(top, x, y);  // +inf while mu is -inf: a pass's first block has a visible key
            }
    bool grow = top > kGrow;
    if constexpr (kMayBeFar) {
        float far = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) far = fmax3(far, fabsf(st.mu[n][0]), fabsf(st.mu[n][1]));
        grow = grow || far > kFar;
    }
    // int8: the logits' weights, those of O times V's row scale and vf; whether one is too large
    uint64_t sum[NT];
    auto weigh = [&]() {
        float most = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) sum[n] = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x, y;
                    unpack_f32x2(p[b][n][h], x, y);
                    const uint64_t w = pack_f32x2(fast_exp2(x), fast_exp2(y));
                    sum[n] = add_f32x2(sum[n], w);
                    p[b][n][h] = mul_f32x2(mul_f32x2(w, pack_f32x2(vs[b][h], vs[b][h])), pack_f32x2(st.vf[n][0], st.vf[n][1]));
                    unpack_f32x2(p[b][n][h], x, y);
                    most = fmax3(most, x, y);
                }
        return most > kVGrow;
    };
    // int8: with 8 heads a group the weights come before the one vote; with 16, whose weights
    // would not fit the registers beside the logits, after it, with a vote of their own (64
    // sequences of up to 2048 keys, 16 heads: 19.3 us, 20.1 with one; 8 heads: 14.3 and 14.0)
    constexpr bool kAhead = !kFp4 && NT == 1;
    if constexpr (kAhead) grow = weigh() || grow;
    for (int turn = 0;; ++turn) {
        if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float keep[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = -INFINITY, scale;
#pragma unroll
                    for (int b = 0; b < NB; ++b) mx = fmax3(mx, logit(b, n, c), logit(b, n, c + 2));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
                    if constexpr (!kFp4) mx = ceilf(mx);  // so that mu moves by whole powers of two, and vf with it
                    const float mn = fmaxf(st.mu[n][c], mx), up = mn - st.mu[n][c];
                    keep[c] = mn == -INFINITY ? 1.f : fast_exp2(-up);
                    st.mu[n][c] = mn;
                    scale = keep[c];
                    if constexpr (!kFp4) {
                        // vf brings the largest product here into [2^4, 2^5), but those before, which mu
                        // has made 2^-up of what they were, to no more than it did; 2^120 at most
                        float m = 0.f;
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                m = fmaxf(m, fast_exp2(__fsub_rn(logit(b, n, c + 2 * h), mn)) * vs[b][h]);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
                        const int moved = static_cast<int>(fminf(up, 1024.f)), old = __float_as_uint(st.vf[n][c]) >> 23;
                        const int now = min(min(258 - static_cast<int>(__float_as_uint(m) >> 23), 247), old + moved);  // exponents
                        st.vf[n][c] = __uint_as_float(static_cast<uint32_t>(now) << 23);
                        // O times keep and the change of vf: at most 1, and below 2^-126 O still is 0
                        const int step = now - old - moved;
                        scale = step < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + step) << 23);
                    }
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        st.o[n][i][c] *= scale;
                        st.o[n][i][c + 2] *= scale;
                    }
                }
                st.l[n] = mul_f32x2(st.l[n], pack_f32x2(keep[0], keep[1]));
            }
            if constexpr (kMayBeFar) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            p[b][n][h] = pack_f32x2(__fsub_rn(logit(b, n, 2 * h), st.mu[n][0]),
                                                    __fsub_rn(logit(b, n, 2 * h + 1), st.mu[n][1]));
            } else {
                logits();
            }
            if constexpr (kAhead) weigh();
        }
        if constexpr (kFp4 || kAhead) break;
        grow = weigh();
        if (turn == 1 || !__any_sync(0xFFFFFFFFu, grow)) break;
    }
    uint32_t pb[NB][NT][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x, y;
                unpack_f32x2(p[b][n][h], x, y);
                if constexpr (kFp4) {
                    x = fast_exp2(x);
                    y = fast_exp2(y);
                    st.l[n] = add_f32x2(st.l[n], pack_f32x2(x, y));
                }
                pb[b][n][h] = movmatrix(pack2<true>(x, y));
            }
    if constexpr (!kFp4) {
#pragma unroll
        for (int n = 0; n < NT; ++n) st.l[n] = add_f32x2(st.l[n], sum[n]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
        accumulate<D, kFp4, NT>(st.o, pb[b], stage + b * C::kBlock + C::kTile, g, ta, tb, vs2[b]);
}

// The chunks of a (sequence, KV head) are one cluster: each joins its share of the
// output from its peers' shared memory (states in comb's first rows, their lse).
// Out of line, so that the merge's registers do not weigh on the main loop.
template <int D, bool kFp4, int NT>
__device__ __noinline__ void merge_cluster(const QuantDecodeArgs& a, float* comb, const float* lse, int split, int kvh,
                                           size_t head0, int nsplit) {
    using C = Cfg<D, kFp4, NT>;
    const int G = a.group;
    cluster_sync();
    float* wts = comb + C::kHeads * C::kCombStride;  // warp 1's rows, free now: [chunk][16]
    float* row_inv = wts + kQuantCluster * 16;
    if (threadIdx.x < G) {
        const int h = threadIdx.x;
        const float sk = a.sinks ? a.sinks[kvh * G + h] : -INFINITY;
        float l[kQuantCluster], M = sk;
#pragma unroll
        for (int c = 0; c < kQuantCluster; ++c) {
            l[c] = c < nsplit ? ld_cluster_f32(cluster_map(smem_u32(&lse[h]), c)) : -INFINITY;
            M = fmaxf(M, l[c]);
        }
        float W = sk == -INFINITY ? 0.f : expf(sk - M);
#pragma unroll
        for (int c = 0; c < kQuantCluster; ++c) {
            const float w = l[c] == -INFINITY ? 0.f : expf(l[c] - M);
            wts[c * 16 + h] = w;
            W += w;
        }
        row_inv[h] = W != 0.f ? 1.f / W : 0.f;
        if (a.lse_out && split == 0) a.lse_out[head0 + h] = W != 0.f ? M + logf(W) : -INFINITY;
    }
    __syncthreads();
    const int total = G * (D / 4);
    for (int i = split * total / nsplit + threadIdx.x; i < (split + 1) * total / nsplit; i += kThreads) {
        const int h = i / (D / 4), d = 4 * (i % (D / 4));
        const uint32_t at = smem_u32(comb + h * C::kCombStride + d);
        float4 x[kQuantCluster];
#pragma unroll
        for (int c = 0; c < kQuantCluster; ++c)
            if (c < nsplit) x[c] = ld_cluster_f32x4(cluster_map(at, c));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kQuantCluster; ++c) {
            const float w = wts[c * 16 + h];
            if (c < nsplit && w != 0.f) {
                v.x += w * x[c].x;
                v.y += w * x[c].y;
                v.z += w * x[c].z;
                v.w += w * x[c].w;
            }
        }
        const float inv = row_inv[h];
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (head0 + h) * D + d) =
            make_uint2(pack2<false>(v.x * inv, v.y * inv), pack2<false>(v.z * inv, v.w * inv));
    }
    cluster_sync();  // no chunk leaves while a peer may still read its state
}

template <int D, bool kFp4, int NT, bool kCluster>
__global__ void __launch_bounds__(kThreads, (Cfg<D, kFp4, NT>::kCtas)) quant_decode_kernel(const __grid_constant__ QuantDecodeArgs a) {
    using C = Cfg<D, kFp4, NT>;
    using R = QuantRecord<D, kFp4>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ __align__(8) float s_sl[kWarps][16];
    __shared__ float s_m[kWarps][16], s_l[kWarps][16], s_v[kFp4 ? 1 : kWarps][16];
    uint8_t* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x, kvh = blockIdx.y, seq = blockIdx.z;
    const int G = a.group;
    pdl_wait();
    pdl_launch_dependents();

    const int32_t* bt = a.block_tables + static_cast<size_t>(seq) * a.mbps;
    // without a window a chunk's blocks do not depend on the length: the ids are
    // read while it is in flight
    int id_next = 0;
    const int early = C::NB * (warp + kWarps * (lane / C::NB)) + lane % C::NB;
    if (a.window <= 0 && early < a.chunk_blocks && split * a.chunk_blocks + early < a.mbps)
        id_next = bt[split * a.chunk_blocks + early];
    int ctx = a.context_lens[seq];
    // q, read while the length and the ids are in flight: lane (g, t) holds head g's
    // dims t D/4 + 4j .. + 3 for k-step j
    const size_t head0 = static_cast<size_t>(seq) * a.hq + kvh * G;  // the group's first row of q, out, lse
    const int g = lane >> 2, t = lane & 3;
    uint32_t qb[NT][D / 16][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint2 v = make_uint2(0u, 0u);
            if (g + 8 * n < G)
                v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) + (head0 + g + 8 * n) * D +
                                                    t * (D / 4) + 4 * j);
            qb[n][j][0] = v.x;
            qb[n][j][1] = v.y;
        }
    if (ctx > a.max_ctx) {
        if (threadIdx.x == 0 && split == 0 && kvh == 0) flag_error(a.err, PKV_DEVERR_LENGTH);
        ctx = a.max_ctx;
    }
    const int lo = a.window > 0 && ctx > a.window ? ctx - a.window : 0;
    if (ctx <= 0) {
        if (split == 0) {
            for (int i = threadIdx.x; i < G * D; i += kThreads)
                static_cast<__nv_bfloat16*>(a.out)[head0 * D + i] = __float2bfloat16_rn(0.f);
            if (a.lse_out && threadIdx.x < G)
                a.lse_out[head0 + threadIdx.x] = a.sinks ? a.sinks[kvh * G + threadIdx.x] : -INFINITY;
        }
        return;
    }
    const int first_blk = lo / kBlockSize, last_blk = (ctx - 1) / kBlockSize;
    const int nsplit = (last_blk - first_blk + a.chunk_blocks) / a.chunk_blocks;
    if (split >= nsplit) return;
    const int b0 = first_blk + split * a.chunk_blocks;
    const int b1 = min(last_blk + 1, b0 + a.chunk_blocks);
    const int hi = b1 > last_blk ? ctx : b1 * kBlockSize;
    // this warp's passes: NB blocks each, warp after warp
    const int passes = ((b1 - b0 + C::NB - 1) / C::NB - warp + kWarps - 1) / kWarps;

    // ids of this warp's blocks, 32 at a time: lane k holds that of its block 32
    // batch + k.  A bad id is flagged and reads block 0.
    auto logical = [&](int k) { return b0 + C::NB * (warp + kWarps * (k / C::NB)) + k % C::NB; };
    auto fetch_ids = [&](int batch) {
        const int lb = logical(32 * batch + lane);
        return lb < b1 ? bt[a.ring > 0 ? lb % a.ring : lb] : 0;
    };
    auto check_id = [&](int id, int batch) {
        if (id < 0 || id >= a.num_blocks) {
            if (logical(32 * batch + lane) < b1) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
            id = 0;
        }
        return id;
    };
    if (a.window > 0) id_next = fetch_ids(0);
    int id_cur = 0;
    // a pass's blocks into a stage: 16 bytes a lane, the two records' last lines
    // together; every call commits one group, empty past the warp's end
    const uint8_t* kp = static_cast<const uint8_t*>(a.k_pool) + static_cast<size_t>(kvh) * R::kBytes + lane * 16;
    const uint8_t* vp = static_cast<const uint8_t*>(a.v_pool) + static_cast<size_t>(kvh) * R::kBytes + lane * 16;
    const uint8_t* tp = (lane < C::kTail ? kp : vp - C::kTail * 16) + C::kFull * 512;
    const uint32_t block_bytes = static_cast<uint32_t>(a.hkv) * R::kBytes;
    uint8_t* ring = smem + warp * C::kStages * C::kStage;
    const uint32_t to = smem_u32(ring) + lane * 16;
    const uint32_t to_tail = to + (lane < C::kTail ? 0 : C::kTile - C::kTail * 16) + C::kFull * 512;
    int lb = b0 + C::NB * warp;  // the next pass's first block
    auto load = [&](int pass, uint32_t stage) {
        const int k0 = pass * C::NB;
        if ((k0 & 31) == 0) {
            id_cur = check_id(id_next, k0 >> 5);
            id_next = fetch_ids((k0 >> 5) + 1);
        }
#pragma unroll
        for (int b = 0; b < C::NB; ++b) {
            const uint32_t id = static_cast<uint32_t>(__shfl_sync(0xFFFFFFFFu, id_cur, (k0 + b) & 31));
            if (lb + b < b1) {
                const uint8_t* ks = kp + static_cast<uint64_t>(block_bytes) * id;
                const uint8_t* vs = vp + static_cast<uint64_t>(block_bytes) * id;
                const uint32_t dst = stage + b * C::kBlock;
#pragma unroll
                for (int i = 0; i < C::kFull; ++i) {
                    copy16(to + dst + 512 * i, ks + 512 * i);
                    copy16(to + dst + C::kTile + 512 * i, vs + 512 * i);
                }
                if (lane < 2 * C::kTail) copy16(to_tail + dst, tp + static_cast<uint64_t>(block_bytes) * id);
            }
        }
        lb += kWarps * C::NB;
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) load(i, i * C::kStage);

    // ---- q as f16, scaled by 2^(12 - e), e the exponent of the group's largest |q|, or where
    // a head's is below 2^-10 of that, of its own
    float m[NT], all = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) m[n] = fmax3(m[n], fabsf(bf16_lo(qb[n][j][i])), fabsf(bf16_hi(qb[n][j][i])));
        m[n] = fmaxf(m[n], __shfl_xor_sync(0xFFFFFFFFu, m[n], 1));
        m[n] = fmaxf(m[n], __shfl_xor_sync(0xFFFFFFFFu, m[n], 2));
        all = fmaxf(all, m[n]);
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) all = fmaxf(all, __shfl_xor_sync(0xFFFFFFFFu, all, x));
    bool apart = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) apart = apart || (m[n] > 0.f && m[n] < all * 9.765625e-4f);
    apart = __any_sync(0xFFFFFFFFu, apart);
    float scale = a.sm_scale * 1.4426950408889634f;
    if constexpr (kFp4) scale *= a.k_scale[kvh];
    float sl = 0.f;  // what the logits are scaled by, times log2 e: where apart, of the lane's last head
    bool far = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float top = apart ? m[n] : all;
        const int qe = top > 0.f ? max(12, static_cast<int>(__float_as_uint(top) >> 23)) : 139;
        const float qf = __uint_as_float(static_cast<uint32_t>(266 - qe) << 23);  // 2^(139 - qe)
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) qb[n][j][i] = pack2<true>(bf16_lo(qb[n][j][i]) * qf, bf16_hi(qb[n][j][i]) * qf);
        // never 0, which would turn a masked logit, -inf, into a NaN
        sl = fmaxf(ldexpf(scale, qe - 139), 1.401298464324817e-45f);
        if (t == 0) s_sl[warp][g + 8 * n] = sl;
        // 4-bit: a key is at most 6 * 448, q as scaled below 2^13
        far = far || (kFp4 && !(sl * (D * 8192.f * 2688.f) <= kFar));
    }
    const bool care = apart || __any_sync(0xFFFFFFFFu, far);
    __syncwarp();

    State<D, NT> st;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        st.mu[n][0] = st.mu[n][1] = -INFINITY;
        st.vf[n][0] = st.vf[n][1] = INFINITY;
        st.l[n] = 0;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.o[n][i][0] = st.o[n][i][1] = st.o[n][i][2] = st.o[n][i][3] = 0.f;
    }

    // pass i sits in stage i mod kStages; pass i + kStages - 1 goes where pass i - 1
    // was, which every lane has read by the time all are past the __syncwarp
    uint32_t here = 0, next = (C::kStages - 1) * C::kStage;
    // a ring's positions run to the end of 31 bits, a pass's last beyond: unsigned
    uint32_t tok = (b0 + C::NB * warp) * kBlockSize;
    for (int i = 0; i < passes; ++i) {
        copy_wait<C::kStages - 2>();  // this lane's copies of pass i have landed
        __syncwarp();                 // and every lane's
        load(i + C::kStages - 1, next);
        if (!care && tok >= static_cast<uint32_t>(lo) && tok + C::NB * kBlockSize <= static_cast<uint32_t>(hi))
            attend<D, kFp4, NT, false>(st, qb, ring + here, lane, tok, lo, hi, s_sl[warp], sl);
        else
            attend<D, kFp4, NT, true>(st, qb, ring + here, lane, tok, lo, hi, s_sl[warp], sl);
        tok += kWarps * C::NB * kBlockSize;
        next = here;
        here = here + C::kStage == C::kStages * C::kStage ? 0 : here + C::kStage;
    }
    copy_wait<0>();

    // ---- the 4 warps' states meet
    float l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        unpack_f32x2(st.l[n], l[n][0], l[n][1]);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], x);
    }
    __syncthreads();  // every warp is done with its ring
    float* comb = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int h = 2 * t + c + 8 * n;
            float* cw = comb + (warp * C::kHeads + h) * C::kCombStride + g * (D / 8);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                *reinterpret_cast<float2*>(cw + 2 * i) = make_float2(st.o[n][i][c], st.o[n][i][c + 2]);
            if (g == 0) {
                s_m[warp][h] = st.mu[n][c];
                s_l[warp][h] = l[n][c];
                // 1 / vf
                if constexpr (!kFp4)
                    s_v[warp][h] = st.vf[n][c] == INFINITY ? 1.f : __uint_as_float((254u << 23) - __float_as_uint(st.vf[n][c]));
            }
        }
    __syncthreads();
    const size_t pair = static_cast<size_t>(seq) * a.hkv + kvh;
    if (threadIdx.x < G) {
        // per head: the warps' weights 2^(mu_w - M) / L, V's scale folded in,
        // replace s_m; the chunk's lse goes to s_l[0]
        const int h = threadIdx.x;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
        float f[kWarps], L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            f[w] = s_m[w][h] == -INFINITY ? 0.f : fast_exp2(s_m[w][h] - M);
            L += f[w] * s_l[w][h];
        }
        float lse = L != 0.f ? M * 0.6931471805599453f + logf(L) : -INFINITY;
        float inv = L != 0.f ? (kFp4 ? a.v_scale[kvh] : 1.f) / L : 0.f;
        if (a.sinks && nsplit == 1) {
            // lse' = ln(e^lse + e^sink), o scaled by e^(lse - lse')
            const float sk = a.sinks[kvh * G + h];
            const float hi = fmaxf(lse, sk);
            const float both = hi == -INFINITY ? hi : hi + logf(expf(lse - hi) + expf(sk - hi));
            if (lse != -INFINITY) inv *= expf(lse - both);
            lse = both;
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s_m[w][h] = f[w] == 0.f ? 0.f : f[w] * inv * (kFp4 ? 1.f : s_v[w][h]);
        s_l[0][h] = lse;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * (D / 4); i += kThreads) {
        const int h = i / (D / 4), d = 4 * (i % (D / 4));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float wt = s_m[w][h];
            const float4 x = *reinterpret_cast<const float4*>(comb + (w * C::kHeads + h) * C::kCombStride + d);
            v.x += wt * x.x;
            v.y += wt * x.y;
            v.z += wt * x.z;
            v.w += wt * x.w;
        }
        if (nsplit == 1) {
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (head0 + h) * D + d) =
                make_uint2(pack2<false>(v.x, v.y), pack2<false>(v.z, v.w));
            if (a.lse_out && d == 0) a.lse_out[head0 + h] = s_l[0][h];
        } else if (kCluster) {  // the chunk's state stays here, in place of warp 0's rows
            *reinterpret_cast<float4*>(comb + h * C::kCombStride + d) = v;
        } else {
            const size_t prow = (pair * a.max_splits + split) * G + h;
            *reinterpret_cast<float4*>(a.part_o + prow * D + d) = v;
            if (d == 0) a.part_lse[prow] = s_l[0][h];
        }
    }
    if constexpr (kCluster)
        if (nsplit > 1) merge_cluster<D, kFp4, NT>(a, comb, s_l[0], split, kvh, head0, nsplit);
}

// ------------------------------------------------------------- merge --
//
// The chunks' states of kHeads query heads of one (sequence, KV head) -> their output
// rows.  kHeads * D / 4 threads hold a float4 column each; where that is less than the
// CTA, thread groups take every kGroups-th chunk and meet in shared memory in a fixed
// order.  8 chunks' loads are in flight beside the lse.
template <int D, int kHeads>
__global__ void __launch_bounds__(kThreads) quant_merge_kernel(const __grid_constant__ QuantDecodeArgs a) {
    constexpr int kCols = D / 4, kWide = kHeads * kCols, kGroups = kThreads / kWide;
    static_assert(kWide <= kThreads && kThreads % kWide == 0, "whole thread groups");
    __shared__ float wts[kHeads][kQuantMaxSplits];
    __shared__ float s_inv[kHeads];
    __shared__ float4 s_sum[kGroups > 1 ? kThreads : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = (a.group + kHeads - 1) / kHeads;  // CTAs per (sequence, KV head)
    const int kvh = blockIdx.x / blocks, g0 = blockIdx.x % blocks * kHeads, seq = blockIdx.y;
    const int heads = min(kHeads, a.group - g0);
    const size_t row0 = static_cast<size_t>(seq) * a.hq + kvh * a.group + g0;
    // the lengths and sinks are older than the launch this one follows, which started
    // only after its own predecessors: they are read before the wait for it
    const int ctx = min(a.context_lens[seq], a.max_ctx);
    const int lo = a.window > 0 && ctx > a.window ? ctx - a.window : 0;
    const int nsplit = ctx <= 0 ? 1 : ((ctx - 1) / kBlockSize - lo / kBlockSize + a.chunk_blocks) / a.chunk_blocks;
    pdl_wait();
    pdl_launch_dependents();
    if (nsplit == 1) return;  // its chunk wrote the output
    const size_t part = (static_cast<size_t>(seq) * a.hkv + kvh) * a.max_splits * a.group + g0;
    // this thread's column; heads past the group read the last one's and write nothing
    const int col = threadIdx.x % kWide, h = min(col / kCols, heads - 1), first = threadIdx.x / kWide;
    const float4* po = reinterpret_cast<const float4*>(a.part_o + (part + h) * D) + col % kCols;
    const size_t step = static_cast<size_t>(a.group) * kCols;
    float4 x[8];
    auto fetch = [&](int c0) {
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = po[min(c0 + u * kGroups, nsplit - 1) * step];
    };
    fetch(first);
    for (int i = warp; i < heads; i += kWarps) {
        constexpr int kPer = kQuantMaxSplits / 32;
        const float sk = a.sinks ? a.sinks[kvh * a.group + g0 + i] : -INFINITY;
        float l[kPer], M = sk;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int c = lane + 32 * u;
            l[u] = c < nsplit ? a.part_lse[part + static_cast<size_t>(c) * a.group + i] : -INFINITY;
        }
#pragma unroll
        for (int u = 0; u < kPer; ++u) M = fmaxf(M, l[u]);
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, s));
        float W = 0.f;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            if (32 * u >= nsplit) break;
            const float w = l[u] == -INFINITY ? 0.f : expf(l[u] - M);
            wts[i][lane + 32 * u] = w;
            W += w;
        }
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) W += __shfl_xor_sync(0xFFFFFFFFu, W, s);
        if (sk != -INFINITY) W += expf(sk - M);
        if (lane == 0) {
            s_inv[i] = W != 0.f ? 1.f / W : 0.f;
            if (a.lse_out) a.lse_out[row0 + i] = W != 0.f ? M + logf(W) : -INFINITY;
        }
    }
    __syncthreads();
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = first; c0 < nsplit;) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int c = c0 + u * kGroups;
            const float w = c < nsplit ? wts[h][c] : 0.f;
            v.x += w * x[u].x;
            v.y += w * x[u].y;
            v.z += w * x[u].z;
            v.w += w * x[u].w;
        }
        c0 += 8 * kGroups;
        if (c0 < nsplit) fetch(c0);
    }
    if constexpr (kGroups > 1) {
        s_sum[threadIdx.x] = v;
        __syncthreads();
        if (first > 0) return;
#pragma unroll
        for (int i = 1; i < kGroups; ++i) {
            const float4 y = s_sum[i * kWide + col];
            v.x += y.x;
            v.y += y.y;
            v.z += y.z;
            v.w += y.w;
        }
    }
    if (col / kCols >= heads) return;
    const float inv = s_inv[h];
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (row0 + h) * D + 4 * (col % kCols)) =
        make_uint2(pack2<false>(v.x * inv, v.y * inv), pack2<false>(v.z * inv, v.w * inv));
}

template <int D>
cudaError_t launch_merge_states(const QuantDecodeArgs& a, cudaStream_t stream) {
    // a head per CTA while all of them are resident at once; the widest CTAs beyond
    constexpr int kMost = 4 * kThreads / D;
    if (static_cast<long long>(a.num_seqs) * a.hq <= 152 * 16)
        return launch_pdl(quant_merge_kernel<D, 1>, dim3(a.hq, a.num_seqs), dim3(kThreads), 0, stream, a);
    return launch_pdl(quant_merge_kernel<D, kMost>, dim3(a.hkv * ((a.group + kMost - 1) / kMost), a.num_seqs), dim3(kThreads), 0,
                      stream, a);
}

template <int D, bool kFp4, int NT, bool kCluster>
cudaError_t launch_t(const QuantDecodeArgs& a, cudaStream_t stream) {
    using C = Cfg<D, kFp4, NT>;
    static_assert(C::kSmem <= 227 * 1024, "shared memory budget");
    static_assert((kQuantCluster + 1) * 16 <= C::kHeads * C::kCombStride, "cluster merge weights");
    auto kern = quant_decode_kernel<D, kFp4, NT, kCluster>;
    // a per-device function attribute, set on the first launch on each device
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    e = launch_pdl_cluster(kern, dim3(a.max_splits, a.hkv, a.num_seqs), dim3(kThreads), C::kSmem, stream,
                           kCluster ? static_cast<unsigned>(a.max_splits) : 1u, a);
    if (e != cudaSuccess || kCluster || a.max_splits == 1) return e;
    return launch_merge_states<D>(a, stream);
}

template <int D, bool kFp4>
cudaError_t launch_g(const QuantDecodeArgs& a, cudaStream_t stream) {
    if (a.cluster) return a.group <= 8 ? launch_t<D, kFp4, 1, true>(a, stream) : launch_t<D, kFp4, 2, true>(a, stream);
    return a.group <= 8 ? launch_t<D, kFp4, 1, false>(a, stream) : launch_t<D, kFp4, 2, false>(a, stream);
}

}  // namespace

int quant_decode_ctas(int d, int group) {
    const bool two = group > 8;
    if (d == 64) return two ? Cfg<64, true, 2>::kCtas : Cfg<64, true, 1>::kCtas;
    return two ? Cfg<128, true, 2>::kCtas : Cfg<128, true, 1>::kCtas;
}

cudaError_t launch_quant_decode(const QuantDecodeArgs& a, cudaStream_t stream) {
    if (a.d == 64) return a.fp4 ? launch_g<64, true>(a, stream) : launch_g<64, false>(a, stream);
    return a.fp4 ? launch_g<128, true>(a, stream) : launch_g<128, false>(a, stream);
}

}  // namespace pkv
