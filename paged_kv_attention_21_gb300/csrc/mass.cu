// mass.cu -- the attention weight that each cached key receives: for sequence s, KV
// head g and key t
//     mass[t] = keep mass[t] + sum over queries i and heads h of g, where i sees t,
//               of exp(x_{i,h,t} - lse[i][h]),
// x the logit under the score rule (score.cuh).
//
// The product K Q^T is taken with the keys as the rows of the MMA: a key's weights
// then sit in one lane's accumulators for every query, and the sum over the queries
// stays in registers.
#include "mass.cuh"

namespace pkv {

namespace {

constexpr int kMassWarps = 4;
constexpr int kMassMaxBlocks = 32;  // of a warp: a block id per lane

// One block's keys as they come from global memory: 16-byte pieces of rows g and g + 8.
template <int D, bool kFp8>
struct MassKeys {
    static constexpr int kPieces = kFp8 ? D / 64 : D / 32;  // of each row, for each lane
    uint4 lo[kPieces], hi[kPieces];
    __device__ __forceinline__ void load(const MassArgs& a, int id, int kvh, int g, int tig) {
        const size_t base = (static_cast<size_t>(id) * a.hkv + kvh) * (kBlockSize * D * (kFp8 ? 1 : 2) / 16);
        const uint4* p = static_cast<const uint4*>(a.k_cache) + base + tig;
        constexpr int row = D * (kFp8 ? 1 : 2) / 16;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            lo[j] = ld_stream(p + g * row + 4 * j);
            hi[j] = ld_stream(p + (g + 8) * row + 4 * j);
        }
    }
    // the A operand of k-step kk: piece j of a row holds the dims of the k-steps' lanes in order
    __device__ __forceinline__ void operand(int kk, uint32_t (&f)[4]) const {
        if constexpr (kFp8) {
            const uint4 u = lo[kk / 4], v = hi[kk / 4];
            const uint32_t x = kk % 4 == 0 ? u.x : kk % 4 == 1 ? u.y : kk % 4 == 2 ? u.z : u.w;
            const uint32_t y = kk % 4 == 0 ? v.x : kk % 4 == 1 ? v.y : kk % 4 == 2 ? v.z : v.w;
            e4m3x4_to_f16x4(x, f[0], f[2]);
            e4m3x4_to_f16x4(y, f[1], f[3]);
        } else {
            const uint4 u = lo[kk / 2], v = hi[kk / 2];
            f[0] = kk % 2 ? u.z : u.x;
            f[1] = kk % 2 ? v.z : v.x;
            f[2] = kk % 2 ? u.w : u.y;
            f[3] = kk % 2 ? v.w : v.y;
        }
    }
    static __device__ __forceinline__ uint4 ld_stream(const uint4* p) {
        uint4 v;
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p));
        return v;
    }
};

// At most 8 NT rows.  A warp holds all of them as B operands and takes its blocks one by
// one, a block's 16 keys as the A operand straight from global memory, the next block's
// on their way meanwhile.  A lane reads 16-byte pieces of K and q and takes them as the
// k-steps' operands in the order they come (the dot product is a sum over dims).
template <int D, bool kFp8, int NT>
__global__ void __launch_bounds__(kMassWarps * 32) mass_rows_kernel(const MassArgs a, const int per_warp) {
    constexpr int KSTEPS = D / 16;
    pdl_wait();
    pdl_launch_dependents();
    const int seq = blockIdx.z, kvh = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int G = a.group;
    const MassSeq s = mass_seq(a, seq, blockIdx.x == 0 && threadIdx.x == 0 && kvh == 0);
    if (!s.ok) return;
    const int nblk = (s.kv_len - 1) / kBlockSize + 1;
    // this warp's blocks: first, first + 4, ...
    const int first = static_cast<int>(blockIdx.x) * kMassWarps * per_warp + warp;
    const int mine = first < nblk ? min(per_warp, (nblk - 1 - first) / kMassWarps + 1) : 0;
    if (mine == 0) return;
    int seen_lo, seen_hi;  // blocks that no query sees are not read: their table entries may name none
    mass_seen(a, s, s.rows / G, seen_lo, seen_hi);
    const int32_t* bt = a.block_tables + static_cast<size_t>(seq) * a.mbps;
    auto block_seen = [&](int blk) { return mass_block_seen(blk, seen_lo, seen_hi); };
    int ids = -1;  // lane k: of the k-th block; -1 where the block is not read or not there
    bool bad = false;
    if (lane < mine && block_seen(first + kMassWarps * lane)) {
        ids = bt[first + kMassWarps * lane];
        bad = ids < 0 || ids >= a.num_blocks;
        if (bad) {
            flag_error(a.err, PKV_DEVERR_BLOCK_ID);
            ids = -1;
        }
    }
    const uint32_t bad_ids = __ballot_sync(0xFFFFFFFFu, bad);
    MassKeys<D, kFp8> next;
    const int id0 = __shfl_sync(0xFFFFFFFFu, ids, 0);
    if (id0 >= 0) next.load(a, id0, kvh, g, tig);

    // B operands: row 8 nt + g, and what the epilogue needs of rows 8 nt + 2 tig and + 1
    uint32_t qb[NT][KSTEPS][2];
    float neg_lse[NT][2], slope2[NT][2];
    int pos[NT][2], lo[NT][2], hi[NT][2];
    int all_lo = 0, all_hi = s.kv_len - 1;  // keys that every row sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = 8 * nt + g;
        const uint4* qp = static_cast<const uint4*>(a.q) +
                          (static_cast<size_t>(s.q0 + r / G) * a.hq + kvh * G + r % G) * (D / 8);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {  // k-steps 2 j and 2 j + 1
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (r < s.rows) w = qp[kFp8 ? (tig + 4 * (j >> 1)) * 2 + (j & 1) : tig + 4 * j];
            if constexpr (kFp8) {
                w.x = pack2<true>(bf16_lo(w.x), bf16_hi(w.x));
                w.y = pack2<true>(bf16_lo(w.y), bf16_hi(w.y));
                w.z = pack2<true>(bf16_lo(w.z), bf16_hi(w.z));
                w.w = pack2<true>(bf16_lo(w.w), bf16_hi(w.w));
            }
            qb[nt][2 * j][0] = w.x, qb[nt][2 * j][1] = w.y;
            qb[nt][2 * j + 1][0] = w.z, qb[nt][2 * j + 1][1] = w.w;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r2 = 8 * nt + 2 * tig + c;
            neg_lse[nt][c] = -INFINITY;
            slope2[nt][c] = 0.f;
            pos[nt][c] = lo[nt][c] = 0;
            hi[nt][c] = -1;
            if (r2 < s.rows) {
                const int h = kvh * G + r2 % G;
                const float lse = a.lse[static_cast<size_t>(s.q0 + r2 / G) * a.hq + h];
                if (a.slopes) slope2[nt][c] = a.slopes[h] * kLog2e;
                pos[nt][c] = s.off + r2 / G;
                if (lse != -INFINITY) {  // else the row sees no key: its q may hold anything
                    neg_lse[nt][c] = -lse * kLog2e;
                    mass_span(a, s, pos[nt][c], lo[nt][c], hi[nt][c]);
                }
            }
            all_lo = max(all_lo, lo[nt][c]);
            all_hi = min(all_hi, hi[nt][c]);  // (-1 with rows past the last: 0 times an infinite k is not taken)
        }
    }
    all_lo = __reduce_max_sync(0xFFFFFFFFu, all_lo);
    all_hi = __reduce_min_sync(0xFFFFFFFFu, all_hi);
    const ScoreScale sc(a.sm_scale, a.cap, kFp8 ? a.k_scale[kvh] : 1.f);
    float* mrow = a.mass + (static_cast<size_t>(seq) * a.hkv + kvh) * a.mass_stride;

    for (int k = 0; k < mine; ++k) {
        const MassKeys<D, kFp8> keys = next;
        const int id = __shfl_sync(0xFFFFFFFFu, ids, k);
        const int id_next = __shfl_sync(0xFFFFFFFFu, ids, (k + 1) & 31);
        if (k + 1 < mine && id_next >= 0) next.load(a, id_next, kvh, g, tig);
        const int t0 = (first + kMassWarps * k) * kBlockSize;
        const int t_mine = t0 + g + 8 * (tig & 1);  // lanes of tig 0 and 1 write
        float old = 0.f;
        if (a.keep != 0.f && tig < 2 && t_mine < s.off) old = a.keep * mrow[t_mine];
        float sum0 = 0.f, sum1 = 0.f;
        if (id >= 0) {
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KSTEPS; ++kk) {
                uint32_t f[4];
                keys.operand(kk, f);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_16816<kFp8>(acc[nt], f, qb[nt][kk][0], qb[nt][kk][1]);
            }
            const bool seen = all_lo <= t0 && all_hi >= min(t0 + (kBlockSize - 1), s.kv_len - 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = t0 + g + 8 * e;
                        float x = sc(acc[nt][2 * e + c], neg_lse[nt][c]);
                        if (a.slopes) x = fmaf(-slope2[nt][c], fabsf(static_cast<float>(pos[nt][c] - t)), x);
                        float w = fast_exp2(x);
                        if (!seen) w = t >= lo[nt][c] && t <= hi[nt][c] ? w : 0.f;
                        if (e == 0) sum0 += w;
                        else sum1 += w;
                    }
                }
            }
            sum0 += __shfl_xor_sync(0xFFFFFFFFu, sum0, 1);
            sum0 += __shfl_xor_sync(0xFFFFFFFFu, sum0, 2);
            sum1 += __shfl_xor_sync(0xFFFFFFFFu, sum1, 1);
            sum1 += __shfl_xor_sync(0xFFFFFFFFu, sum1, 2);
        }
        if (tig < 2 && t_mine < s.kv_len && !((bad_ids >> k) & 1u)) mrow[t_mine] = old + (tig ? sum1 : sum0);
    }
}

template <int D, bool kFp8, int NT>
cudaError_t launch_mass_rows_n(const MassArgs& a, cudaStream_t stream) {
    // blocks per warp: about one wave of four CTAs an SM, ragged lengths averaging half the longest
    const int64_t blocks = (a.max_kv - 1) / kBlockSize + 1;
    const double warps = 16.0 * max(1, a.num_sms);
    const double want = 0.55 * static_cast<double>(blocks) * a.hkv * a.num_seqs / warps;
    const int per_warp = static_cast<int>(min(static_cast<double>(kMassMaxBlocks), max(2.0, want + 1.0)));
    const int64_t per_cta = static_cast<int64_t>(kMassWarps) * per_warp;
    const dim3 grid(static_cast<unsigned>((blocks + per_cta - 1) / per_cta), a.hkv, a.num_seqs);
    return launch_pdl(mass_rows_kernel<D, kFp8, NT>, grid, dim3(kMassWarps * 32), 0, stream, a, per_warp);
}

template <int D, bool kFp8>
cudaError_t launch_mass_rows_t(const MassArgs& a, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(a.max_q) * a.group;
    return rows <= 8 ? launch_mass_rows_n<D, kFp8, 1>(a, stream)
         : rows <= 16 ? launch_mass_rows_n<D, kFp8, 2>(a, stream) : launch_mass_rows_n<D, kFp8, 4>(a, stream);
}

}  // namespace

cudaError_t launch_mass_rows(const MassArgs& a, cudaStream_t stream) {
    if (a.fp8) return a.d == 64 ? launch_mass_rows_t<64, true>(a, stream) : launch_mass_rows_t<128, true>(a, stream);
    return a.d == 64 ? launch_mass_rows_t<64, false>(a, stream) : launch_mass_rows_t<128, false>(a, stream);
}

}  // namespace pkv
