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
constexpr int kMassBlocksPerWarp = 4;

// Any number of rows: a warp holds a block's 16 keys as A operands and takes the
// rows eight at a time.  A lane reads 16-byte pieces of K and q and takes them as
// the k-steps' operands in the order they come (the dot product is a sum over dims).
template <int D, bool kFp8>
__global__ void __launch_bounds__(kMassWarps * 32) mass_rows_kernel(const MassArgs a) {
    constexpr int KSTEPS = D / 16;
    pdl_wait();
    pdl_launch_dependents();
    const int seq = blockIdx.z, kvh = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int G = a.group;
    const MassSeq s = mass_seq(a, seq, blockIdx.x == 0 && threadIdx.x == 0 && kvh == 0);
    if (!s.ok) return;
    const ScoreScale sc(a.sm_scale, a.cap, kFp8 ? a.k_scale[kvh] : 1.f);
    const int32_t* bt = a.block_tables + static_cast<size_t>(seq) * a.mbps;
    float* mrow = a.mass + (static_cast<size_t>(seq) * a.hkv + kvh) * a.mass_stride;
    const int nblk = (s.kv_len + kBlockSize - 1) / kBlockSize;
    int seen_lo, seen_hi;  // blocks that no query sees are not read
    mass_seen(a, s, s.rows / G, seen_lo, seen_hi);
    for (int i = 0; i < kMassBlocksPerWarp; ++i) {
        const int blk = (static_cast<int>(blockIdx.x) * kMassBlocksPerWarp + i) * kMassWarps + warp;
        if (blk >= nblk) return;
        const int t0 = blk * kBlockSize;
        float sum0 = 0.f, sum1 = 0.f;
        if (t0 <= seen_hi && t0 + kBlockSize > seen_lo) {
            int id = bt[blk];
            if (id < 0 || id >= a.num_blocks) {
                if (lane == 0) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                continue;  // these keys' weights stay as they are
            }
            uint32_t ka[KSTEPS][4];
            const size_t base = (static_cast<size_t>(id) * a.hkv + kvh) * kBlockSize * D;
            if constexpr (kFp8) {
                const uint8_t* kp = static_cast<const uint8_t*>(a.k_cache) + base;
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const uint4 u = *reinterpret_cast<const uint4*>(kp + g * D + (tig + 4 * j) * 16);
                    const uint4 v = *reinterpret_cast<const uint4*>(kp + (g + 8) * D + (tig + 4 * j) * 16);
                    const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        e4m3x4_to_f16x4(uw[w], ka[4 * j + w][0], ka[4 * j + w][2]);
                        e4m3x4_to_f16x4(vw[w], ka[4 * j + w][1], ka[4 * j + w][3]);
                    }
                }
            } else {
                const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(a.k_cache) + base;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const uint4 u = *reinterpret_cast<const uint4*>(kp + g * D + (tig + 4 * j) * 8);
                    const uint4 v = *reinterpret_cast<const uint4*>(kp + (g + 8) * D + (tig + 4 * j) * 8);
                    ka[2 * j][0] = u.x, ka[2 * j][1] = v.x, ka[2 * j][2] = u.y, ka[2 * j][3] = v.y;
                    ka[2 * j + 1][0] = u.z, ka[2 * j + 1][1] = v.z, ka[2 * j + 1][2] = u.w, ka[2 * j + 1][3] = v.w;
                }
            }
            for (int n0 = 0; n0 < s.rows; n0 += 8) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                const int n = n0 + g;
                const bool real = n < s.rows;
                const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) +
                                          (static_cast<size_t>(s.q0 + n / G) * a.hq + kvh * G + n % G) * D;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    // k-steps 2 j and 2 j + 1
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    const int at = kFp8 ? (tig + 4 * (j >> 1)) * 16 + (j & 1) * 8 : (tig + 4 * j) * 8;
                    if (real) w = *reinterpret_cast<const uint4*>(qp + at);
                    if constexpr (kFp8) {
                        w.x = pack2<true>(bf16_lo(w.x), bf16_hi(w.x));
                        w.y = pack2<true>(bf16_lo(w.y), bf16_hi(w.y));
                        w.z = pack2<true>(bf16_lo(w.z), bf16_hi(w.z));
                        w.w = pack2<true>(bf16_lo(w.w), bf16_hi(w.w));
                    }
                    mma_16816<kFp8>(acc, ka[2 * j], w.x, w.y);
                    mma_16816<kFp8>(acc, ka[2 * j + 1], w.z, w.w);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = n0 + 2 * tig + c;
                    if (r >= s.rows) continue;
                    const int h = kvh * G + r % G, pos = s.off + r / G;
                    const float lse = a.lse[static_cast<size_t>(s.q0 + r / G) * a.hq + h];
                    if (lse == -INFINITY) continue;
                    const float slope2 = a.slopes ? a.slopes[h] * kLog2e : 0.f;
                    int lo, hi;
                    mass_span(a, s, pos, lo, hi);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = t0 + g + 8 * e;
                        float x = sc(acc[2 * e + c], -lse * kLog2e);
                        if (a.slopes) x = fmaf(-slope2, fabsf(static_cast<float>(pos - t)), x);
                        const float w = fast_exp2(x);
                        if (t >= lo && t <= hi) {
                            if (e == 0) sum0 += w; else sum1 += w;
                        }
                    }
                }
            }
            sum0 += __shfl_xor_sync(0xFFFFFFFFu, sum0, 1);
            sum0 += __shfl_xor_sync(0xFFFFFFFFu, sum0, 2);
            sum1 += __shfl_xor_sync(0xFFFFFFFFu, sum1, 1);
            sum1 += __shfl_xor_sync(0xFFFFFFFFu, sum1, 2);
        }
        if (tig < 2) {
            const int t = t0 + g + 8 * tig;
            if (t < s.kv_len) {
                const float old = a.keep != 0.f && t < s.off ? a.keep * mrow[t] : 0.f;
                mrow[t] = old + (tig ? sum1 : sum0);
            }
        }
    }
}

template <int D, bool kFp8>
cudaError_t launch_mass_t(const MassArgs& a, cudaStream_t stream) {
    constexpr int per_cta = kMassWarps * kMassBlocksPerWarp;
    const int blocks = (a.max_kv + kBlockSize - 1) / kBlockSize;
    const dim3 grid((blocks + per_cta - 1) / per_cta, a.hkv, a.num_seqs);
    return launch_pdl(mass_rows_kernel<D, kFp8>, grid, dim3(kMassWarps * 32), 0, stream, a);
}

}  // namespace

cudaError_t launch_mass_rows(const MassArgs& a, cudaStream_t stream) {
    if (a.fp8) return a.d == 64 ? launch_mass_t<64, true>(a, stream) : launch_mass_t<128, true>(a, stream);
    return a.d == 64 ? launch_mass_t<64, false>(a, stream) : launch_mass_t<128, false>(a, stream);
}

}  // namespace pkv
