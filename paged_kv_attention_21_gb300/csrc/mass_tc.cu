// mass_tc.cu -- the weight that each cached key receives from many queries, on the
// 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
// S^T = K Q^T with 128 keys as the rows of the MMA and up to 256 query rows (query
// token x head of the KV group) as its columns: a thread of the epilogue owns one key
// (its TMEM lane), so a key's sum over the queries is a sum over columns in one
// register, and the same constants (a query's lse) serve all lanes of a warp.
//
// One CTA owns consecutive tiles of 128 keys of one (sequence, KV head) and takes them two
// at a time over the steps of 256 query rows that see them: a step's 64 KB of q come from
// L2 once for 256 keys (one tile at a time was bound by those reads).  Warps:
//   0      TMA: the key tiles (two stages), the query steps (two stages; at most two
//          steps stay where they are, and a single one leaves its second stage's place
//          to more key tiles in flight), and each step's constants per query row;
//   1      MMA issuer: S of (step, tile) into the tile's TMEM buffer of 256 columns;
//   2..17  epilogue: 2^(x - lse) summed over the columns; eight warps for each tile of
//          the pair, four for each half of a step's columns, 32 at a time.
// e4m3 codes become bf16 in shared memory (exactly; the epilogue's warps convert a
// tile as it lands), so that q stays as it is.
#include "mass.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kMtKeys = 128;                      // keys per tile
constexpr int kMtBlocks = kMtKeys / kBlockSize;
constexpr int kMtCols = 256;                      // query rows per step: two tiles of 128
constexpr int kMtEpiWarps = 16;
constexpr int kMtThreads = (2 + kMtEpiWarps) * 32;

template <int D, bool kFp8>
struct MtCfg {
    static constexpr int kHalves = D / 64;               // 64-column (128-byte) slices of a row
    static constexpr int kKBytes = kMtKeys * D * 2;
    static constexpr int kBlkBytes = kBlockSize * D * 2;
    static constexpr int kGrpBytes = kHalves * 1024;     // between 8-row groups of a key tile
    static constexpr int kQHalf = kMtCols * 128;         // one 64-column slice of a step
    static constexpr int kQBytes = kHalves * kQHalf;
    static constexpr int kRawBytes = kFp8 ? kMtKeys * D : 0;  // e4m3: a tile of codes
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + 2 * kQBytes;
    static constexpr int kOffRaw = kOffK + 2 * kKBytes;
    static constexpr int kBody = kOffRaw + kRawBytes;
    // stages of key tiles and (e4m3) of codes, with one query step or more; those
    // beyond the first two (one) lie in the second query stage
    static constexpr int kMaxK = kFp8 ? 2 : 4;
    static constexpr int kMaxRaw = kFp8 ? 4 : 1;
    __device__ static uint32_t k_stage(int i) { return i < 2 ? kOffK + i * kKBytes : kOffQ + kQBytes + (i - 2) * kKBytes; }
    __device__ static uint32_t raw_stage(int i) { return i < 1 ? kOffRaw : kOffQ + kQBytes + (i - 1) * kRawBytes; }
    // at least 120 KB, so that one CTA has an SM and its 512 TMEM columns
    static constexpr int kSmemBytes = kBody + 1024 > 120 * 1024 ? kBody + 1024 : 120 * 1024;
};

// What the epilogue needs of a step's query rows, by column.
struct MtRows {
    float neg_lse[kMtCols];   // -log2(e) lse; -inf: the row adds nothing
    float slope[kMtCols];     // log2 units
    float tok[kMtCols];       // token index
    int2 span[kMtCols];       // the keys [x, y] that it sees; [0, -1]: no such row
    int4 chunk[kMtCols / 32]; // of 32 columns: keys [x, y] that all see, [z, w] outside of which none does
};

// The weights of 32 columns, all seen by this key, without a bias, summed.
template <bool kCap>
__device__ __forceinline__ float sum_seen(const float (&v)[32], const float* neg_lse, uint64_t scl, const TanhPair& tp) {
    uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
    for (int u = 0; u < 16; u += 2) {
        const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(neg_lse + 2 * u);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const uint64_t s = pack_f32x2(v[2 * (u + w)], v[2 * (u + w) + 1]);
            const uint64_t n = w ? nl.y : nl.x;
            const uint64_t e = kCap ? tp(s, n) : fma_f32x2(s, scl, n);
            float x0, x1;
            unpack_f32x2(e, x0, x1);
            acc[w] = add_f32x2(acc[w], pack_f32x2(fast_exp2(x0), fast_exp2(x1)));
        }
    }
    float a0, a1;
    unpack_f32x2(add_f32x2(acc[0], acc[1]), a0, a1);
    return a0 + a1;
}

// The weights of 32 columns, of which this key (tf: its distance to the first query) may
// be hidden from some.  poly: the polynomial holds for every score of the warp.
__device__ __forceinline__ float sum_edge(const float (&v)[32], const MtRows& q, int c0, const ScoreScale& sc,
                                          const TanhPair& tp, bool poly, bool biased, float tf, int t) {
    float x[32];
    if (poly && sc.out > 0.f) {
#pragma unroll
        for (int e = 0; e < 32; e += 2)
            unpack_f32x2(tp(pack_f32x2(v[e], v[e + 1]), pack_f32x2(q.neg_lse[c0 + e], q.neg_lse[c0 + e + 1])), x[e], x[e + 1]);
    } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = sc(v[e], q.neg_lse[c0 + e]);
    }
    float part[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        const int c = c0 + e;
        float z = x[e];
        if (biased) z = fmaf(-q.slope[c], fabsf(q.tok[c] - tf), z);
        const float w = fast_exp2(z);
        const int2 sp = q.span[c];
        part[e & 1] += t >= sp.x && t <= sp.y ? w : 0.f;
    }
    return part[0] + part[1];
}

// A tile's codes to bf16, exactly, by the epilogue's threads, in the layout that the
// tile-group box writes: a block's rows in 8-row groups of 128-byte slices, 16-byte
// chunks swizzled by the row.
template <int D>
__device__ __forceinline__ void convert_keys(const uint8_t* raw, uint8_t* dst, int thread) {
    using C = MtCfg<D, true>;
    constexpr int kCh = D / 8;  // chunks of 8 dims of a row
#pragma unroll 2
    for (int i = thread; i < kMtKeys * kCh; i += kMtEpiWarps * 32) {
        const int row = i / kCh, ch = i % kCh, r8 = row & 7;
        const uint2 w = *reinterpret_cast<const uint2*>(raw + row * D + ch * 8);
        uint32_t f[4];
        e4m3x4_to_f16x4(w.x, f[0], f[1]);
        e4m3x4_to_f16x4(w.y, f[2], f[3]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&f[u]));
            f[u] = pack2<false>(p.x, p.y);
        }
        *reinterpret_cast<uint4*>(dst + (row >> 4) * C::kBlkBytes + ((row >> 3) & 1) * C::kGrpBytes + (ch >> 3) * 1024 +
                                  r8 * 128 + (((ch & 7) ^ r8) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
    }
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kMtThreads, 1)
    mass_tc_kernel(const MassArgs a, const int tiles_per_cta, const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap) {
    using C = MtCfg<D, kFp8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    __shared__ __align__(16) MtRows rows[2];
    __shared__ float s_part[2][2][kMtKeys];
    __shared__ __align__(8) uint64_t bar_raw[C::kMaxRaw], bar_raw_empty[C::kMaxRaw];
    __shared__ __align__(8) uint64_t bar_k[C::kMaxK], bar_k_empty[C::kMaxK];
    __shared__ __align__(8) uint64_t bar_q[2], bar_s[2], bar_s_empty[2], bar_step[2], bar_fin;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    pdl_wait();
    pdl_launch_dependents();
    const int seq = blockIdx.z, kvh = blockIdx.y, G = a.group, QT = a.q_tile;
    const MassSeq s = mass_seq(a, seq, blockIdx.x == 0 && threadIdx.x == 0 && kvh == 0);
    const int ntiles = s.ok ? (s.kv_len + kMtKeys - 1) / kMtKeys : 0;
    const int tile0 = static_cast<int>(blockIdx.x) * tiles_per_cta;
    const int tile1 = min(ntiles, tile0 + tiles_per_cta);
    if (tile0 >= tile1) return;
    const int ntok = s.rows / G;
    const int per_step = 2 * QT;
    const int nsteps_all = (ntok + per_step - 1) / per_step;
    const bool resident = nsteps_all <= 2;
    const int nk = nsteps_all <= 1 ? C::kMaxK : 2, nraw = nsteps_all <= 1 ? C::kMaxRaw : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kMaxRaw; ++i) {
            mbar_init(&bar_raw[i], 1);
            mbar_init(&bar_raw_empty[i], kMtEpiWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar_q[i], 2);  // the copies, and the rows' constants
            mbar_init(&bar_s[i], 1);
            mbar_init(&bar_s_empty[i], kMtEpiWarps / 2);
            mbar_init(&bar_step[i], kMtEpiWarps);
        }
        for (int i = 0; i < C::kMaxK; ++i) {
            mbar_init(&bar_k[i], kFp8 ? kMtEpiWarps : 1);
            mbar_init(&bar_k_empty[i], 1);
        }
        mbar_init(&bar_fin, 1);
        s_fail = 0;
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
    }
    if (warp == 1) {
        tc::tmem_alloc(&s_tmem, 512);
        tc::tmem_relinquish();
    }
    fence_barrier_init();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    const volatile int* abort = &s_fail;
    const int32_t* bt = a.block_tables + static_cast<size_t>(seq) * a.mbps;

    // the steps [lo, hi) that see the pair of key tiles kt, kt + 1; how many of these there are
    auto steps_of = [&](int kt, int& lo, int& hi) {
        const int nt = min(2, tile1 - kt);
        int first, last;
        mass_tokens(a, s, ntok, kt * kMtKeys, min((kt + nt) * kMtKeys, s.kv_len) - 1, first, last);
        const bool some = last >= first;
        lo = some && nsteps_all > 1 ? first / per_step : 0;
        hi = !some ? 0 : nsteps_all > 1 ? last / per_step + 1 : 1;
        return nt;
    };
    // keys outside of these are seen by no query: their blocks may be any
    int seen_lo, seen_hi;
    mass_seen(a, s, ntok, seen_lo, seen_hi);
    auto block_seen = [&](int blk) { return blk * kBlockSize <= seen_hi && blk * kBlockSize + kBlockSize > seen_lo; };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int nload = 0;      // key tiles loaded
        int step = 0;       // steps begun, as the MMA warp and the epilogue count them
        bool ok = true;
        int nq[2] = {0, 0};   // loads of each query stage
        // this lane's rows of a 128-row tile: token and head of r = lane + 32 i
        int row_tok[4], row_head[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            row_tok[i] = (lane + 32 * i) / G;
            row_head[i] = (lane + 32 * i) % G;
        }
        auto load_q = [&](int qs, int st) {
            const int t0 = qs * per_step;
            const int nt = ntok - t0 > QT ? 2 : 1;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar_q[st], nt * C::kHalves * 64 * 2 * G * QT);
                for (int x = 0; x < nt; ++x)
                    for (int h = 0; h < C::kHalves; ++h)
                        tma_load_3d(smem + C::kOffQ + st * C::kQBytes + h * C::kQHalf + x * (128 * 128), &qmap,
                                    &bar_q[st], h * 64, kvh * G, s.q0 + t0 + x * QT);
            }
#pragma unroll
            for (int i = 0; i < kMtCols / 32; ++i) {
                const int c = lane + 32 * i;
                const int tok = t0 + (i >> 2) * QT + row_tok[i & 3];
                const bool real = row_tok[i & 3] < QT && tok < ntok;
                float nl = -INFINITY, slope = 0.f;
                int lo = 0, hi = -1;
                if (real) {
                    const int h = kvh * G + row_head[i & 3];
                    const float lse = a.lse[static_cast<size_t>(s.q0 + tok) * a.hq + h];
                    nl = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
                    if (a.slopes) slope = a.slopes[h] * kLog2e;
                    mass_span(a, s, s.off + tok, lo, hi);
                }
                rows[st].neg_lse[c] = nl;
                rows[st].slope[c] = slope;
                rows[st].tok[c] = static_cast<float>(tok);
                rows[st].span[c] = make_int2(lo, hi);
                const int all_lo = __reduce_max_sync(0xFFFFFFFFu, lo), all_hi = __reduce_min_sync(0xFFFFFFFFu, hi);
                const int any_lo = __reduce_min_sync(0xFFFFFFFFu, real ? lo : INT32_MAX);
                const int any_hi = __reduce_max_sync(0xFFFFFFFFu, hi);
                if (lane == 0) rows[st].chunk[i] = make_int4(all_lo, all_hi, any_lo, any_hi);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_q[st]);
            ++nq[st];
        };
        if (resident)
            for (int qs = 0; qs < nsteps_all; ++qs) load_q(qs, qs);
        // block ids: lane l has block l % 8 of tile l / 8 of a group of four tiles; the next
        // group's are read one group ahead
        const int nblk = (s.kv_len + kBlockSize - 1) / kBlockSize;
        auto read_ids = [&](int grp) {
            const int blk = (tile0 + 4 * grp) * kMtBlocks + lane;
            return blk < min(nblk, tile1 * kMtBlocks) && block_seen(blk) ? __ldg(bt + blk) : 0;
        };
        auto check_ids = [&](int id) {
            if (id < 0 || id >= a.num_blocks) {
                flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                id = 0;  // read a valid block; the keys' weights are not written
            }
            return id;
        };
        int ids_grp = 0, ids = check_ids(read_ids(0)), ids_next = read_ids(1);
        auto load_keys = [&](int kt) {
            while (ids_grp < (kt - tile0) >> 2) {
                ids = check_ids(ids_next);
                ids_next = read_ids(++ids_grp + 1);
            }
            const int id = __shfl_sync(0xFFFFFFFFu, ids, ((kt - tile0) & 3) * kMtBlocks + (lane & (kMtBlocks - 1)));
            const int nvalid = min(kMtBlocks, nblk - kt * kMtBlocks);
            if constexpr (kFp8) {
                const int st = nload % nraw;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bar_raw_empty[st], ((nload / nraw) & 1) ^ 1, kWaitLimitNs, abort)))
                    return false;
                if (lane == 0) mbar_arrive_expect_tx(&bar_raw[st], nvalid * (C::kBlkBytes / 2));
                __syncwarp();
                if (lane < nvalid)
                    tma_load_4d(smem + C::raw_stage(st) + lane * (C::kBlkBytes / 2), &kmap, &bar_raw[st], 0, 0, kvh, id);
            } else {
                const int st = nload % nk;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bar_k_empty[st], ((nload / nk) & 1) ^ 1, kWaitLimitNs, abort)))
                    return false;
                if (lane == 0) mbar_arrive_expect_tx(&bar_k[st], nvalid * C::kBlkBytes);
                __syncwarp();
                if (lane < nvalid)
                    tma_load_5d(smem + C::k_stage(st) + lane * C::kBlkBytes, &kmap, &bar_k[st], 0, 0, 0, 0, id * a.hkv + kvh);
            }
            ++nload;
            return true;
        };
        for (int kt = tile0; ok && kt < tile1; kt += 2) {
            int lo, hi;
            const int nt = steps_of(kt, lo, hi);
            if (lo >= hi) continue;  // no query sees them: nothing of them is read
            ok = load_keys(kt);
            if (resident) {
                if (ok && nt > 1) ok = load_keys(kt + 1);
                continue;
            }
            for (int qs = lo; ok && qs < hi; ++qs, ++step) {
                // the stage's last step has been read from TMEM for the pair's last tile, which every
                // step has an arrival of: its MMAs and its constants are done with
                const int st = step & 1;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_step[st], ((step >> 1) & 1) ^ 1, kWaitLimitNs, abort));
                if (ok) load_q(qs, st);
                if (ok && qs == lo && nt > 1) ok = load_keys(kt + 1);
            }
        }
        if (!ok && lane == 0) atomicOr(&s_fail, 1);
        // drain: every copy issued has landed before this CTA exits
        for (int i = 0; i < 2; ++i)
            if (nq[i] > 0) (void)mbar_wait(&bar_q[i], (nq[i] - 1) & 1);
        if constexpr (kFp8) {
            for (int j = max(0, nload - nraw); j < nload; ++j) (void)mbar_wait(&bar_raw[j % nraw], (j / nraw) & 1);
        } else {
            for (int j = max(0, nload - nk); j < nload; ++j) (void)mbar_wait(&bar_k[j % nk], (j / nk) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer
        constexpr uint32_t kWide = tc::idesc_bf16_f32(kMtKeys, 256, false, false);
        constexpr uint32_t kHalf = tc::idesc_bf16_f32(kMtKeys, 128, false, false);
        int nload = 0, step = 0, used[2] = {0, 0};  // S buffer x: times used
        bool ok = true;
        for (int kt = tile0; ok && kt < tile1; kt += 2) {
            int lo, hi;
            const int nt = steps_of(kt, lo, hi);
            for (int qs = lo; ok && qs < hi; ++qs, ++step) {
                const int st = resident ? qs : step & 1;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_q[st], resident ? 0 : (step >> 1) & 1, kWaitLimitNs, abort));
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!ok || x >= nt) break;
                    const int ks = (nload + x) % nk;
                    bool r = qs > lo || mbar_wait(&bar_k[ks], ((nload + x) / nk) & 1, kWaitLimitNs, abort);
                    r = r && mbar_wait(&bar_s_empty[x], (used[x] & 1) ^ 1, kWaitLimitNs, abort);
                    ok = __all_sync(0xFFFFFFFFu, r);
                    if (!ok) break;
                    ++used[x];
                    tc::fence_after_sync();
                    if (lane == 0) {
                        const uint32_t idesc = ntok - qs * per_step > QT ? kWide : kHalf;
                        const uint32_t sk = smem_u32(smem + C::k_stage(ks));
                        const uint32_t sq = smem_u32(smem + C::kOffQ + st * C::kQBytes);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const int h = kk >> 2;
                            const uint32_t ko = (kk & 3) * 32;
                            const uint64_t ad = tc::smem_desc(sk + h * 1024 + ko, 16, C::kGrpBytes);
                            const uint64_t bd = tc::smem_desc(sq + h * C::kQHalf + ko, 16, 1024);
                            tc::mma_bf16(tmem + x * kMtCols, ad, bd, idesc, kk > 0 ? 1u : 0u);
                        }
                        tc::commit(&bar_s[x]);
                        if (qs == hi - 1) tc::commit(&bar_k_empty[ks]);
                    }
                    __syncwarp();
                }
            }
            if (lo < hi) nload += nt;
        }
        if (!ok && lane == 0) {
            flag_error(a.err, PKV_DEVERR_TIMEOUT);
            atomicOr(&s_fail, 1);
        }
        // drain: every MMA is complete before TMEM is freed
        if (lane == 0) tc::commit(&bar_fin);
        __syncwarp();
        (void)mbar_wait(&bar_fin, 0);
        tc::fence_after_sync();
    } else {
        // ------------------------------------------------------------ epilogue
        const int ew = warp - 2, x = ew >> 3, second = (ew >> 2) & 1;  // tile of the pair, half of the columns
        const int key = (warp & 3) * 32 + lane;  // the TMEM lane this thread may read
        const uint32_t s_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + x * kMtCols;
        const ScoreScale sc(a.sm_scale, a.cap, kFp8 ? a.k_scale[kvh] : 1.f);
        const bool capped = sc.out > 0.f, biased = a.slopes != nullptr;
        const TanhPair tp(sc);
        const uint64_t scl = pack_f32x2(sc.in, sc.in);
        float* mrow = a.mass + (static_cast<size_t>(seq) * a.hkv + kvh) * a.mass_stride;
        int nload = 0, step = 0, turn = 0, used = 0;
        bool ok = true, q_here = false;
        for (int kt = tile0; kt < tile1; kt += 2, ++turn) {
            int slo, shi;
            const int nt = steps_of(kt, slo, shi);
            const int k0 = (kt + x) * kMtKeys, t = k0 + key;
            const int k_last = min(k0 + kMtKeys, s.kv_len) - 1;
            float old = 0.f, sum = 0.f;
            int id = 0;
            const bool mine = !second && t < s.kv_len && x < nt;
            if (mine) {
                if (a.keep != 0.f && t < s.off) old = a.keep * mrow[t];
                if (slo < shi && block_seen(t / kBlockSize)) id = bt[t / kBlockSize];
            }
            if constexpr (kFp8) {
                for (int y = 0; ok && slo < shi && y < nt; ++y) {
                    const int rs = nload % nraw, ks = nload % nk;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_raw[rs], (nload / nraw) & 1, kWaitLimitNs, abort) &&
                                                     mbar_wait(&bar_k_empty[ks], ((nload / nk) & 1) ^ 1, kWaitLimitNs,
                                                               abort));
                    if (ok) {
                        convert_keys<D>(smem + C::raw_stage(rs), smem + C::k_stage(ks), ew * 32 + lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&bar_k[ks]);
                            mbar_arrive(&bar_raw_empty[rs]);
                        }
                        ++nload;
                    }
                }
            }
            for (int qs = slo; ok && qs < shi; ++qs, ++step) {
                const int st = resident ? qs : step & 1;
                // (warps without a tile in this pair wait too: their arrival on bar_step must not
                // run ahead of the step)
                if (!resident || !q_here)
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_q[st], resident ? 0 : (step >> 1) & 1, kWaitLimitNs, abort));
                if (!ok) break;
                if (x < nt) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_s[x], used & 1, kWaitLimitNs, abort));
                    if (!ok) break;
                    ++used;
                    tc::fence_after_sync();
                    const MtRows& q = rows[st];
                    const int cols = ntok - qs * per_step > QT ? 128 : 64;  // of this half
                    const int c_end = (second + 1) * cols;
                    for (int c = second * cols; c < c_end; c += 32) {
                        float v[32];
                        tc::ld32(s_base + c, v);
                        tc::wait_ld();
                        if (c + 32 == c_end) {
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar_s_empty[x]);
                        }
                        const int4 ch = q.chunk[c >> 5];
                        if (ch.z > k_last || ch.w < k0) continue;
                        const bool poly = !capped || __all_sync(0xFFFFFFFFu, in_poly(v, sc.in));
                        if (ch.x <= k0 && ch.y >= k_last && poly && !biased)
                            sum += capped ? sum_seen<true>(v, q.neg_lse + c, scl, tp)
                                          : sum_seen<false>(v, q.neg_lse + c, scl, tp);
                        else
                            sum += sum_edge(v, q, c, sc, tp, poly, biased, static_cast<float>(t - s.off), t);
                    }
                }
                __syncwarp();
                if (!resident && lane == 0) mbar_arrive(&bar_step[step & 1]);
            }
            q_here = q_here || (slo == 0 && shi == nsteps_all);
            if (!ok && lane == 0) atomicOr(&s_fail, 1);
            // the halves' sums meet; a warp that gave up comes here for every pair all the same
            if (second) s_part[turn & 1][x][key] = sum;
            asm volatile("bar.sync 1, %0;" ::"n"(kMtEpiWarps * 32) : "memory");
            if (mine && id >= 0 && id < a.num_blocks && *abort == 0) mrow[t] = old + (sum + s_part[turn & 1][x][key]);
        }
        if (!ok && lane == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D, bool kFp8>
cudaError_t launch_mass_tc_t(const MassArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap, cudaStream_t stream) {
    using C = MtCfg<D, kFp8>;
    static_assert(C::kSmemBytes <= 227 * 1024 - 14 * 1024, "shared memory: the arena, the rows' constants, the barriers");
    auto kern = mass_tc_kernel<D, kFp8>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const int tiles = (a.max_kv + kMtKeys - 1) / kMtKeys;
    const int steps = (a.max_q + 2 * a.q_tile - 1) / (2 * a.q_tile);
    // Pairs of tiles per CTA: about 16 (pair, step)s, as long as that leaves four CTAs an SM.
    const int64_t pairs = static_cast<int64_t>((tiles + 1) / 2) * a.hkv * a.num_seqs;
    int per = (16 + steps - 1) / steps;
    per = 2 * static_cast<int>(max(int64_t{1}, min(int64_t{per}, pairs / (4 * max(1, a.num_sms)))));
    const dim3 grid((tiles + per - 1) / per, a.hkv, a.num_seqs);
    return launch_pdl(kern, grid, dim3(kMtThreads), C::kSmemBytes, stream, a, per, qmap, kmap);
}

}  // namespace

cudaError_t launch_mass_tc(const MassArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap, cudaStream_t stream) {
    if (a.fp8)
        return a.d == 64 ? launch_mass_tc_t<64, true>(a, qmap, kmap, stream)
                         : launch_mass_tc_t<128, true>(a, qmap, kmap, stream);
    return a.d == 64 ? launch_mass_tc_t<64, false>(a, qmap, kmap, stream)
                     : launch_mass_tc_t<128, false>(a, qmap, kmap, stream);
}

}  // namespace pkv
