// mass_tc.cu -- the weight that each cached key receives from many queries, on the
// 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
// S^T = K Q^T with 128 keys as the rows of the MMA and 128 query rows (query token x head
// of the KV group) as its columns: a thread of the epilogue owns one key (its TMEM lane),
// so a key's sum over the queries is a sum over columns in one register, and the same
// constants (a query's lse) serve all lanes of a warp.
//
// One CTA per SM takes an equal part of the work, cut along (sequence, KV head, key tile)
// with a sequence's tiles weighted by its steps of 128 query rows; it goes, up to four tiles
// at a time, over the steps that see them: a step's 32 KB of q come from L2 once for 512 keys
// (one tile at a time was bound by those reads).  Warps:
//   0      TMA: the key tiles (four stages), the query steps (two stages; at most two
//          steps stay where they are), and each step's constants per query row;
//   1      MMA issuer: S of (step, tile) into the tile's TMEM buffer of 128 columns;
//   2..17  epilogue: 2^(x - lse) summed over the columns, 32 at a time; four warps for
//          each tile of the four, which meet no others.
// e4m3 codes become bf16 in shared memory (exactly; the epilogue's warps convert a
// tile as it lands), so that q stays as it is.
#include "mass.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kMtKeys = 128;                      // keys per tile
constexpr int kMtBlocks = kMtKeys / kBlockSize;
constexpr int kMtTiles = 4;                       // key tiles side by side
constexpr int kMtCols = 128;                      // query rows per step
constexpr int kMtEpiWarps = 4 * kMtTiles;
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
    static constexpr int kOffRaw = kOffK + kMtTiles * kKBytes;
    static constexpr int kBody = kOffRaw + kRawBytes;
    // stages of codes: one, or three where no sequence has more than one step: two then lie in
    // the second query stage (32 observers of 64 sequences: 40 us with one)
    static constexpr int kMaxRaw = 3;
    __device__ static uint32_t raw_stage(int i) { return i == 0 ? kOffRaw : kOffQ + kQBytes + (i - 1) * kRawBytes; }
    // at least 120 KB, so that one CTA has an SM and its 512 TMEM columns
    static constexpr int kSmemBytes = kBody + 1024 > 120 * 1024 ? kBody + 1024 : 120 * 1024;
};

// What a score rule asks of the epilogue: neither cap nor bias, a cap alone, a bias with or
// without a cap.
enum MtMode { kMtNone, kMtCap, kMtBias };

// What the epilogue needs of a step's query rows, by column.
struct MtRows {
    float neg_lse[kMtCols];   // -log2(e) lse; -inf: the row adds nothing
    float slope[kMtCols];     // log2 units
    float tok[kMtCols];       // token index
    int2 span[kMtCols];       // the keys [x, y] that it sees; [0, -1]: no such row, or none that counts
    int4 chunk[kMtCols / 32]; // of 32 columns: keys [x, y] that all see, [z, w] outside of which none does
};

// The weights of 32 columns, all seen by this key, without a bias, summed.
enum { kMtPlain, kMtNear, kMtPoly };  // no cap; every |y| <= kTanhNear, kTanhPoly
template <int kCap>
__device__ __forceinline__ float sum_seen(const float (&v)[32], const float* neg_lse, const ScoreScale& sc,
                                          const TanhPair& tp) {
    const uint64_t scl = pack_f32x2(sc.in, sc.in);
    uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
    for (int u = 0; u < 16; u += 2) {
        const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(neg_lse + 2 * u);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const uint64_t s = pack_f32x2(v[2 * (u + w)], v[2 * (u + w) + 1]);
            const uint64_t n = w ? nl.y : nl.x;
            const uint64_t e = kCap == kMtNear ? tp.near(s, n) : kCap == kMtPoly ? tp(s, n) : fma_f32x2(s, scl, n);
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
template <int kMode>
__device__ __forceinline__ float sum_edge(const float (&v)[32], const MtRows& q, int c0, const ScoreScale& sc,
                                          const TanhPair& tp, bool poly, float tf, int t) {
    float x[32];
    if (kMode != kMtNone && poly && sc.out > 0.f) {
#pragma unroll
        for (int e = 0; e < 32; e += 2)
            unpack_f32x2(tp(pack_f32x2(v[e], v[e + 1]), pack_f32x2(q.neg_lse[c0 + e], q.neg_lse[c0 + e + 1])), x[e], x[e + 1]);
    } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = kMode == kMtNone ? fmaf(v[e], sc.in, q.neg_lse[c0 + e]) : sc(v[e], q.neg_lse[c0 + e]);
    }
    float part[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        const int c = c0 + e;
        float z = x[e];
        if (kMode == kMtBias) z = fmaf(-q.slope[c], fabsf(q.tok[c] - tf), z);
        const float w = fast_exp2(z);
        const int2 sp = q.span[c];
        part[e & 1] += t >= sp.x && t <= sp.y ? w : 0.f;
    }
    return part[0] + part[1];
}

// A tile's codes to bf16, exactly, by the tile's four warps, in the layout that the
// tile-group box writes: a block's rows in 8-row groups of 128-byte slices, 16-byte
// chunks swizzled by the row.
template <int D>
__device__ __forceinline__ void convert_keys(const uint8_t* raw, uint8_t* dst, int thread) {
    using C = MtCfg<D, true>;
    constexpr int kCh = D / 8;  // chunks of 8 dims of a row
#pragma unroll 2
    for (int i = thread; i < kMtKeys * kCh; i += 128) {
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

// The cost of a sequence's key tiles, as the work is cut over the CTAs: a tile's steps, and
// what a tile costs without any.
struct MtCost {
    int tiles, weight;  // tiles per head; of a tile
    __device__ __forceinline__ MtCost(const MassSeq& s, int group, int per_step) {
        tiles = s.ok ? (s.kv_len - 1) / kMtKeys + 1 : 0;
        weight = 1 + 2 * ((s.rows / group + per_step - 1) / per_step);
    }
    __device__ __forceinline__ int64_t all(int hkv) const { return static_cast<int64_t>(tiles) * weight * hkv; }
};

// A CTA's part of the work: the tiles, in the order (sequence, head, tile), whose costs
// before them lie in [lo, hi) of the whole, taken up to four of a head at a time.  Every
// warp walks it by itself.
struct MtWalk {
    const MassArgs& a;
    int64_t base, hi, left;  // costs before the sequence and at the end; tiles of it to come
    int seq, kvh, tile, n, tiles, weight, per_step;  // now: n tiles from `tile` on
    MassSeq s;
    int ntok, nsteps, seen_lo, seen_hi;
    bool resident, fresh;  // fresh: the first ones of a (sequence, head)
    __device__ __forceinline__ MtWalk(const MassArgs& args, int seq0, int64_t base0, int64_t lo, int64_t hi_)
        : a(args), base(base0), hi(hi_), seq(seq0), n(0), per_step(args.q_tile), fresh(false), first_(true) {
        load();
        const int64_t item = (lo - base + weight - 1) / weight;  // hkv * tiles at most
        kvh = static_cast<int>(item / tiles);
        tile = static_cast<int>(item % tiles);
        left -= item;
    }
    __device__ __forceinline__ bool next() {
        fresh = first_;
        first_ = false;
        tile += n;
        if (tile == tiles) {
            tile = 0;
            ++kvh;
            fresh = true;
        }
        while (kvh == a.hkv) {  // (sequences without work have no tiles)
            base += static_cast<int64_t>(tiles) * weight * a.hkv;
            if (base >= hi || ++seq >= a.num_seqs) return false;
            load();
            kvh = tiles > 0 ? 0 : a.hkv;
            fresh = true;
        }
        if (left <= 0) return false;
        n = static_cast<int>(min(min(int64_t{kMtTiles}, left), int64_t{tiles - tile}));
        left -= n;
        return true;
    }
    // the steps [lo, hi) that see the tiles' keys
    __device__ __forceinline__ void steps(int& lo, int& hi_) const {
        const int k0 = tile * kMtKeys;
        int first, last;
        mass_tokens(a, s, ntok, k0, k0 + min(n * kMtKeys, s.kv_len - k0) - 1, first, last);
        const bool some = last >= first;
        lo = some && nsteps > 1 ? first / per_step : 0;
        hi_ = !some ? 0 : nsteps > 1 ? last / per_step + 1 : 1;
    }
    // blocks that no query sees are not read: their table entries may name none
    __device__ __forceinline__ bool block_seen(int blk) const {
        return mass_block_seen(blk, seen_lo, seen_hi);
    }

   private:
    bool first_;
    __device__ __forceinline__ void load() {
        s = mass_seq(a, seq, false);
        const MtCost c(s, a.group, per_step);
        tiles = c.tiles;
        weight = c.weight;
        left = (hi - base + weight - 1) / weight;
        ntok = s.rows / a.group;
        nsteps = (ntok + per_step - 1) / per_step;
        resident = nsteps <= 2;
        mass_seen(a, s, ntok, seen_lo, seen_hi);
    }
};

// Which stage the next step's (or a resident segment's) rows of q are in, as the producer,
// the MMA warp and the epilogue each count it: uses[i] loads of stage i so far.
struct MtStages {
    int uses[2] = {0, 0}, turn = 0;
    __device__ __forceinline__ int parity(int st) const { return (uses[st] - 1) & 1; }
};

template <int D, bool kFp8, int kMode>
__global__ void __launch_bounds__(kMtThreads, 1)
    mass_tc_kernel(const MassArgs a, const int raw_stages, const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap) {
    using C = MtCfg<D, kFp8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    __shared__ __align__(16) MtRows rows[2];
    __shared__ __align__(8) uint64_t bar_raw[kMtTiles], bar_conv[kMtTiles], bar_q[2], bar_step[2], bar_fin;
    __shared__ __align__(8) uint64_t bar_k[kMtTiles], bar_k_empty[kMtTiles], bar_s[kMtTiles], bar_s_empty[kMtTiles];
    __shared__ int64_t s_cost[kMtThreads / 32];
    __shared__ int64_t s_base;
    __shared__ int s_seq;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    pdl_wait();
    pdl_launch_dependents();
    const int G = a.group, QT = a.q_tile, per_step = QT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar_q[i], 2);  // the copies, and the rows' constants
            mbar_init(&bar_step[i], kMtEpiWarps);
        }
        for (int i = 0; i < kMtTiles; ++i) {
            mbar_init(&bar_raw[i], 1);
            mbar_init(&bar_conv[i], 4);
            mbar_init(&bar_k[i], kFp8 ? 4 : 1);
            mbar_init(&bar_k_empty[i], 1);
            mbar_init(&bar_s[i], 1);
            mbar_init(&bar_s_empty[i], 4);
        }
        mbar_init(&bar_fin, 1);
        s_fail = 0;
        s_seq = -1;
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
    }
    // The cut: thread i sums the costs of its part of the sequences; the CTA's part of the
    // whole begins in the part of one thread, which finds the sequence.
    int64_t lo, hi;
    {
        const int per = (a.num_seqs + kMtThreads - 1) / kMtThreads;
        const int s0 = min(a.num_seqs, static_cast<int>(threadIdx.x) * per), s1 = min(a.num_seqs, s0 + per);
        int64_t mine = 0;
        for (int i = s0; i < s1; ++i) mine += MtCost(mass_seq(a, i, blockIdx.x == 0), G, per_step).all(a.hkv);
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) s_cost[warp] = upto;
        __syncthreads();
        int64_t total = 0;
        for (int w = 0; w < kMtThreads / 32; ++w) {
            if (w == warp) upto += total;
            total += s_cost[w];
        }
        const int64_t n = gridDim.x, part = total / n, rest = total % n, c = blockIdx.x;
        lo = part * c + min(c, rest);
        hi = lo + part + (c < rest ? 1 : 0);
        int64_t base = upto - mine;
        if (mine > 0 && base <= lo && lo < upto) {
            for (int i = s0; i < s1; ++i) {
                const int64_t cost = MtCost(mass_seq(a, i, false), G, per_step).all(a.hkv);
                if (lo < base + cost) {
                    s_seq = i;
                    s_base = base;
                    break;
                }
                base += cost;
            }
        }
    }
    __syncthreads();
    if (lo >= hi || s_seq < 0) return;
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
    MtWalk w(a, s_seq, s_base, lo, hi);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int nraw = 0, loads[kMtTiles] = {0, 0, 0, 0};  // key tiles: in all, and by stage
        bool ok = true;
        MtStages q;
        // this lane's rows of a step: token and head of row lane + 32 i
        int row_tok[4], row_head[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            row_tok[i] = (lane + 32 * i) / G;
            row_head[i] = (lane + 32 * i) % G;
        }
        // step qs into stage st, once the epilogue is done with what was there
        auto load_q = [&](int qs, int st) {
            if (q.uses[st] > 0 &&
                !__all_sync(0xFFFFFFFFu, mbar_wait(&bar_step[st], q.parity(st), kWaitLimitNs, abort)))
                return false;
            const int t0 = qs * per_step;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar_q[st], C::kHalves * 64 * 2 * G * QT);
                for (int h = 0; h < C::kHalves; ++h)
                    tma_load_3d(smem + C::kOffQ + st * C::kQBytes + h * C::kQHalf, &qmap, &bar_q[st], h * 64, w.kvh * G,
                                w.s.q0 + t0);
            }
#pragma unroll
            for (int i = 0; i < kMtCols / 32; ++i) {
                const int c = lane + 32 * i;
                const int tok = t0 + row_tok[i];
                bool real = row_tok[i] < QT && tok < w.ntok;
                float nl = -INFINITY, slope = 0.f;
                int klo = 0, khi = -1;
                if (real) {
                    const int h = w.kvh * G + row_head[i];
                    const float lse = a.lse[static_cast<size_t>(w.s.q0 + tok) * a.hq + h];
                    real = lse != -INFINITY;  // such a row sees no key: its q may hold anything
                    if (real) {
                        nl = -lse * kLog2e;
                        if (a.slopes) slope = a.slopes[h] * kLog2e;
                        mass_span(a, w.s, w.s.off + tok, klo, khi);
                    }
                }
                rows[st].neg_lse[c] = nl;
                rows[st].slope[c] = slope;
                rows[st].tok[c] = static_cast<float>(tok);
                rows[st].span[c] = make_int2(klo, khi);
                const int all_lo = __reduce_max_sync(0xFFFFFFFFu, klo), all_hi = __reduce_min_sync(0xFFFFFFFFu, khi);
                const int any_lo = __reduce_min_sync(0xFFFFFFFFu, real ? klo : INT32_MAX);
                const int any_hi = __reduce_max_sync(0xFFFFFFFFu, khi);
                if (lane == 0) rows[st].chunk[i] = make_int4(all_lo, all_hi, any_lo, any_hi);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_q[st]);
            ++q.uses[st];
            return true;
        };
        // block ids: lane l has block l of the tiles; the next ones' are read ahead
        int ids_tile = 0, ids = 0, ids_next = 0;
        auto read_ids = [&](int tile) {
            const int64_t blk = static_cast<int64_t>(tile) * kMtBlocks + lane;
            return blk * kBlockSize < w.s.kv_len && w.block_seen(static_cast<int>(blk))
                       ? __ldg(a.block_tables + static_cast<size_t>(w.seq) * a.mbps + blk)
                       : 0;
        };
        // e4m3: the first `count` loads of tile x have been converted; what each stage of codes holds
        int done[kMtTiles] = {0, 0, 0, 0}, in_stage[C::kMaxRaw] = {0, 0, 0}, stage_load[C::kMaxRaw] = {0, 0, 0};
        auto converted = [&](int x, int count) {
            if (done[x] >= count) return true;  // (count is at most one more)
            done[x] = count;
            return __all_sync(0xFFFFFFFFu, mbar_wait(&bar_conv[x], (count - 1) & 1, kWaitLimitNs, abort)) != 0;
        };
        // tile x of them into stage x
        auto load_keys = [&](int x) {
            const int id = __shfl_sync(0xFFFFFFFFu, ids, x * kMtBlocks + (lane & (kMtBlocks - 1)));
            const int nvalid = min(kMtBlocks, (w.s.kv_len - 1) / kBlockSize + 1 - (w.tile + x) * kMtBlocks);
            if constexpr (kFp8) {
                // the tile's codes before these have been converted (so that its warps see every phase
                // of bar_raw[x]), and so have those that the stage holds
                const int rs = nraw % raw_stages;
                if (!converted(x, loads[x]) || (nraw >= raw_stages && !converted(in_stage[rs], stage_load[rs]))) return false;
                ++nraw;
                ++loads[x];
                in_stage[rs] = x;
                stage_load[rs] = loads[x];
                if (lane == 0) mbar_arrive_expect_tx(&bar_raw[x], nvalid * (C::kBlkBytes / 2));
                __syncwarp();
                if (lane < nvalid)
                    tma_load_4d(smem + C::raw_stage(rs) + lane * (C::kBlkBytes / 2), &kmap, &bar_raw[x], 0, 0, w.kvh, id);
            } else {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bar_k_empty[x], (loads[x] & 1) ^ 1, kWaitLimitNs, abort))) return false;
                ++loads[x];
                if (lane == 0) mbar_arrive_expect_tx(&bar_k[x], nvalid * C::kBlkBytes);
                __syncwarp();
                if (lane < nvalid)
                    tma_load_5d(smem + C::kOffK + x * C::kKBytes + lane * C::kBlkBytes, &kmap, &bar_k[x], 0, 0, 0, 0,
                                id * a.hkv + w.kvh);
            }
            return true;
        };
        bool q_due = false;  // a resident segment's rows are not loaded yet
        while (ok && w.next()) {
            int slo, shi;
            w.steps(slo, shi);
            const int nt = w.n;
            q_due = q_due || w.fresh;
            if (slo >= shi) continue;  // no query sees the tiles: nothing of them is read
            ids = !w.fresh && ids_tile == w.tile ? ids_next : read_ids(w.tile);
            ids_tile = w.tile + nt;
            ids_next = read_ids(ids_tile);
            if (ids < 0 || ids >= a.num_blocks) {
                flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                ids = 0;  // read a valid block; the keys' weights are not written
            }
            ok = load_keys(0);
            if (w.resident) {
                for (int qs = 0; ok && q_due && qs < w.nsteps; ++qs) ok = load_q(qs, qs);
                q_due = false;
                for (int x = 1; ok && x < kMtTiles; ++x)
                    if (x < nt) ok = load_keys(x);
            } else {
                for (int qs = slo; ok && qs < shi; ++qs) {
                    ok = load_q(qs, q.turn);
                    q.turn ^= 1;
                    for (int x = 1; ok && qs == slo && x < kMtTiles; ++x)
                        if (x < nt) ok = load_keys(x);
                }
            }
        }
        if (!ok && lane == 0) atomicOr(&s_fail, 1);
        // drain: every copy issued has landed before this CTA exits
        for (int i = 0; i < 2; ++i)
            if (q.uses[i] > 0) (void)mbar_wait(&bar_q[i], q.parity(i));
        for (int x = 0; x < kMtTiles; ++x)
            if (loads[x] > 0) (void)mbar_wait(kFp8 ? &bar_raw[x] : &bar_k[x], (loads[x] - 1) & 1);
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer
        constexpr uint32_t kIdesc = tc::idesc_bf16_f32(kMtKeys, kMtCols, false, false);
        int loads[kMtTiles] = {0, 0, 0, 0}, used[kMtTiles] = {0, 0, 0, 0};  // of key stage and S buffer x
        bool ok = true, q_due = false;
        MtStages q;
        while (ok && w.next()) {
            q_due = q_due || w.fresh;
            int slo, shi;
            w.steps(slo, shi);
            const int nt = w.n;
            if (slo >= shi) continue;
            if (w.resident && q_due)
                for (int qs = 0; qs < w.nsteps; ++qs) ++q.uses[qs];
            q_due = false;
            for (int qs = slo; ok && qs < shi; ++qs) {
                int st = qs;
                if (!w.resident) {
                    st = q.turn;
                    ++q.uses[st];
                    q.turn ^= 1;
                }
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_q[st], q.parity(st), kWaitLimitNs, abort));
#pragma unroll
                for (int x = 0; x < kMtTiles; ++x) {
                    if (!ok || x >= nt) break;
                    bool r = true;
                    if (qs == slo) r = mbar_wait(&bar_k[x], loads[x]++ & 1, kWaitLimitNs, abort);
                    r = r && mbar_wait(&bar_s_empty[x], (used[x]++ & 1) ^ 1, kWaitLimitNs, abort);
                    ok = __all_sync(0xFFFFFFFFu, r);
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (lane == 0) {
                        const uint32_t sk = smem_u32(smem + C::kOffK + x * C::kKBytes);
                        const uint32_t sq = smem_u32(smem + C::kOffQ + st * C::kQBytes);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const int h = kk >> 2;
                            const uint32_t ko = (kk & 3) * 32;
                            const uint64_t ad = tc::smem_desc(sk + h * 1024 + ko, 16, C::kGrpBytes);
                            const uint64_t bd = tc::smem_desc(sq + h * C::kQHalf + ko, 16, 1024);
                            tc::mma_bf16(tmem + x * kMtCols, ad, bd, kIdesc, kk > 0 ? 1u : 0u);
                        }
                        tc::commit(&bar_s[x]);
                        if (qs == shi - 1) tc::commit(&bar_k_empty[x]);
                    }
                    __syncwarp();
                }
            }
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
        const int x = (warp - 2) >> 2;           // its tile of those at hand
        const int key = (warp & 3) * 32 + lane;  // the TMEM lane this thread may read
        const uint32_t s_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + x * kMtCols;
        ScoreScale sc(a.sm_scale, a.cap, 1.f);
        TanhPair tp(sc);
        const float in1 = sc.in;  // with a scale of 1
        const bool capped = kMode == kMtCap || (kMode == kMtBias && sc.out > 0.f);
        int nraw = 0, loads = 0, used = 0, held = 0;  // held: stages of a resident segment's rows in use
        bool ok = true, q_due = false;
        MtStages q;
        while (w.next()) {
            const int k0 = (w.tile + min(x, w.n - 1)) * kMtKeys, t = k0 + key;  // (x < n where it counts)
            if (w.fresh) {
                // a resident segment is over: its stages may be loaded anew
                __syncwarp();
                if (lane == 0)
                    for (int i = 0; i < held; ++i) mbar_arrive(&bar_step[i]);
                held = 0;
                q_due = true;
                if constexpr (kFp8) {
                    sc.in = in1 * a.k_scale[w.kvh];
                    tp.in = pack_f32x2(sc.in, sc.in);
                }
            }
            int slo, shi;
            w.steps(slo, shi);
            const int nt = w.n;
            const int k_last = min(k0 + (kMtKeys - 1), w.s.kv_len - 1);
            float* at = a.mass + (static_cast<size_t>(w.seq) * a.hkv + w.kvh) * a.mass_stride + t;
            float old = 0.f, sum = 0.f;
            int id = 0;
            const bool mine = x < nt && t < w.s.kv_len;
            if (mine) {
                if (a.keep != 0.f && t < w.s.off) old = a.keep * *at;
                if (slo < shi && w.block_seen(t / kBlockSize))
                    id = a.block_tables[static_cast<size_t>(w.seq) * a.mbps + t / kBlockSize];
            }
            if constexpr (kFp8) {
                // the codes come one tile after the other through the stages; a tile's own warps convert them
                const int rs = (nraw + x) % raw_stages;
                if (slo < shi) nraw += nt;
                if (ok && slo < shi && x < nt) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_raw[x], loads & 1, kWaitLimitNs, abort) &&
                                                     mbar_wait(&bar_k_empty[x], (loads & 1) ^ 1, kWaitLimitNs, abort));
                    ++loads;
                    if (ok) {
                        convert_keys<D>(smem + C::raw_stage(rs), smem + C::kOffK + x * C::kKBytes, (warp - 2 - 4 * x) * 32 + lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&bar_k[x]);
                            mbar_arrive(&bar_conv[x]);
                        }
                    }
                }
            }
            if (w.resident && q_due && slo < shi) {
                for (int qs = 0; ok && qs < w.nsteps; ++qs) {
                    ++q.uses[qs];
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_q[qs], q.parity(qs), kWaitLimitNs, abort));
                }
                held = w.nsteps;
                q_due = false;
            }
            for (int qs = slo; ok && qs < shi; ++qs) {
                int st = qs;
                if (!w.resident) {
                    // (warps without a tile of these wait too: their arrival on bar_step must not
                    // run ahead of the step)
                    st = q.turn;
                    ++q.uses[st];
                    q.turn ^= 1;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_q[st], q.parity(st), kWaitLimitNs, abort));
                    if (!ok) break;
                }
                if (x < nt) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bar_s[x], used++ & 1, kWaitLimitNs, abort));
                    if (!ok) break;
                    tc::fence_after_sync();
                    const MtRows& r = rows[st];
#pragma unroll 1
                    for (int c = 0; c < kMtCols; c += 32) {
                        float v[32];
                        tc::ld32(s_addr + c, v);
                        tc::wait_ld();
                        if (c + 32 == kMtCols) {
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar_s_empty[x]);
                        }
                        const int4 ch = r.chunk[c >> 5];
                        if (ch.z > k_last || ch.w < k0) continue;
                        // (keys past the last are whatever the tile holds: not looked at)
                        const float y = capped && t <= k_last ? largest(v, sc.in) : 0.f;
                        const bool poly = __all_sync(0xFFFFFFFFu, y <= kTanhPoly);
                        if (kMode != kMtBias && ch.x <= k0 && ch.y >= k_last && poly) {
                            if constexpr (kMode == kMtNone)
                                sum += sum_seen<kMtPlain>(v, r.neg_lse + c, sc, tp);
                            else
                                sum += __all_sync(0xFFFFFFFFu, y <= kTanhNear) ? sum_seen<kMtNear>(v, r.neg_lse + c, sc, tp)
                                                                               : sum_seen<kMtPoly>(v, r.neg_lse + c, sc, tp);
                        } else {
                            sum += sum_edge<kMode>(v, r, c, sc, tp, poly, static_cast<float>(t - w.s.off), t);
                        }
                    }
                }
                __syncwarp();
                if (!w.resident && lane == 0) mbar_arrive(&bar_step[st]);
            }
            if (!ok) break;
            if (mine && id >= 0 && id < a.num_blocks) *at = old + sum;
        }
        if (!ok && lane == 0) {
            flag_error(a.err, PKV_DEVERR_TIMEOUT);
            atomicOr(&s_fail, 1);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D, bool kFp8, int kMode>
cudaError_t launch_mass_tc_m(const MassArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap, cudaStream_t stream) {
    using C = MtCfg<D, kFp8>;
    static_assert(C::kSmemBytes <= 227 * 1024 - 14 * 1024, "shared memory: the arena, the rows' constants, the barriers");
    auto kern = mass_tc_kernel<D, kFp8, kMode>;
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
    // one CTA an SM, fewer where there are fewer tiles
    const int64_t tiles = static_cast<int64_t>((a.max_kv - 1) / kMtKeys + 1) * a.hkv * a.num_seqs;
    const dim3 grid(static_cast<unsigned>(min(int64_t{max(1, a.num_sms)}, tiles)));
    return launch_pdl(kern, grid, dim3(kMtThreads), C::kSmemBytes, stream, a, a.max_q <= a.q_tile ? C::kMaxRaw : 1,
                      qmap, kmap);
}

template <int D, bool kFp8>
cudaError_t launch_mass_tc_t(const MassArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap, cudaStream_t stream) {
    if (a.slopes) return launch_mass_tc_m<D, kFp8, kMtBias>(a, qmap, kmap, stream);
    return a.cap > 0.f ? launch_mass_tc_m<D, kFp8, kMtCap>(a, qmap, kmap, stream)
                       : launch_mass_tc_m<D, kFp8, kMtNone>(a, qmap, kmap, stream);
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
