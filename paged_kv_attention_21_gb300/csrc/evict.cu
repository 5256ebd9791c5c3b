// evict.cu -- eviction from the cache by accumulated weight: which positions to keep,
// and their rows moved together.
#include "common.cuh"
#include "internal.h"

namespace pkv {

namespace {

// ------------------------------------------------------------- selection --

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;

// An unsigned integer that orders as the weights do: NaN below every number, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t b = __float_as_uint(w + 0.f);
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
    return (b >> 31) ? ~b : b | 0x80000000u;
}

// Exclusive prefix sum over the block's threads; *total: the sum of all.  `part`: a word
// per warp and one more, free again after the next barrier.
__device__ __forceinline__ int block_scan(int v, int* part, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int p = lane < kSelWarps ? part[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, p, o);
            if (lane >= o) p += y;
        }
        if (lane < kSelWarps) part[lane] = p;
    }
    __syncthreads();
    *total = part[kSelWarps - 1];
    return x - v + (warp > 0 ? part[warp - 1] : 0);
}

// A cluster of C CTAs per (KV head, sequence), each with a contiguous part of the row, held
// in shared memory as ordered integers where it fits.  The first and the last keys, kept in
// any case, count as larger than any weight, so that one selection of the `budget` largest
// is left.  The threshold is found digit by digit (11, 11 and 10 bits) from histograms,
// which the CTAs read from one another; no further digit is looked at once the keys that
// share the found ones are all kept.  The first digit's histogram is of all keys.  Then a
// thread takes up to 32 neighbouring keys and has a bit for each that is above the digits and
// for each that shares them; later digits look at the latter alone, and at the end a scan
// over the threads' counts says where each writes its own.  Instructions bound it (512 rows of
// up to 16384 keys: 31 us with one key at a time, 20 with every digit over all keys and the
// places from a ballot for every 32 keys, 17 so; the loads alone 6.8).
template <int C>
__global__ void __launch_bounds__(kSelThreads, 3) select_kernel(const SelectArgs a, const int cached) {
    extern __shared__ uint4 s_key[];                 // [cached / 4]
    __shared__ __align__(16) int hist[kSelBins];
    // the cluster's histogram: the CTAs add their bins to one another's, by turns to one of two
    __shared__ __align__(16) int whole[C > 1 ? 2 : 1][C > 1 ? kSelBins : 4];
    __shared__ int part[kSelWarps];
    __shared__ int s_digit, s_rest, s_all;
    __shared__ int s_sum[2];
    pdl_wait();
    pdl_launch_dependents();
    const int seq = blockIdx.y, head = blockIdx.x / C, rank = blockIdx.x % C;
    const int tid = threadIdx.x;
    int n = a.kv_lens[seq];
    if (n > a.max_kv) {
        if (tid == 0 && blockIdx.x == 0) flag_error(a.err, PKV_DEVERR_LENGTH);
        n = a.max_kv;
    }
    n = max(n, 0);
    if (tid == 0 && blockIdx.x == 0) a.kept_lens[seq] = min(n, a.budget);
    int* out = a.kept + (static_cast<size_t>(seq) * a.hkv + head) * a.kept_stride;
    if (n <= a.budget) {
        for (int64_t t = rank * kSelThreads + tid; t < n; t += C * kSelThreads) out[t] = static_cast<int>(t);
        return;
    }
    const float* row = a.mass + (static_cast<size_t>(seq) * a.hkv + head) * a.mass_stride;
    const int lo = a.first, hi = n - a.recent;
    int rest = a.budget;  // to keep of the keys that share the digits found so far
    // this CTA's part [c0, c0 + m) of the row: whole fours, but for the row's end
    const int64_t size = (static_cast<int64_t>((n - 1) / C + 1) + 3) / 4 * 4;
    const int c0 = static_cast<int>(min(static_cast<int64_t>(n), rank * size));
    const int m = static_cast<int>(min(static_cast<int64_t>(n - c0), size));
    const int fours = (m - 1) / 4 + (m > 0 ? 1 : 0);
    const bool in_smem = m <= cached;
    // keys 4 i .. 4 i + 3 of the part; those past the row's end are 0: the least, and the last of their equals
    const bool wide = reinterpret_cast<uintptr_t>(row) % 16 == 0;
    auto load = [&](int i) {
        const int t = c0 + 4 * i, left = m - 4 * i;
        float w[4] = {0.f, 0.f, 0.f, 0.f};
        if (wide && left >= 4) {
            const float4 v = *reinterpret_cast<const float4*>(row + t);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (u < left) w[u] = row[t + u];
        }
        uint32_t k[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) k[u] = weight_key(w[u]);
        if (t < lo || t > hi - 4) {  // (left < 4 is past hi; t + 4 may pass 32 bits)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (t + u < lo || t + u >= hi) k[u] = 0xFFFFFFFFu;
                if (u >= left) k[u] = 0u;
            }
        }
        return make_uint4(k[0], k[1], k[2], k[3]);
    };
    // fours are stored so that neither eight neighbours nor eight that lie two, four or eight apart meet in a bank
    auto slot = [](int i) { return i ^ (i >> 3 & 7); };
    auto key_at = [&](int j) {  // key j of the part
        if (in_smem) return reinterpret_cast<const uint32_t*>(s_key)[4 * slot(j >> 2) + (j & 3)];
        if (j >= m) return 0u;
        return c0 + j < lo || c0 + j >= hi ? 0xFFFFFFFFu : weight_key(row[c0 + j]);
    };
    uint32_t found = 0, mask = 0;  // the threshold's digits so far
    // From the second digit on a thread has up to eight neighbouring fours, a bit for each key; a part
    // of more than 16384 keys takes several rounds.  A key is kept if its digits are above the found ones,
    // and the first `rest` of those that share them
    const int per = min(8, (fours + kSelThreads - 1) / kSelThreads);
    const int rounds = per > 0 ? (fours - 1) / (kSelThreads * per) + 1 : 1;
    auto first_key = [&](int round) { return (round * kSelThreads + tid) * per * 4; };
    auto classify = [&](int round, uint32_t& above, uint32_t& equal) {
        const uint32_t top = found | ~mask;
        const int i0 = (round * kSelThreads + tid) * per;
        uint32_t a_ = 0, e_ = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (u >= per || i0 + u >= fours) break;
            const uint4 q = in_smem ? s_key[slot(i0 + u)] : load(i0 + u);
            const uint32_t k[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (k[c] > top) a_ |= 1u << (4 * u + c);
                if (k[c] >= found) e_ |= 1u << (4 * u + c);
            }
        }
        above = a_, equal = e_ & ~a_;
    };
    uint32_t gt = 0, eq = 0;  // of the first round
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digit = pass == 2 ? 1023u : 2047u;
        int* h = hist;
        reinterpret_cast<int4*>(h)[tid] = make_int4(0, 0, 0, 0);
        if constexpr (C > 1) {  // (peers add to the first after the pass's first cluster barrier, to the other later)
            reinterpret_cast<int4*>(whole[pass & 1])[tid] = make_int4(0, 0, 0, 0);
            cluster_arrive();
        }
        __syncthreads();
        if (pass == 0) {  // the row comes in, and all of it counts
#pragma unroll 4
            for (int i = tid; i < fours; i += kSelThreads) {
                const uint4 q = load(i);
                if (in_smem) s_key[slot(i)] = q;
                atomicAdd(&h[q.x >> 21], 1);
                atomicAdd(&h[q.y >> 21], 1);
                atomicAdd(&h[q.z >> 21], 1);
                atomicAdd(&h[q.w >> 21], 1);
            }
        } else {
            for (int r = 0; r < rounds; ++r) {
                uint32_t g = gt, e = eq;
                if (r > 0 || pass == 1) classify(r, g, e);
                if (r == 0) gt = g, eq = e;
                for (uint32_t x = e; x; x &= x - 1) atomicAdd(&h[(key_at(first_key(r) + __ffs(x) - 1) >> shift) & digit], 1);
            }
        }
        __syncthreads();
        // thread i has the bins 2047 - 4 i .. 2044 - 4 i: the largest first
        const int at = kSelBins - 4 - 4 * tid;
        int4 c = *reinterpret_cast<const int4*>(h + at);
        if constexpr (C > 1) {
            cluster_wait();  // every CTA has cleared its whole[]
            const uint32_t to = smem_u32(whole[pass & 1] + at);
            const int v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (v[u])  // few bins are in use
                    for (int r = 0; r < C; ++r) red_cluster_add(cluster_map(to + 4 * u, r), v[u]);
            cluster_sync();
            c = *reinterpret_cast<const int4*>(whole[pass & 1] + at);
        }
        const int bins[4] = {c.w, c.z, c.y, c.x};
        int total;
        int before = block_scan(c.x + c.y + c.z + c.w, part, &total);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (before < rest && before + bins[u] >= rest) {
                s_digit = kSelBins - 1 - 4 * tid - u;
                s_rest = rest - before;
                s_all = before + bins[u] == rest;
            }
            before += bins[u];
        }
        __syncthreads();
        found |= static_cast<uint32_t>(s_digit) << shift;
        mask |= digit << shift;
        rest = s_rest;
        const uint32_t top = found | ~mask;
        if (pass > 0)  // the first round's keys that shared the digits before
            for (uint32_t x = eq; x; x &= x - 1) {
                const uint32_t bit = x & -x, k = key_at(first_key(0) + __ffs(x) - 1);
                if (k > top) gt |= bit;
                if (k > top || k < found) eq &= ~bit;
            }
        else if (s_all) classify(0, gt, eq);
        if (s_all) break;
        // (s_digit is written again after two barriers at least)
    }
    // counts of a round, above in the low half, equal in the high: at most 16384 each
    int total;
    int before = block_scan(__popc(gt) | __popc(eq) << 16, part, &total);
    int gt_before = 0, eq_before = 0;
    if constexpr (C > 1) {
        int gts = total & 0xFFFF, eqs = total >> 16;
#pragma unroll 1
        for (int r = 1; r < rounds; ++r) {
            uint32_t g, e;
            classify(r, g, e);
            int more;
            __syncthreads();
            (void)block_scan(__popc(g) | __popc(e) << 16, part, &more);
            gts += more & 0xFFFF, eqs += more >> 16;
        }
        if (tid == 0) s_sum[0] = gts, s_sum[1] = eqs;
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            gt_before += __float_as_int(ld_cluster_f32(cluster_map(smem_u32(&s_sum[0]), r)));
            eq_before += __float_as_int(ld_cluster_f32(cluster_map(smem_u32(&s_sum[1]), r)));
        }
    }
#pragma unroll 1
    for (int r = 0;;) {
        const int e0 = eq_before + (before >> 16);
        while (eq && e0 + __popc(eq) > rest) eq ^= 0x80000000u >> __clz(eq);
        int* to = out + gt_before + (before & 0xFFFF) + min(e0, rest);
        const int j0 = first_key(r) - 1;
        for (uint32_t x = gt | eq; x; x &= x - 1) *to++ = c0 + (j0 + __ffs(x));
        if (++r >= rounds) break;
        gt_before += total & 0xFFFF, eq_before += total >> 16;
        classify(r, gt, eq);
        __syncthreads();
        before = block_scan(__popc(gt) | __popc(eq) << 16, part, &total);
    }
    if constexpr (C > 1) cluster_sync();  // no CTA leaves while a peer may still read its shared memory
}

template <int C>
cudaError_t launch_select_t(const SelectArgs& a, cudaStream_t stream) {
    auto kern = select_kernel<C>;
    constexpr int kMost = 48 * 1024;  // keys a CTA holds (192 KB beside 25 KB of histograms)
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost * 4);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const int cached = static_cast<int>(min((static_cast<int64_t>((a.max_kv - 1) / C + 1) + 31) / 32 * 32, int64_t{kMost}));
    // Three CTAs an SM serve where two leave CTAs waiting (512 rows of up to 16384 keys: 19.2 us with two,
    // 17.3 with three), but where two hold all, three would gather on some of the SMs (256 rows of 16384
    // keys: 12.7 and 16.5 us): shared memory that no second fellow fits beside keeps them apart.
    const bool two = static_cast<int64_t>(a.hkv) * a.num_seqs * C <= 2 * a.num_sms;
    const size_t bytes = max(static_cast<size_t>(cached) * 4, two ? size_t{70 * 1024} : size_t{0});
    return launch_pdl_cluster(kern, dim3(a.hkv * C, a.num_seqs), dim3(kSelThreads), bytes, stream, static_cast<unsigned>(C), a,
                              cached);
}

// ------------------------------------------------------------ compaction --

constexpr int kCmpThreads = 256;

// Where the rows j0, j0 + step, ... below n of (seq, head) come from and go to, in 16-byte
// pieces of the pools; bit r of the answer: row r is there, its position and block ids in
// range.  Every load of a kind is issued before one is looked at: row by row, a step took
// as many round trips as it has rows (8192 rows of one sequence of 8 heads in place: 150 us
// with eight rows a thread and step, 98 so with kInRows).
// (Row numbers are unsigned: those behind the last row, up to 2^31 - 2, pass 31 bits.)
template <int R>
__device__ __forceinline__ uint32_t compact_rows(const CompactArgs& a, int seq, int head, uint32_t j0, uint32_t step, uint32_t n,
                                                 int pieces, int (&pos)[R], size_t (&src)[R], size_t (&dst)[R]) {
    const int* kept = a.kept + (static_cast<size_t>(seq) * a.hkv + head) * a.kept_stride;
    const int* from = a.src_tables + static_cast<size_t>(seq) * a.src_mbps;
    const int* to = a.dst_tables + static_cast<size_t>(seq) * a.dst_mbps;
    uint32_t ok = 0, there = 0;
    int sb[R], db[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        pos[r] = 0;
        if (j0 + r * step < n) {
            there |= 1u << r;
            pos[r] = kept[j0 + r * step];
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool good = pos[r] >= 0 && pos[r] / kBlockSize < a.src_mbps && (!a.mass || pos[r] < a.mass_stride);
        if ((there >> r & 1u) && good) ok |= 1u << r;
        const bool look = ok >> r & 1u;
        sb[r] = look ? from[pos[r] / kBlockSize] : 0;
        db[r] = look ? to[(j0 + r * step) / kBlockSize] : 0;
    }
    uint32_t bad = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (sb[r] < 0 || sb[r] >= a.src_blocks || db[r] < 0 || db[r] >= a.dst_blocks) bad |= 1u << r;
        src[r] = ((static_cast<size_t>(sb[r]) * a.hkv + head) * kBlockSize + pos[r] % kBlockSize) * pieces;
        dst[r] = ((static_cast<size_t>(db[r]) * a.hkv + head) * kBlockSize + (j0 + r * step) % kBlockSize) * pieces;
    }
    if (there != ok) flag_error(a.err, PKV_DEVERR_POSITION);
    if (bad) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
    return ok & ~bad;
}

__device__ __forceinline__ uint32_t compact_count(const CompactArgs& a, int seq, bool flag) {
    const int n = a.kept_lens[seq];
    if (n > a.max_kept && flag) flag_error(a.err, PKV_DEVERR_LENGTH);
    return static_cast<uint32_t>(max(0, min(n, a.max_kept)));
}

// A thread moves one 16-byte piece of the K and V of kCmpRows rows.
constexpr int kCmpRows = 2;
__global__ void __launch_bounds__(kCmpThreads) compact_kernel(const CompactArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int seq = blockIdx.z, head = blockIdx.y;
    const int pieces = a.row_bytes / 16;
    const uint32_t step = kCmpThreads / pieces;
    const uint32_t n = compact_count(a, seq, blockIdx.x == 0 && head == 0 && threadIdx.x == 0);
    const uint32_t j0 = blockIdx.x * step * kCmpRows + threadIdx.x / pieces;
    const int c = threadIdx.x % pieces;
    if (j0 >= n) return;
    const size_t line = static_cast<size_t>(seq) * a.hkv + head;
    int pos[kCmpRows];
    size_t src[kCmpRows], dst[kCmpRows];
    uint4 k[kCmpRows], v[kCmpRows];
    float w[kCmpRows];
    const uint32_t ok = compact_rows(a, seq, head, j0, step, n, pieces, pos, src, dst);
#pragma unroll
    for (int r = 0; r < kCmpRows; ++r) {
        if (!(ok >> r & 1u)) continue;
        k[r] = __ldg(static_cast<const uint4*>(a.k_src) + src[r] + c);
        v[r] = __ldg(static_cast<const uint4*>(a.v_src) + src[r] + c);
        if (a.mass && c == 0) w[r] = a.mass[line * a.mass_stride + pos[r]];
    }
#pragma unroll
    for (int r = 0; r < kCmpRows; ++r) {
        if (!(ok >> r & 1u)) continue;
        static_cast<uint4*>(a.k_dst)[dst[r] + c] = k[r];
        static_cast<uint4*>(a.v_dst)[dst[r] + c] = v[r];
        if (a.mass && c == 0) a.mass_out[line * a.mass_out_stride + j0 + r * step] = w[r];
    }
}

// In place: kept ascends, so row j comes from a row at or behind j.  One CTA per (KV head,
// sequence, pool, 128-byte slice of its rows) -- slices never meet -- takes the rows in steps:
// every thread has read its rows of a step before any is written, and what later steps read
// lies behind all that is written.  A step costs a round trip to memory, so it is long: kInRows
// rows a thread.  Slice 0 of K takes the weights along.
constexpr int kInRows = 4;
__global__ void __launch_bounds__(kCmpThreads) compact_in_place_kernel(const CompactArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int seq = blockIdx.z, head = blockIdx.y;
    const int pieces = a.row_bytes / 16, mine = min(pieces, 8);
    const uint32_t step = kCmpThreads / mine;
    const int slice = blockIdx.x >> 1;
    uint4* pool = static_cast<uint4*>(blockIdx.x & 1 ? a.v_dst : a.k_dst) + slice * 8;
    const uint32_t n = compact_count(a, seq, blockIdx.x == 0 && head == 0 && threadIdx.x == 0);
    const int c = threadIdx.x % mine;
    const uint32_t row = threadIdx.x / mine;
    const bool weights = a.mass && blockIdx.x == 0 && c == 0;
    const size_t line = static_cast<size_t>(seq) * a.hkv + head;
    int pos[kInRows];
    size_t src[kInRows], dst[kInRows];
    uint32_t ok = compact_rows(a, seq, head, row, step, n, pieces, pos, src, dst);
    for (uint32_t j0 = row; j0 - row < n; j0 += step * kInRows) {
        uint4 x[kInRows];
        float w[kInRows];
#pragma unroll
        for (int r = 0; r < kInRows; ++r) {
            if (!(ok >> r & 1u)) continue;
            x[r] = pool[src[r] + c];
            if (weights) w[r] = a.mass[line * a.mass_stride + pos[r]];
        }
        // the next step's addresses, while these rows are on their way
        size_t dst_next[kInRows];
        const uint32_t ok_next = compact_rows(a, seq, head, j0 + step * kInRows, step, n, pieces, pos, src, dst_next);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kInRows; ++r) {
            if (ok >> r & 1u) {
                pool[dst[r] + c] = x[r];
                if (weights) a.mass_out[line * a.mass_out_stride + j0 + r * step] = w[r];
            }
            dst[r] = dst_next[r];
        }
        ok = ok_next;
    }
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, cudaStream_t stream) {
    // CTAs per row.  A CTA alone takes 6.6 us for 8192 keys, 8.7 for 16384 and 13.1 for 32768; eight
    // take 7.7, 7.8 and 8.8 for one of two rows, but clusters are launched one after the other, some 27
    // CTAs a microsecond: 128 rows of 16384 keys take 9.7, 12, 19 and 35 us with 1, 2, 4 and 8, 32 rows of
    // them 9.5, 9.7, 9.4 and 12, 32 rows of 32768 keys 15, 12, 10 and 12, 256 of these 36 and 31 with 1 and 2.
    // So: as many as hold 16384 keys each, and more while the CTAs are few.
    const int64_t rows = static_cast<int64_t>(a.hkv) * a.num_seqs;
    const int few = min(128, a.max_kv / 256);
    int c = 1;
    while (c < 8 && (a.max_kv > 16384 * c || (a.max_kv > 8192 && rows * 2 * c <= few))) c *= 2;
    return c == 1 ? launch_select_t<1>(a, stream) : c == 2 ? launch_select_t<2>(a, stream)
         : c == 4 ? launch_select_t<4>(a, stream) : launch_select_t<8>(a, stream);
}

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream) {
    if (a.in_place) {
        const unsigned slices = (a.row_bytes + 127) / 128;
        return launch_pdl(compact_in_place_kernel, dim3(2 * slices, a.hkv, a.num_seqs), dim3(kCmpThreads), 0, stream, a);
    }
    const int64_t step = static_cast<int64_t>(kCmpThreads) / (a.row_bytes / 16) * kCmpRows;
    const dim3 grid(static_cast<unsigned>((a.max_kept + step - 1) / step), a.hkv, a.num_seqs);
    return launch_pdl(compact_kernel, grid, dim3(kCmpThreads), 0, stream, a);
}

}  // namespace pkv
