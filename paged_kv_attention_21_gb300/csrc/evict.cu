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
// share the found ones are all kept.  Then every warp counts what it keeps of a contiguous
// part, and writes it in order.  Four keys a thread: instructions bound it (one key at a
// time took 31 us for 512 rows of up to 16384 keys).
template <int C>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a, const int cached) {
    extern __shared__ uint4 s_key[];                 // [cached / 4]
    __shared__ __align__(16) int hist[kSelBins];
    // the cluster's histogram: the CTAs add their bins to one another's, by turns to one of two
    __shared__ __align__(16) int whole[C > 1 ? 2 : 1][C > 1 ? kSelBins : 4];
    __shared__ int part[kSelWarps];
    __shared__ int s_digit, s_rest, s_all;
    __shared__ int s_gt[kSelWarps], s_eq[kSelWarps], s_sum[2];
    pdl_wait();
    pdl_launch_dependents();
    const int seq = blockIdx.y, head = blockIdx.x / C, rank = blockIdx.x % C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
        if (t < lo || t + 4 > hi) {  // (left < 4 is past hi)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (t + u < lo || t + u >= hi) k[u] = 0xFFFFFFFFu;
                if (u >= left) k[u] = 0u;
            }
        }
        return make_uint4(k[0], k[1], k[2], k[3]);
    };
    auto keys = [&](int i) { return in_smem ? s_key[i] : load(i); };
    uint32_t found = 0, mask = 0;  // the threshold's digits so far
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
                if (in_smem) s_key[i] = q;
                atomicAdd(&h[q.x >> 21], 1);
                atomicAdd(&h[q.y >> 21], 1);
                atomicAdd(&h[q.z >> 21], 1);
                atomicAdd(&h[q.w >> 21], 1);
            }
        } else {
#pragma unroll 2
            for (int i = tid; i < fours; i += kSelThreads) {  // (the fours that this thread stored)
                const uint4 q = keys(i);
                if ((q.x & mask) == found) atomicAdd(&h[(q.x >> shift) & digit], 1);
                if ((q.y & mask) == found) atomicAdd(&h[(q.y >> shift) & digit], 1);
                if ((q.z & mask) == found) atomicAdd(&h[(q.z >> shift) & digit], 1);
                if ((q.w & mask) == found) atomicAdd(&h[(q.w >> shift) & digit], 1);
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
        if (s_all) break;
        // (s_digit is written again after two barriers at least)
    }
    // a key is kept if its digits are above the found ones, and the first `rest` of those that share them.
    // Of four keys: bits 0..3 above, bits 16..19 equal
    const uint32_t top = found | ~mask;
    auto look = [&](int i) {
        const uint4 q = keys(i);
        uint32_t x = 0;
        x |= q.x > top ? 0x1u : q.x >= found ? 0x10000u : 0u;
        x |= q.y > top ? 0x2u : q.y >= found ? 0x20000u : 0u;
        x |= q.z > top ? 0x4u : q.z >= found ? 0x40000u : 0u;
        x |= q.w > top ? 0x8u : q.w >= found ? 0x80000u : 0u;
        return x;
    };
    // a warp's part: whole 32 fours, contiguous; what its first eight turns saw is kept for the writing
    constexpr int kSeen = 8;
    const int per = (fours + kSelThreads - 1) / kSelThreads * 32;
    const int f0 = min(fours, warp * per), f1 = min(fours, f0 + per);
    uint32_t seen[kSeen];
    int gts = 0, eqs = 0;
#pragma unroll
    for (int u = 0; u < kSeen; ++u) {
        const int i = f0 + lane + 32 * u;
        seen[u] = i < f1 ? look(i) : 0u;
        gts += __popc(seen[u] & 0xFu);
        eqs += __popc(seen[u] >> 16);
    }
    for (int i = f0 + lane + 32 * kSeen; i < f1; i += 32) {
        const uint32_t x = look(i);
        gts += __popc(x & 0xFu);
        eqs += __popc(x >> 16);
    }
    gts = __reduce_add_sync(0xFFFFFFFFu, gts);
    eqs = __reduce_add_sync(0xFFFFFFFFu, eqs);
    if (lane == 0) s_gt[warp] = gts, s_eq[warp] = eqs;
    __syncthreads();
    int gt_before = 0, eq_before = 0;
    if constexpr (C > 1) {
        if (tid == 0) {
            int x = 0, y = 0;
            for (int w = 0; w < kSelWarps; ++w) x += s_gt[w], y += s_eq[w];
            s_sum[0] = x, s_sum[1] = y;
        }
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            gt_before += __float_as_int(ld_cluster_f32(cluster_map(smem_u32(&s_sum[0]), r)));
            eq_before += __float_as_int(ld_cluster_f32(cluster_map(smem_u32(&s_sum[1]), r)));
        }
    }
    for (int w = 0; w < warp; ++w) gt_before += s_gt[w], eq_before += s_eq[w];
    auto write = [&](int i, uint32_t x) {
        const uint32_t below = (1u << lane) - 1;
        int g = gt_before, e = eq_before;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t b = __ballot_sync(0xFFFFFFFFu, x >> u & 1);
            g += __popc(b & below);
            gt_before += __popc(b);
        }
        if (__any_sync(0xFFFFFFFFu, x >> 16)) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t b = __ballot_sync(0xFFFFFFFFu, x >> (16 + u) & 1);
                e += __popc(b & below);
                eq_before += __popc(b);
            }
        }
        if (x) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool is_gt = x >> u & 1, is_eq = x >> (16 + u) & 1;
                if (is_gt || (is_eq && e < rest)) out[g + min(e, rest)] = c0 + 4 * i + u;
                g += is_gt;
                e += is_eq;
            }
        }
    };
#pragma unroll
    for (int u = 0; u < kSeen; ++u)
        if (f0 + 32 * u < f1) write(f0 + lane + 32 * u, seen[u]);
    for (int ib = f0 + 32 * kSeen; ib < f1; ib += 32) write(ib + lane, ib + lane < f1 ? look(ib + lane) : 0u);
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
    const int cached = static_cast<int>(min((static_cast<int64_t>((a.max_kv - 1) / C + 1) + 3) / 4 * 4, int64_t{kMost}));
    return launch_pdl_cluster(kern, dim3(a.hkv * C, a.num_seqs), dim3(kSelThreads), static_cast<size_t>(cached) * 4, stream,
                              static_cast<unsigned>(C), a, cached);
}

// ------------------------------------------------------------ compaction --

constexpr int kCmpThreads = 256;

// Where the rows j0, j0 + step, ... below n of (seq, head) come from and go to, in 16-byte
// pieces of the pools; bit r of the answer: row r is there, its position and block ids in
// range.  Every load of a kind is issued before one is looked at: row by row, a step of
// eight rows took eight times the round trips (8192 rows of a head in place: 136 us, now 98).
template <int R>
__device__ __forceinline__ uint32_t compact_rows(const CompactArgs& a, int seq, int head, int j0, int step, int n, int pieces,
                                                 int (&pos)[R], size_t (&src)[R], size_t (&dst)[R]) {
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

__device__ __forceinline__ int compact_count(const CompactArgs& a, int seq, bool flag) {
    const int n = a.kept_lens[seq];
    if (n > a.max_kept && flag) flag_error(a.err, PKV_DEVERR_LENGTH);
    return min(n, a.max_kept);
}

// A thread moves one 16-byte piece of the K and V of kCmpRows rows.
constexpr int kCmpRows = 2;
__global__ void __launch_bounds__(kCmpThreads) compact_kernel(const CompactArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int seq = blockIdx.z, head = blockIdx.y;
    const int pieces = a.row_bytes / 16, step = kCmpThreads / pieces;
    const int n = compact_count(a, seq, blockIdx.x == 0 && head == 0 && threadIdx.x == 0);
    const int j0 = blockIdx.x * step * kCmpRows + threadIdx.x / pieces;
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
    const int pieces = a.row_bytes / 16, mine = min(pieces, 8), step = kCmpThreads / mine;
    const int slice = blockIdx.x >> 1;
    uint4* pool = static_cast<uint4*>(blockIdx.x & 1 ? a.v_dst : a.k_dst) + slice * 8;
    const int n = compact_count(a, seq, blockIdx.x == 0 && head == 0 && threadIdx.x == 0);
    const int c = threadIdx.x % mine, row = threadIdx.x / mine;
    const bool weights = a.mass && blockIdx.x == 0 && c == 0;
    const size_t line = static_cast<size_t>(seq) * a.hkv + head;
    int pos[kInRows];
    size_t src[kInRows], dst[kInRows];
    uint32_t ok = compact_rows(a, seq, head, row, step, n, pieces, pos, src, dst);
    for (int j0 = row; j0 - row < n; j0 += step * kInRows) {
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
    // CTAs per row.  A CTA alone takes 7.5 us for 8192 keys, 10 for 16384 and 17 for 32768;
    // eight take 8, 8 and 9 for one of a few rows, but clusters are launched one after the other,
    // some 27 CTAs a microsecond: 128 rows of 16384 keys take 11.5, 14, 22 and 42 us with 1, 2, 4
    // and 8, 256 rows of 32768 keys 42 and 38 with 1 and 2.  So: as many as hold 16384 keys each, and more
    // while the CTAs are few.
    const int64_t rows = static_cast<int64_t>(a.hkv) * a.num_seqs;
    int c = 1;
    while (c < 8 && (a.max_kv > 16384 * c || (a.max_kv > 8192 && rows * 2 * c <= 128))) c *= 2;
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
