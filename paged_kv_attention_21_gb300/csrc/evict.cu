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

// One CTA per (KV head, sequence).  The k-th largest key is found digit by digit (11, 11
// and 10 bits) by histograms; then every warp takes a contiguous part of the row, counts
// what it keeps, and writes it in order.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
    __shared__ int hist[kSelBins];
    __shared__ int part[kSelWarps];
    __shared__ int s_digit, s_rest;
    __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
    pdl_wait();
    pdl_launch_dependents();
    const int seq = blockIdx.y, head = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n = a.kv_lens[seq];
    if (n > a.max_kv) {
        if (tid == 0 && head == 0) flag_error(a.err, PKV_DEVERR_LENGTH);
        n = a.max_kv;
    }
    n = max(n, 0);
    if (tid == 0 && head == 0) a.kept_lens[seq] = min(n, a.budget);
    int* out = a.kept + (static_cast<size_t>(seq) * a.hkv + head) * a.kept_stride;
    if (n <= a.budget) {
        for (int t = tid; t < n; t += kSelThreads) out[t] = t;
        return;
    }
    const float* row = a.mass + (static_cast<size_t>(seq) * a.hkv + head) * a.mass_stride;
    const int lo = a.first, hi = n - a.recent;  // the middle, at least one longer than what it may keep
    int rest = a.budget - a.first - a.recent;   // of it to keep
    uint32_t key = 0xFFFFFFFFu;                 // threshold: keep keys above it, and `rest` equal ones
    if (rest > 0) {
        uint32_t found = 0, mask = 0;
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bits = pass == 2 ? 10 : 11;
            for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (int t = lo + tid; t < hi; t += kSelThreads) {
                const uint32_t k = weight_key(row[t]);
                if ((k & mask) == found) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
            }
            __syncthreads();
            // thread i has the bins 2047 - 4 i .. 2044 - 4 i: the largest first
            int c[4], sum = 0, total;
#pragma unroll
            for (int u = 0; u < 4; ++u) sum += c[u] = hist[kSelBins - 1 - 4 * tid - u];
            int before = block_scan(sum, part, &total);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (before < rest && before + c[u] >= rest) {
                    s_digit = kSelBins - 1 - 4 * tid - u;
                    s_rest = rest - before;
                }
                before += c[u];
            }
            __syncthreads();
            found |= static_cast<uint32_t>(s_digit) << shift;
            mask |= ((1u << bits) - 1) << shift;
            rest = s_rest;
            __syncthreads();
        }
        key = found;
    }
    // a warp's part: whole 32s, contiguous
    const int per = ((n + kSelThreads - 1) / kSelThreads) * 32;
    const int t0 = min(n, warp * per), t1 = min(n, t0 + per);
    int gt = 0, eq = 0;
    for (int t = t0 + lane; t < t1; t += 32) {
        if (t < lo || t >= hi) {
            ++gt;
        } else if (rest > 0) {
            const uint32_t k = weight_key(row[t]);
            gt += k > key;
            eq += k == key;
        }
    }
    gt = __reduce_add_sync(0xFFFFFFFFu, gt);
    eq = __reduce_add_sync(0xFFFFFFFFu, eq);
    if (lane == 0) s_gt[warp] = gt, s_eq[warp] = eq;
    __syncthreads();
    int at = 0, eq_left = rest;
    for (int w = 0; w < warp; ++w) {
        const int take = min(eq_left, s_eq[w]);
        at += s_gt[w] + take;
        eq_left -= take;
    }
    for (int tb = t0; tb < t1; tb += 32) {
        const int t = tb + lane;
        bool keep = false, tie = false;
        if (t < t1) {
            if (t < lo || t >= hi) {
                keep = true;
            } else if (rest > 0) {
                const uint32_t k = weight_key(row[t]);
                keep = k > key;
                tie = k == key;
            }
        }
        const uint32_t below = (1u << lane) - 1;
        const uint32_t ties = __ballot_sync(0xFFFFFFFFu, tie);
        keep = keep || (tie && __popc(ties & below) < eq_left);
        eq_left -= min(eq_left, __popc(ties));
        const uint32_t kept = __ballot_sync(0xFFFFFFFFu, keep);
        if (keep) out[at + __popc(kept & below)] = t;
        at += __popc(kept);
    }
}

// ------------------------------------------------------------ compaction --

constexpr int kCmpThreads = 256;

// Where row j of (seq, head) comes from and goes to, in 16-byte pieces of the pools; a
// position or block id out of range: false.
__device__ __forceinline__ bool compact_rows(const CompactArgs& a, int seq, int head, int j, int pieces, int* pos,
                                             size_t* src, size_t* dst) {
    const int r = a.kept[(static_cast<size_t>(seq) * a.hkv + head) * a.kept_stride + j];
    *pos = r;
    if (r < 0 || r / kBlockSize >= a.src_mbps || (a.mass && r >= a.mass_stride)) {
        flag_error(a.err, PKV_DEVERR_POSITION);
        return false;
    }
    const int sb = a.src_tables[static_cast<size_t>(seq) * a.src_mbps + r / kBlockSize];
    const int db = a.dst_tables[static_cast<size_t>(seq) * a.dst_mbps + j / kBlockSize];
    if (sb < 0 || sb >= a.src_blocks || db < 0 || db >= a.dst_blocks) {
        flag_error(a.err, PKV_DEVERR_BLOCK_ID);
        return false;
    }
    *src = ((static_cast<size_t>(sb) * a.hkv + head) * kBlockSize + r % kBlockSize) * pieces;
    *dst = ((static_cast<size_t>(db) * a.hkv + head) * kBlockSize + j % kBlockSize) * pieces;
    return true;
}

__device__ __forceinline__ int compact_count(const CompactArgs& a, int seq, bool flag) {
    const int n = a.kept_lens[seq];
    if (n > a.max_kept && flag) flag_error(a.err, PKV_DEVERR_LENGTH);
    return min(n, a.max_kept);
}

// A thread moves one 16-byte piece of a row's K and V.
__global__ void __launch_bounds__(kCmpThreads) compact_kernel(const CompactArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int seq = blockIdx.z, head = blockIdx.y;
    const int pieces = a.row_bytes / 16;
    const int n = compact_count(a, seq, blockIdx.x == 0 && head == 0 && threadIdx.x == 0);
    const int j = blockIdx.x * (kCmpThreads / pieces) + threadIdx.x / pieces;
    const int c = threadIdx.x % pieces;
    if (j >= n) return;
    int pos;
    size_t src, dst;
    if (!compact_rows(a, seq, head, j, pieces, &pos, &src, &dst)) return;
    const uint4 k = __ldg(static_cast<const uint4*>(a.k_src) + src + c);
    const uint4 v = __ldg(static_cast<const uint4*>(a.v_src) + src + c);
    static_cast<uint4*>(a.k_dst)[dst + c] = k;
    static_cast<uint4*>(a.v_dst)[dst + c] = v;
    if (a.mass && c == 0) {
        const size_t line = static_cast<size_t>(seq) * a.hkv + head;
        a.mass_out[line * a.mass_out_stride + j] = a.mass[line * a.mass_stride + pos];
    }
}

// In place, one CTA per (KV head, sequence): kept ascends, so row j comes from a row
// at or behind j.  The rows are taken in steps; every thread has read its row of the step
// before any is written, and what later steps read lies behind all that is written.
__global__ void __launch_bounds__(kCmpThreads) compact_in_place_kernel(const CompactArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int seq = blockIdx.y, head = blockIdx.x;
    const int pieces = a.row_bytes / 16;
    const int step = kCmpThreads / pieces;
    const int n = compact_count(a, seq, head == 0 && threadIdx.x == 0);
    const int c = threadIdx.x % pieces;
    const size_t line = static_cast<size_t>(seq) * a.hkv + head;
    for (int j0 = 0; j0 < n; j0 += step) {
        const int j = j0 + threadIdx.x / pieces;
        int pos = 0;
        size_t src = 0, dst = 0;
        bool ok = j < n && compact_rows(a, seq, head, j, pieces, &pos, &src, &dst);
        uint4 k, v;
        float w = 0.f;
        if (ok) {
            k = static_cast<const uint4*>(a.k_dst)[src + c];
            v = static_cast<const uint4*>(a.v_dst)[src + c];
            if (a.mass && c == 0) w = a.mass[line * a.mass_stride + pos];
        }
        __syncthreads();
        if (ok) {
            static_cast<uint4*>(a.k_dst)[dst + c] = k;
            static_cast<uint4*>(a.v_dst)[dst + c] = v;
            if (a.mass && c == 0) a.mass_out[line * a.mass_out_stride + j] = w;
        }
    }
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, cudaStream_t stream) {
    return launch_pdl(select_kernel, dim3(a.hkv, a.num_seqs), dim3(kSelThreads), 0, stream, a);
}

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream) {
    if (a.in_place) return launch_pdl(compact_in_place_kernel, dim3(a.hkv, a.num_seqs), dim3(kCmpThreads), 0, stream, a);
    const int step = kCmpThreads / (a.row_bytes / 16);
    const dim3 grid((a.max_kept + step - 1) / step, a.hkv, a.num_seqs);
    return launch_pdl(compact_kernel, grid, dim3(kCmpThreads), 0, stream, a);
}

}  // namespace pkv
