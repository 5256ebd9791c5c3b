// mass.cuh -- what the weight kernels (mass.cu, mass_tc.cu) share: a sequence's
// queries, and the keys that each of them sees.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "score.cuh"

namespace pkv {

// One sequence's queries and the keys they see.
struct MassSeq {
    int q0, q_len, rows;  // first query row of q, queries, rows counted (queries x group)
    int kv_len, off;      // keys; position of the first query
    int prefix;           // 0 .. kv_len (or 0)
    bool ok;
};

__device__ __forceinline__ MassSeq mass_seq(const MassArgs& a, int seq, bool flag) {
    MassSeq s;
    s.q0 = a.qo_indptr ? a.qo_indptr[seq] : seq;
    s.q_len = a.qo_indptr ? a.qo_indptr[seq + 1] - s.q0 : 1;
    s.kv_len = a.kv_lens[seq];
    s.ok = s.kv_len > 0;
    if (s.ok && (s.q0 < 0 || s.q_len < 0 || s.q_len > a.total_q - s.q0 || s.kv_len < s.q_len)) {
        if (flag) flag_error(a.err, PKV_DEVERR_POSITION);
        s.ok = false;
    }
    if (s.kv_len > a.max_kv) {
        if (flag) flag_error(a.err, PKV_DEVERR_LENGTH);
        s.kv_len = a.max_kv;
        if (s.kv_len < s.q_len) s.ok = false;
    }
    s.prefix = a.prefix_lens ? max(0, min(a.prefix_lens[seq], s.kv_len)) : 0;
    s.off = s.kv_len - s.q_len;
    int counted = s.q_len;
    if (counted > a.max_q) {
        if (flag && s.ok) flag_error(a.err, PKV_DEVERR_LENGTH);
        counted = a.max_q;
    }
    s.rows = s.ok ? counted * a.group : 0;
    return s;
}

// The tokens [first, last] of the first ntok that see some key of [k0, k1] (last < first:
// none).  hi and lo of mass_span both ascend with the position.
__device__ __forceinline__ void mass_tokens(const MassArgs& a, const MassSeq& s, int ntok, int k0, int k1, int& first,
                                            int& last) {
    first = 0;
    if (a.causal && !(s.off < s.prefix && k0 < s.prefix)) first = max(0, k0 - s.off);
    last = ntok - 1;
    // the last position that sees k1 is k1 + window - 1 (past 32 bits: every one does)
    if (a.window > 0 && a.window - 1 < INT32_MAX - k1) last = min(last, k1 + a.window - 1 - s.off);
}

// The keys [lo, hi] that a query at position pos sees (hi < lo: none).
__device__ __forceinline__ void mass_span(const MassArgs& a, const MassSeq& s, int pos, int& lo, int& hi) {
    hi = s.kv_len - 1;
    if (a.causal) hi = min(hi, pos < s.prefix ? s.prefix - 1 : pos);
    lo = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
}

// The keys [lo, hi] outside of which none of the first ntok queries sees one.
__device__ __forceinline__ void mass_seen(const MassArgs& a, const MassSeq& s, int ntok, int& lo, int& hi) {
    int unused;
    mass_span(a, s, s.off, lo, unused);
    mass_span(a, s, s.off + ntok - 1, unused, hi);
    if (a.causal && s.off < s.prefix) hi = max(hi, s.prefix - 1);
    if (ntok <= 0) lo = 0, hi = -1;
}

// Whether some key of block blk lies in [lo, hi].  (The sums of the last block and of the last
// tile pass 32 bits in contexts that end there: what is compared stays at or below the last key.)
__device__ __forceinline__ bool mass_block_seen(int blk, int lo, int hi) {
    return blk * kBlockSize <= hi && blk * kBlockSize > lo - kBlockSize;
}

}  // namespace pkv
