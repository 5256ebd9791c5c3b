// quant_decode.cu -- decode attention over the quantised paged pools.
//
//   o = softmax(sm_scale * q k^T) v over the visible keys, k and v the records'
//   values; a sink logit joins the normaliser with a zero value.
//
// One warp per (sequence, query head): lane l owns dims [l D/32, (l + 1) D/32),
// one pass over the keys with a running maximum and sum in fp32.
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace pkv {

namespace {

template <int D, bool kFp4>
__global__ void __launch_bounds__(128) quant_decode_kernel(QuantDecodeArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    using R = QuantRecord<D, kFp4>;
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int seq = blockIdx.y;
    const int hq = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (hq >= a.hq) return;
    const int h = hq / a.group;
    int ctx = a.context_lens[seq];
    if (ctx > a.max_ctx) {
        if (lane == 0) flag_error(a.err, PKV_DEVERR_LENGTH);
        ctx = a.max_ctx;
    }
    const int lo = a.window > 0 && ctx > a.window ? ctx - a.window : 0;
    const float kg = kFp4 ? a.k_scale[h] : 1.f, vg = kFp4 ? a.v_scale[h] : 1.f;
    const size_t row0 = static_cast<size_t>(seq) * a.hq + hq;
    float q[E], o[E] = {};
#pragma unroll
    for (int e = 0; e < E; ++e)
        q[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[row0 * D + lane * E + e]) * a.sm_scale * kg;
    float m = a.sinks ? a.sinks[hq] : -INFINITY;
    float l = a.sinks ? 1.f : 0.f;
    for (int t = lo; t < ctx; ++t) {
        const int b = t / kBlockSize, r = t % kBlockSize;
        int blk = a.block_tables[static_cast<size_t>(seq) * a.mbps + (a.ring > 0 ? b % a.ring : b)];
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
            blk = 0;
        }
        const size_t at = (static_cast<size_t>(blk) * a.hkv + h) * R::kBytes;
        const uint8_t* kr = static_cast<const uint8_t*>(a.k_pool) + at;
        const uint8_t* vr = static_cast<const uint8_t*>(a.v_pool) + at;
        float k[E], v[E], x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            k[e] = quant_value<D, kFp4>(kr, r, lane * E + e, 1.f);
            v[e] = quant_value<D, kFp4>(vr, r, lane * E + e, vg);
            x += q[e] * k[e];
        }
#pragma unroll
        for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, s);
        const float mn = fmaxf(m, x);
        const float keep = m == -INFINITY ? 0.f : expf(m - mn), p = expf(x - mn);
        l = l * keep + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * keep + p * v[e];
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        static_cast<__nv_bfloat16*>(a.out)[row0 * D + lane * E + e] = __float2bfloat16_rn(o[e] * inv);
    if (a.lse_out && lane == 0) a.lse_out[row0] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <int D, bool kFp4>
cudaError_t launch_t(const QuantDecodeArgs& a, cudaStream_t stream) {
    return launch_pdl(quant_decode_kernel<D, kFp4>, dim3((a.hq + 3) / 4, a.num_seqs), dim3(128), 0, stream, a);
}

}  // namespace

cudaError_t launch_quant_decode(const QuantDecodeArgs& a, cudaStream_t stream) {
    if (a.d == 64) return a.fp4 ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
    return a.fp4 ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
}

}  // namespace pkv
