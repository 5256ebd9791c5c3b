// score_prefill_bias.cu -- ragged prefill whose logits fall with the distance to the key,
// with or without a cap (prefill_tc_kernel.cuh).
#include "prefill_tc_kernel.cuh"

namespace pkv {

cudaError_t launch_bias_prefill_tc(const PrefillArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                   const CUtensorMap& vmap, cudaStream_t stream) {
    return a.cap > 0.f ? launch_prefill_tc_any<kTcBoth>(a, qmap, kmap, vmap, stream)
                       : launch_prefill_tc_any<kTcBias>(a, qmap, kmap, vmap, stream);
}

}  // namespace pkv
