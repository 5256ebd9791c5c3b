// score_prefill.cu -- ragged prefill under a score rule without a bias: logits capped by
// a tanh, a prefix that its own positions see whole, sinks (prefill_tc_kernel.cuh,
// short_query_kernel.cuh); score_prefill_bias.cu has the kernels with a bias.
#include "prefill_tc_kernel.cuh"
#include "short_query_kernel.cuh"

namespace pkv {

cudaError_t launch_score_prefill_tc(const PrefillArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                    const CUtensorMap& vmap, cudaStream_t stream) {
    if (a.slopes) return launch_bias_prefill_tc(a, qmap, kmap, vmap, stream);
    return a.cap > 0.f ? launch_prefill_tc_any<kTcCap>(a, qmap, kmap, vmap, stream)
                       : launch_prefill_tc_any<kTcRule>(a, qmap, kmap, vmap, stream);
}

cudaError_t launch_score_short_query(const PrefillArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                     cudaStream_t stream) {
    return launch_sq_any<true>(a, kmap, vmap, stream);
}

}  // namespace pkv
