// score_prefill.cu -- ragged prefill whose logits are capped by a tanh or fall with
// the distance to the key, with a prefix that its own positions see whole:
// prefill_tc_kernel.cuh and short_query_kernel.cuh under a score rule.
#include "prefill_tc_kernel.cuh"
#include "short_query_kernel.cuh"

namespace pkv {

cudaError_t launch_score_prefill_tc(const PrefillArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                    const CUtensorMap& vmap, cudaStream_t stream) {
    return launch_prefill_tc_any<true>(a, qmap, kmap, vmap, stream);
}

cudaError_t launch_score_short_query(const PrefillArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                     cudaStream_t stream) {
    return launch_sq_any<true>(a, kmap, vmap, stream);
}

}  // namespace pkv
