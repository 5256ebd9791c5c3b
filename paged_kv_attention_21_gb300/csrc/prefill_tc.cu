// prefill_tc.cu -- ragged prefill with plain logits (prefill_tc_kernel.cuh).
#include "prefill_tc_kernel.cuh"

namespace pkv {

int prefill_tc_q_tile(int group) { return group >= 1 && group <= kTcM ? kTcM / group : 0; }

cudaError_t launch_prefill_tc(const PrefillArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                              const CUtensorMap& vmap, cudaStream_t stream) {
    return launch_prefill_tc_any<kTcPlain>(a, qmap, kmap, vmap, stream);
}

}  // namespace pkv
