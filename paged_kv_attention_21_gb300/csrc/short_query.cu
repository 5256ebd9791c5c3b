// short_query.cu -- a few query tokens per sequence, plain logits
// (short_query_kernel.cuh).
#include "short_query_kernel.cuh"

namespace pkv {

cudaError_t launch_short_query(const PrefillArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                               cudaStream_t stream) {
    return launch_sq_any<false>(a, kmap, vmap, stream);
}

}  // namespace pkv
