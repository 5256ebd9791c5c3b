// score_decode.cu -- decode attention whose logits are capped by a tanh or fall
// with the distance to the key: decode_kernel.cuh under a score rule.
#include "decode_kernel.cuh"

namespace pkv {

cudaError_t launch_score_decode(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                cudaStream_t stream) {
    return launch_decode_any<true>(a, kmap, vmap, stream);
}

}  // namespace pkv
