// decode.cu -- decode attention with plain logits (decode_kernel.cuh).
#include "decode_kernel.cuh"

namespace pkv {

bool decode_uses_tickets(int splits) { return splits > kMaxClusterSplits; }

int decode_smem_bytes(int d, int fp8) {
    if (d == 64) return fp8 ? DecodeCfg<64, true>::kSmemBytes : DecodeCfg<64, false>::kSmemBytes;
    return fp8 ? DecodeCfg<128, true>::kSmemBytes : DecodeCfg<128, false>::kSmemBytes;
}

cudaError_t launch_decode(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          cudaStream_t stream) {
    return launch_decode_any<false>(a, kmap, vmap, stream);
}

}  // namespace pkv
