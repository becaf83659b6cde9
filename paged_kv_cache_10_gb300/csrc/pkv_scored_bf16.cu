// pkv_scored_bf16.cu -- scored decode over bf16 pools (bf16 q): the dense kernels
// with capped, biased and masked scores.
#include "pkv_decode_mma.cuh"

namespace pkv {
cudaError_t launch_decode_scored_bf16(const DecodeParams& p, int G, const CUtensorMap* tk, const CUtensorMap* tv,
                                     cudaStream_t st) {
    return tk ? launch_decode_mma_family<BF16, BF16, false, true>(p, G, *tk, *tv, st)
              : launch_decode_family<BF16, BF16, false, true>(p, G, st);
}
}  // namespace pkv
