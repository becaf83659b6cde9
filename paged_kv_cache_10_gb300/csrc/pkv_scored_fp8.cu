// pkv_scored_fp8.cu -- scored decode over fp8 E4M3 pools (bf16 or f16 q): the
// dense kernels with capped, biased and masked scores.
#include "pkv_decode_mma.cuh"

namespace pkv {
cudaError_t launch_decode_scored_fp8(const DecodeParams& p, int G, int q_dtype, const CUtensorMap* tk,
                                     const CUtensorMap* tv, cudaStream_t st) {
    if (q_dtype == PKV_BF16)
        return tk ? launch_decode_mma_family<E4M3, BF16, false, true>(p, G, *tk, *tv, st)
                  : launch_decode_family<E4M3, BF16, false, true>(p, G, st);
    return tk ? launch_decode_mma_family<E4M3, F16, false, true>(p, G, *tk, *tv, st)
              : launch_decode_family<E4M3, F16, false, true>(p, G, st);
}
}  // namespace pkv
