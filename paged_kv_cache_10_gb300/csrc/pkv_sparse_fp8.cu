// pkv_sparse_fp8.cu -- sparse decode over fp8 E4M3 pools: the dense kernels
// walking each (sequence, KV head)'s list of selected blocks.
#include "pkv_decode_mma.cuh"

namespace pkv {
cudaError_t launch_decode_sparse_fp8(const DecodeParams& p, int G, int q_dtype, const CUtensorMap* tk,
                                     const CUtensorMap* tv, cudaStream_t st) {
    if (q_dtype == PKV_BF16)
        return tk ? launch_decode_mma_family<E4M3, BF16, true>(p, G, *tk, *tv, st)
                  : launch_decode_family<E4M3, BF16, true>(p, G, st);
    return tk ? launch_decode_mma_family<E4M3, F16, true>(p, G, *tk, *tv, st)
              : launch_decode_family<E4M3, F16, true>(p, G, st);
}
}  // namespace pkv
