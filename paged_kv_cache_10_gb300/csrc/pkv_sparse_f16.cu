// pkv_sparse_f16.cu -- sparse decode over f16 pools: the dense kernels walking
// each (sequence, KV head)'s list of selected blocks.
#include "pkv_decode_mma.cuh"

namespace pkv {
cudaError_t launch_decode_sparse_f16(const DecodeParams& p, int G, const CUtensorMap* tk, const CUtensorMap* tv,
                                     cudaStream_t st) {
    return tk ? launch_decode_mma_family<F16, F16, true>(p, G, *tk, *tv, st)
              : launch_decode_family<F16, F16, true>(p, G, st);
}
}  // namespace pkv
