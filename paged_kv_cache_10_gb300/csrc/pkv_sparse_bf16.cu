// pkv_sparse_bf16.cu -- sparse decode over bf16 pools: the dense kernels walking
// each (sequence, KV head)'s list of selected blocks.
#include "pkv_decode_mma.cuh"

namespace pkv {
cudaError_t launch_decode_sparse_bf16(const DecodeParams& p, int G, const CUtensorMap* tk, const CUtensorMap* tv,
                                      cudaStream_t st) {
    return tk ? launch_decode_mma_family<BF16, BF16, true>(p, G, *tk, *tv, st)
              : launch_decode_family<BF16, BF16, true>(p, G, st);
}
}  // namespace pkv
