// pkv_scored_int8.cu -- scored decode over 8-bit integer-coded pools.
#include "pkv_decode_int.cuh"

namespace pkv {
cudaError_t launch_decode_scored_int8(const DecodeParams& p, int G, int q_dtype, cudaStream_t st) {
    return launch_decode_int<8, true>(p, G, q_dtype, st);
}
}  // namespace pkv
