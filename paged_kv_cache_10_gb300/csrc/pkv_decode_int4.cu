// pkv_decode_int4.cu -- decode attention instantiations for 4-bit integer-coded pools.
#include "pkv_decode_int.cuh"

namespace pkv {
cudaError_t launch_decode_int4(const DecodeParams& p, int G, int q_dtype, cudaStream_t st) {
    return launch_decode_int<4>(p, G, q_dtype, st);
}
}  // namespace pkv
