// fd_fp4_decode_f32.cu -- the decode kernel over a 4-bit cache for fp32 outputs.
#include "fd_fp4_decode.cuh"

namespace fd {

int launch_fp4_decode_f32(const Fp4Params &p, int G, cudaStream_t st) { return launch_decode<true>(p, G, st); }

}  // namespace fd
