// fd_fp4_decode.cu -- the decode kernel over a 4-bit cache for bf16 outputs, and
// what the host asks of its shapes.
#include "fd_fp4_decode.cuh"

namespace fd {

int fp4_tile_tokens(int d, int rows) {
    static const int tile[4] = {Cfg<1, 1>::TILE, Cfg<1, 2>::TILE, Cfg<1, 3>::TILE, Cfg<1, 4>::TILE};
    return tile[(rows - 1) / 8] / (d / 128);   // pairs of warps at d = 256
}

int fp4_blocks_per_sm(int rows) { return rows <= 16 ? Cfg<1, 1>::OCC : Cfg<1, 3>::OCC; }

int launch_fp4_decode(const Fp4Params &p, int G, cudaStream_t st) {
    return p.p.out_f32 ? launch_fp4_decode_f32(p, G, st) : launch_decode<false>(p, G, st);
}

}  // namespace fd
