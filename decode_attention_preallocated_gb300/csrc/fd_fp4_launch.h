// fd_fp4_launch.h -- launch parameters of the 4-bit cache kernels.
#pragma once

#include <cuda_runtime.h>

#include "fd_internal.h"

namespace fd {

// Decode over a 4-bit cache (fd_fp4_decode.cuh).  `p` describes the launch to
// the split partitioner: p.k / p.v are the code caches (strides in bytes), a
// segment is (sequence, kv head, part of the kv head's query rows), p.Hkv
// counts (kv head, part) pairs and p.rows the rows of a part.
struct Fp4Params {
    Params p;
    const uint8_t *ks; int64_t kss[3];   // e4m3 scales, strides in bytes
    const uint8_t *vs; int64_t vss[3];
    float v_global;
    int32_t parts;       // parts of each kv head's query rows
    int32_t all_rows;    // g * n_q
    int32_t q_aligned8;  // q's base and strides are multiples of 8 bytes
    int32_t *groups;     // counters of the joins of 8 pieces, one per slot, zero
                         // between launches
};
// Rows that one part holds at most.
constexpr int kFp4PartRows = 32;
// What the start and end of a piece are charged, in positions; at least two of
// its tiles.  24 rows at d = 256 (tiles of 128), ragged: 79.5 us with 2 tiles,
// 77.7 with 4, 78.8 with 6.  4 rows at d = 128 (256), 64 ragged sequences over
// pages: 61 with 2, 63 with 3, 66 with 4.  16 rows at d = 128 (192): 24.9 with
// 2, 26.2 with 3.
constexpr int kFp4PiecePositions = 512;
inline int fp4_seg_units(int tile) { return kFp4PiecePositions / tile > 2 ? kFp4PiecePositions / tile : 2; }
// Cache positions per tile of the partitioner, and blocks that an SM holds, for
// parts of this many rows.
int fp4_tile_tokens(int d, int rows);
int fp4_blocks_per_sm(int rows);
int launch_fp4_decode(const Fp4Params &p, int num_ctas, cudaStream_t stream);
int launch_fp4_decode_f32(const Fp4Params &p, int num_ctas, cudaStream_t stream);   // its fp32 outputs

// The rows of a 4-bit cache between bf16 (or fp32) and its own format
// (fd_fp4_rows.cu).  Cache strides in bytes: [sequence or page, kv head, row].
struct Fp4Rows {
    int32_t B, n, Hkv, d;
    int32_t aligned32;            // the bf16 rows' bases and strides are multiples of 32 bytes
    int64_t cap;
    // (row, kv head) units per block, and how far the units of one thread lie
    // apart; set by the launch
    int64_t span;
    int32_t step_i, step_hk;
    uint8_t *k, *v, *ks, *vs;
    int64_t kst[3], vst[3], kss[3], vss[3];
    float k_global, v_global;
    const int32_t *block_table;   // null: flat
    int32_t page_size, page_shift, max_pages;
    int64_t num_pages;
    const int32_t *lengths;       // append: filled positions; read: positions that exist
    int32_t *status;
    // append: new rows [B, n, Hkv, d] bf16 (strides in elements), how many of
    // them each sequence really has (null: n), and where the new lengths go
    // (null: nowhere)
    const uint16_t *k_new, *v_new;
    int64_t kns[3], vns[3];
    const int32_t *new_lengths;
    int32_t *lengths_out;
    int32_t *grid;                // non-null: lengths_out overlaps lengths, so the
                                  // last block to finish writes it
    // read: first position of each sequence (null: 0) and [B, n, Hkv, d]
    // outputs, bf16 or fp32 (strides in elements)
    const int32_t *start;
    void *k_out, *v_out;
    int64_t kos[3], vos[3];
    int32_t out_f32;
};
int launch_fp4_append(Fp4Rows p, cudaStream_t stream);
int launch_fp4_read(Fp4Rows p, cudaStream_t stream);

}  // namespace fd
