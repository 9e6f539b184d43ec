// fd_serve.h -- launch parameters of the calls around decode: rows appended to
// a bf16 or int8 cache, attention of a chunk of new tokens, beam selection.
#pragma once

#include <cuda_runtime.h>

#include "fd_internal.h"

namespace fd {

// A bf16 or int8 cache, flat or paged (strides in elements: sequence or page,
// kv head, row).
struct KvCache {
    void *k, *v;
    float *k_scale, *v_scale;      // int8
    int64_t ks[3], vs[3], kss[3], vss[3];
    int64_t lead, cap;             // sequences or pages; positions
    int32_t Hkv, d, int8;
    const int32_t *block_table;    // null: flat
    int32_t page_size, page_shift, max_pages;   // page_shift -1: no power of two
};

// fd_rows.cu
struct RowsParams {
    KvCache c;
    int32_t B, n, Hq, r, interleaved;
    int64_t positions;             // rows of the rotation table
    const float *rope; int64_t rope_stride;
    const uint16_t *k_new, *v_new, *q;
    uint16_t *q_out;
    int64_t kns[3], vns[3], qs[3], qos[3];
    const int32_t *new_lengths, *lengths;
    int32_t *lengths_out, *status;
    int32_t *grid;                 // non-null: lengths_out is lengths, so the last
                                   // block to finish writes it
};
int launch_append_rows(const RowsParams &p, cudaStream_t st);

// fd_prefill.cu, fd_prefill_tc.cu (launchers: fd_prefill.h)
struct PrefillParams {
    KvCache c;
    int32_t B, n, Hq, g, causal;
    float scale_log2;              // scale * log2(e)
    const uint16_t *q; int64_t qs[3];
    uint16_t *out; int64_t os[3];
    const int32_t *lengths, *new_lengths;
    int32_t *status;
    float *partials;
    int32_t per;                   // tcgen05: set by the launch
    int32_t wait_rounds;           // tcgen05: bound on each internal wait, in rounds of about 1 us
};

// fd_beam.cu
struct BeamParams {
    const void *logits; int64_t ls[2];   // strides of request and beam
    int32_t bf16;
    int32_t B, K, V, n_out;
    const float *scores;
    const int32_t *finished;
    int32_t end_token;
    float *scores_out;
    int32_t *beams_out, *tokens_out;
    char *scratch;
    int32_t *tickets;                    // [B], zero between launches
};
int64_t beam_scratch_bytes(int64_t B, int K, int64_t V, int n_out);
int launch_beam_select(const BeamParams &p, cudaStream_t st);

}  // namespace fd
