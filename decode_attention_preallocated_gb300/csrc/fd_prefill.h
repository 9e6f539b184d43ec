// fd_prefill.h -- launchers of the attention of a chunk of new tokens.
#pragma once

#include "fd_serve.h"

namespace fd {

// Warp-level matrix instructions, every layout (fd_prefill.cu).
int launch_prefill_simple(const PrefillParams &p, cudaStream_t st);
// tcgen05 (fd_prefill_tc.cu): -2 where a tensor map cannot describe the layout.
bool prefill_tc_supports(const PrefillParams &p);
// Floats of one partial slot; a launch of `grid` blocks uses two a block.
int64_t prefill_slot_floats(int d);
int launch_prefill_tc(const PrefillParams &p, int grid, cudaStream_t st);

}  // namespace fd
