// fd_api.h -- what the C ABI's translation units share: the workspace behind
// fd_workspace and the structural checks of a tensor descriptor.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "fd.h"

struct fd_workspace {
    void *base;
    size_t bytes;
    int64_t max_segments;
    int32_t max_rows, head_dim, max_ctas;
    int32_t *counters;       // [max_segments], zero between launches
    int32_t *groups;         // [max_segments + max_ctas], likewise
    int32_t *status;
    float *partials;
    size_t partial_floats;
    int device;
    std::mutex turn;         // held while a call queues its launches: what one of
                             // them leaves in the partials for the next is not
                             // overwritten by another thread's call between them
};

namespace fd {

constexpr uint64_t kDefaultWaitNs = 2000000000ull;   // 2 s per internal wait

inline int esize(int32_t dt) {
    switch (dt) {
        case FD_BF16: return 2;
        case FD_F32: return 4;
        case FD_I8: return 1;
        case FD_I32: return 4;
        case FD_U8: return 1;
        case FD_E4M3: return 1;
        default: return 0;
    }
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Basic structural check of a tensor descriptor.
inline int check_tensor(const fd_tensor *t, int ndim) {
    if (!t || !t->data || t->ndim != ndim || esize(t->dtype) == 0) return FD_ERR_ARG;
    for (int i = 0; i < ndim; ++i)
        if (t->shape[i] < 0 || t->stride[i] < 0) return FD_ERR_ARG;
    return FD_OK;
}

// Streaming multiprocessors of the current device (0 on error).
int sm_count_current();

}  // namespace fd
