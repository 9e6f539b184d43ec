// fd_tensor_map.h -- host-side encoding of TMA tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>
#include <mutex>

namespace fd {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Tensor maps are encoded on the host for every launch; a decode loop passes
// the same caches (and often the same q) each step, so the last encodings
// are kept, keyed by every argument that goes into one.
struct MapKey {
    const void *base;
    uint32_t dtype, rank, swizzle, pad;
    cuuint64_t dims[4], strides[3];
    cuuint32_t box[4];
};

inline EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                                         cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<EncodeTiledFn>(ptr) : nullptr;
    }();
    return fn;
}

// cuTensorMapEncodeTiled wants a context that is current to the host thread.  The runtime
// makes the device's one so only with a thread's first call that needs it, which this may
// precede.
inline CUresult encode_tiled(CUtensorMap *m, CUtensorMapDataType dtype, cuuint32_t rank, void *base,
                             const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
                             const cuuint32_t *estr, CUtensorMapSwizzle swizzle) {
    const EncodeTiledFn fn = encode_fn();
    if (!fn) return CUDA_ERROR_NOT_SUPPORTED;
    const auto call = [&] {
        return fn(m, dtype, rank, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = call();
    if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) {
        int device;
        if (cudaGetDevice(&device) == cudaSuccess && cudaSetDevice(device) == cudaSuccess) r = call();
    }
    return r;
}

inline CUresult encode_cached(CUtensorMap *m, CUtensorMapDataType dtype, cuuint32_t rank, void *base,
                       const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
                       const cuuint32_t *estr, CUtensorMapSwizzle swizzle) {
    MapKey k;
    memset(&k, 0, sizeof k);
    k.base = base;
    k.dtype = (uint32_t)dtype;
    k.rank = rank;
    k.swizzle = (uint32_t)swizzle;
    for (cuuint32_t i = 0; i < rank; ++i) {
        k.dims[i] = dims[i];
        k.box[i] = box[i];
        if (i + 1 < rank) k.strides[i] = strides[i];
    }
    constexpr int kEntries = 32;
    static std::mutex mu;
    static MapKey keys[kEntries];
    static CUtensorMap maps[kEntries];
    static int used = 0, next = 0;
    {
        std::lock_guard<std::mutex> lk(mu);
        for (int i = 0; i < used; ++i)
            if (memcmp(&keys[i], &k, sizeof k) == 0) {
                *m = maps[i];
                return CUDA_SUCCESS;
            }
    }
    const CUresult r = encode_tiled(m, dtype, rank, base, dims, strides, box, estr, swizzle);
    if (r == CUDA_SUCCESS) {
        std::lock_guard<std::mutex> lk(mu);
        keys[next] = k;
        maps[next] = *m;
        next = (next + 1) % kEntries;
        if (used < kEntries) ++used;
    }
    return r;
}

}  // namespace fd
