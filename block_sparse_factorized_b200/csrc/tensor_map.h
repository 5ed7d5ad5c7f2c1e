// tensor_map.h -- the driver's tensor-map encoder, looked up through the runtime (host only).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace st {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn lookup_encode()
{
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        return reinterpret_cast<EncodeTiledFn>(ptr);
    return nullptr;
}

// The driver's tensor-map encoder, looked up once (thread-safe static initialisation; a failed
// lookup is retried by the next call).
inline EncodeTiledFn encode_fn()
{
    static std::atomic<EncodeTiledFn> fn{lookup_encode()};
    EncodeTiledFn f = fn.load(std::memory_order_acquire);
    if (!f && (f = lookup_encode())) fn.store(f, std::memory_order_release);
    return f;
}

inline bool encode(CUtensorMap *m, const void *base, CUtensorMapDataType dt, cuuint32_t rank,
            const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
            CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B)
{
    const cuuint32_t es[4] = {1, 1, 1, 1};
    auto run = [&]() {
        return encode_fn()(m, dt, rank, const_cast<void *>(base), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (run()) return true;
    // The encoder is a driver call: it fails where the calling thread has no context current yet, as
    // where this is the thread's first CUDA call (a framework's backward thread); the runtime makes the
    // device's own current.
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && run();
}

}  // namespace st
