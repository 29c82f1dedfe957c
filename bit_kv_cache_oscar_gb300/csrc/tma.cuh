// Tensor-map encoding for the TMA (cp.async.bulk.tensor) kernels of liboscar.so.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace oscar {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled from the driver, looked up once per process through the runtime
// (nullptr when the driver does not provide it).
inline EncodeTiledFn driver_encode_fn() {
    static EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        EncodeTiledFn f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            f = reinterpret_cast<EncodeTiledFn>(p);
        cudaGetLastError();
        return f;
    }();
    return fn;
}

// The driver's call wants a context, which a thread whose first CUDA call this is does not have yet: the
// runtime binds its device's there, and the call is made again.
inline CUresult encode_tiled(CUtensorMap *tm, CUtensorMapDataType type, cuuint32_t rank, void *base, const cuuint64_t *dims,
                             const cuuint64_t *strides, const cuuint32_t *box, const cuuint32_t *estr, CUtensorMapInterleave il,
                             CUtensorMapSwizzle sw, CUtensorMapL2promotion l2, CUtensorMapFloatOOBfill oob) {
    const EncodeTiledFn fn = driver_encode_fn();
    const CUresult r = fn(tm, type, rank, base, dims, strides, box, estr, il, sw, l2, oob);
    int dev = 0;
    if (r == CUDA_SUCCESS || cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return r;
    return fn(tm, type, rank, base, dims, strides, box, estr, il, sw, l2, oob);
}
inline EncodeTiledFn encode_fn() { return driver_encode_fn() ? &encode_tiled : nullptr; }

}  // namespace oscar
