// The 4-bit rows of an INT4 pool: where they lie, and the sizes every kernel on them shares.
#pragma once

#include "oscar_internal.cuh"

namespace oscar {

constexpr int kRow4 = kHeadDim / 2;                   // bytes of one row's codes

// Launch set up while the kernel before it in the stream still runs: every CTA of `kern` calls pdl_wait()
// before its first access to memory, so the order of the stream holds as for a plain launch.  The kernels
// launched like this do not let a next one start early themselves: what they write may be read before its
// own wait by a kernel launched under the launch-overlap switch.
template <typename... P, typename... A>
inline cudaError_t launch_ahead(void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// log2 of the page size (16, 32 or 64): positions are split by shifts, not by divisions.
inline int page_shift(const oscar_layout_t &L) { return L.page_size == 16 ? 4 : L.page_size == 32 ? 5 : 6; }

// Row index of (page, kv head, slot) in the pool's arrays: a page holds one head's tokens together.
__device__ __forceinline__ size_t row4(int page, int n_kv, int h, int page_shift, int slot) {
    return (((size_t)page * n_kv + h) << page_shift) + slot;
}

}  // namespace oscar
