// The 4-bit history: the launch functions that api.cu calls after validating arguments, where an INT4
// pool's rows lie, and what every kernel on them shares.
#pragma once

#include "oscar_int4.h"
#include "oscar_internal.cuh"

namespace oscar {

constexpr int kRow4 = kHeadDim / 2;                   // bytes of one row's codes
constexpr int kSms = 152;                             // of the one GPU that this is built for: launch rules count with them

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

// ---------------------------------------------------------------- launches --

struct Int4PoolView {
    uint8_t *codes_k, *codes_v;
    uint16_t *scale_zero;
    int n_pages;
};

// New tokens' heads: token i at q + i * q_stride elements (q NULL: keys and values only).
struct AppendInput {
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;
};
cudaError_t launch_append(const oscar_layout_t &L, const AppendInput &in, int n, const uint16_t *wq, const uint16_t *wk,
                          float eps, const float *rope, int rope_rows, int rot, bool pairs, Bf16PoolView pool,
                          const int32_t *pt, int max_pages, int batch, const int32_t *req, const int32_t *pos,
                          const int32_t *rope_pos, uint16_t *q_out, int32_t *status, cudaStream_t st);

cudaError_t launch_demote4(const oscar_layout_t &L, Bf16PoolView src, const int32_t *bpt, Int4PoolView dst,
                           const int32_t *ipt, int max_pages, int batch, const int32_t *begin, const int32_t *end,
                           float cK, float cV, int32_t *status, cudaStream_t st);
cudaError_t launch_promote4(const oscar_layout_t &L, Int4PoolView src, const int32_t *ipt, Bf16PoolView dst,
                            const int32_t *bpt, int max_pages, int batch, const int32_t *begin, const int32_t *end,
                            int32_t *status, cudaStream_t st);

// What decode attention and the attention weights read: one query per request, both pools.
struct Attn4Input {
    const uint16_t *q;
    Bf16PoolView bf;
    const int32_t *bpt;
    Int4PoolView i4;
    const int32_t *ipt;
    int max_pages;
    const int32_t *seq_len, *hist_end;
    float sm_scale;
};
int suggest_splits4(const oscar_layout_t &L, int batch, int max_hist, int sm_count);
// counters: NULL (the merge, if any, is a second launch) or int32 [batch * n_kv_heads], zero and left zero
cudaError_t launch_decode4(const oscar_layout_t &L, const Attn4Input &in, int batch, PartialsView out, uint16_t *o,
                           float *of, float *lse, int32_t *counters, int32_t *status, cudaStream_t st);
cudaError_t launch_mass4(const oscar_layout_t &L, const Attn4Input &in, int batch, const float *lse, float *mass,
                         int32_t *status, cudaStream_t st);

cudaError_t launch_evict(const oscar_layout_t &L, Int4PoolView src, const int32_t *spt, Int4PoolView dst,
                         const int32_t *dpt, int max_pages, int batch, const int32_t *seq_len, const int32_t *hist_end,
                         const int32_t *keep, const float *mass, float *mass_out, int32_t *kept, int kept_stride,
                         int32_t *status, cudaStream_t st);

}  // namespace oscar
