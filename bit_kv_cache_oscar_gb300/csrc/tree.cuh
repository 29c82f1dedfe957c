// A step of speculative decoding: the launch functions that api.cu calls after validating arguments.
#pragma once

#include "int4.cuh"
#include "oscar_tree.h"

namespace oscar {

// The trees of a batch: rows [begin[b], begin[b + 1]) of the n node rows are request b's.
struct TreeInput {
    const int32_t *begin;
    int n, max_nodes;
};

// Request b's first row and node count; 0 nodes (flagged) for a range that is not one.
__device__ __forceinline__ int read_nodes(const TreeInput &t, int b, int32_t *status, int &first) {
    first = t.begin[b];
    const int end = t.begin[b + 1];
    if (first >= 0 && end >= first && end <= t.n && end - first <= t.max_nodes) return end - first;
    if (threadIdx.x == 0) flag_status(status, OSCAR_DEV_BAD_LENGTH);
    first = 0;
    return 0;
}

int suggest_splits_tree(const oscar_layout_t &L, int batch, int max_nodes, int max_hist, int sm_count);
// max_hist: tokens of the longest history, as the splits were suggested for
cudaError_t launch_tree_attention(const oscar_layout_t &L, const Attn4Input &in, const TreeInput &t, const int32_t *mask, int mask_words,
                                  int max_hist, int batch, PartialsView part, uint16_t *out, float *lse, int32_t *status, cudaStream_t st);

struct SampleInput {
    const void *logits;
    int dtype;
    long long stride;
    int rows, vocab;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
};
cudaError_t launch_sample(const SampleInput &in, int32_t *tokens, cudaStream_t st);

struct AcceptInput {
    const int32_t *target, *draft, *parents, *seq_len;
};
struct AcceptOutput {
    int32_t *accepted, *path, *tokens, *new_len;
    int stride;
};
cudaError_t launch_tree_accept(const oscar_layout_t &L, const AcceptInput &in, const TreeInput &t, int batch, const AcceptOutput &out,
                               const oscar_bf16_pool_t *pools, int n_pools, const int32_t *pt, int max_pages, int32_t *status, cudaStream_t st);

}  // namespace oscar
