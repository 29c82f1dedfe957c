// What the tree attention kernels take and share.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "pairs.cuh"
#include "ptx.cuh"
#include "tree.cuh"

namespace oscar {

constexpr int kBlock4 = 32;                      // tokens of one box of the INT4 pool

constexpr uint32_t kM0 = 0x000F000Fu, kM1 = 0x00F000F0u;    // nibbles 0 and 1 of a word's two halves

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Codes of nibbles 0 (low) or 1 (high) of a word's two halves, less 8: (1024 + n) - 1032, (1024 + 16 n) / 16 - 72.
__device__ __forceinline__ uint32_t centred_low(uint32_t w) {
    uint32_t d;
    asm("{\n.reg .b32 t;\nlop3.b32 t, %1, 0x000F000F, 0x64006400, 0xEA;\nadd.f16x2 %0, t, %2;\n}" : "=r"(d) : "r"(w), "r"(0xE408E408u));
    return d;
}
__device__ __forceinline__ uint32_t centred_high(uint32_t w) {
    uint32_t d;
    asm("{\n.reg .b32 t;\nlop3.b32 t, %1, 0x00F000F0, 0x64006400, 0xEA;\nfma.rn.f16x2 %0, t, %2, %3;\n}"
        : "=r"(d) : "r"(w), "r"(0x2C002C00u), "r"(0xD480D480u));
    return d;
}

struct TreeArgs {
    const uint16_t *q;
    TreeInput t;
    const int32_t *mask;
    int mask_words;
    Bf16PoolView bf;
    const int32_t *bpt;
    const uint8_t *codes_k, *codes_v;
    const uint16_t *sz;
    int i4_pages;
    const int32_t *ipt;
    int max_pages, page_shift, n_kv, G, sink;
    const int32_t *seq_len, *hist_end;
    float scale2;
    PartialsView part;                           // rows are (node row, query head)
    uint16_t *o;
    float *lse;
    int32_t *status;
};

// A request's lengths and nodes as every kernel of the call reads them; n = 0: it is skipped.
struct TreeRequest {
    int first, n, T, he;
    __device__ __forceinline__ TreeRequest(const TreeArgs &a, int b) {
        n = read_nodes(a.t, b, a.status, first);
        T = he = 0;
        if (n == 0) return;
        read_lengths(a.seq_len, a.hist_end, b, a.sink, a.max_pages << a.page_shift, a.status, T, he);
        if (T + n > a.max_pages << a.page_shift) {
            if (threadIdx.x == 0) flag_status(a.status, OSCAR_DEV_BAD_LENGTH);
            n = 0;
        }
    }
};

// Row index of (node row, query head) in out, lse and, times S + 1, in the partials.
__device__ __forceinline__ size_t tree_row(const TreeArgs &a, const TreeRequest &r, int h, int row) {
    return ((size_t)(r.first + row / a.G) * a.n_kv + h) * a.G + row % a.G;
}

// Every slot of the partials with the history on the 5th-generation tensor cores (group 128), 128 query rows of a kv head at a time;
// where its grid fits.
bool tree_tc_fits(const TreeArgs &a, int max_rows, int batch);
cudaError_t launch_tree_tc(const TreeArgs &a, int max_rows, int batch, cudaStream_t st);

}  // namespace oscar
