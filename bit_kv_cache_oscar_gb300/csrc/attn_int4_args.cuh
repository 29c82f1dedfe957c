// What the INT4 attention kernels take, shared by their instantiations and the host side.
#pragma once

#include <cuda.h>

#include "int4.cuh"

namespace oscar {

constexpr int kSms = 152;
constexpr int kBlock = 32;                       // tokens of one stage

struct Attn4Args {
    const uint16_t *q;
    Bf16PoolView bf;
    const int32_t *bpt;
    const uint16_t *sz;
    int i4_pages;
    const int32_t *ipt;
    int max_pages, page_shift, n_kv, sink;
    const int32_t *seq_len, *hist_end;
    float scale2;
    PartialsView out;
    uint16_t *o;
    float *of, *o_lse;
    int32_t *counters;
    const float *lse;          // weights only
    float *mass;
    int32_t *status;
};

// One instantiation per number of query heads a kv head (G), each in a file of its own.
template <int G>
cudaError_t launch_attn4(const Attn4Args &a, int group, bool mass, const CUtensorMap &tmk, const CUtensorMap &tmv, int batch,
                         cudaStream_t st);

}  // namespace oscar
