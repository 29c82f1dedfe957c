// Decode attention and attention weights over an INT4 history: the host side of attn_int4.cuh.

#include <algorithm>

#include "attn_int4_args.cuh"
#include "tma.cuh"

namespace oscar {
namespace {

bool rows_tensor_map(CUtensorMap *tm, const uint8_t *base, long long rows, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {kRow4, (cuuint64_t)rows}, strides[1] = {kRow4};
    const cuuint32_t box[2] = {kRow4, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch(const oscar_layout_t &L, const Attn4Input &in, Attn4Args a, bool mass, int batch, cudaStream_t st) {
    a.q = in.q;
    a.bf = in.bf;
    a.bpt = in.bpt;
    a.sz = in.i4.scale_zero;
    a.i4_pages = in.i4.n_pages;
    a.ipt = in.ipt;
    a.max_pages = in.max_pages;
    a.page_shift = page_shift(L);
    a.n_kv = L.n_kv_heads;
    a.sink = L.sink;
    a.seq_len = in.seq_len;
    a.hist_end = in.hist_end;
    a.scale2 = in.sm_scale * kLog2e;
    CUtensorMap tmk, tmv;
    const long long rows = (long long)in.i4.n_pages * L.n_kv_heads * L.page_size;
    const int box = L.page_size < kBlock ? L.page_size : kBlock;
    if (!rows_tensor_map(&tmk, in.i4.codes_k, rows, box) || !rows_tensor_map(&tmv, in.i4.codes_v, rows, box))
        return cudaErrorInvalidValue;
    switch (L.gqa) {
        case 1: return launch_attn4<1>(a, L.group, mass, tmk, tmv, batch, st);
        case 2: return launch_attn4<2>(a, L.group, mass, tmk, tmv, batch, st);
        case 4: return launch_attn4<4>(a, L.group, mass, tmk, tmv, batch, st);
        default: return launch_attn4<8>(a, L.group, mass, tmk, tmv, batch, st);
    }
}

}  // namespace

// Splits of at least 256 tokens (8 blocks): shorter ones cost more in the merge than they save.  Up to that
// bound one CTA of 16 warps an SM where that fills nine SMs in ten; else, while the heads leave each four
// splits, one wave of CTAs of 8 warps, two an SM; else about six waves of those, so that requests of
// different lengths finish evenly.  (100K tokens, 8 heads: 30.8 us with 19 splits of 16 warps, 35.1 with 37 of
// 8; 4 x 131K: 145 us with 9 splits in one wave, 152 with 4 of 16 warps, 196 with 10; ragged batch of 32:
// 497, 494, 488, 493 and 497 us with 5, 6, 7, 8 and 10.)
int suggest_splits4(const oscar_layout_t &L, int batch, int max_hist, int sm_count) {
    const long long per = (long long)batch * L.n_kv_heads, wide = sm_count / per, slots = 2LL * sm_count;
    long long want = wide * per * 10 >= sm_count * 9LL ? wide : per * 4 <= slots ? slots / per : 6 * slots / per;
    const long long most = ((long long)max_hist + 255) / 256;
    if (want > most) want = most;
    return (int)(want < 1 ? 1 : want > 1024 ? 1024 : want);
}

cudaError_t launch_decode4(const oscar_layout_t &L, const Attn4Input &in, int batch, PartialsView out, uint16_t *o,
                           float *of, float *lse, int32_t *counters, int32_t *status, cudaStream_t st) {
    const bool merge = o || of;
    Attn4Args a{};
    a.out = out;
    a.status = status;
    a.counters = merge ? counters : nullptr;
    a.o = o;
    a.of = of;
    a.o_lse = lse;
    if (cudaError_t e = launch(L, in, a, false, batch, st)) return e;
    return merge && !counters ? launch_merge(L, out, nullptr, batch, o, of, lse, st) : cudaSuccess;
}

cudaError_t launch_mass4(const oscar_layout_t &L, const Attn4Input &in, int batch, const float *lse, float *mass,
                         int32_t *status, cudaStream_t st) {
    Attn4Args a{};
    // no merge to pay for: about two waves of CTAs of 4 warps even where one would hold the splits (a ragged
    // batch of 8: 135, 89, 80 and 80 us with 4, 9, 19 and 28; of 8 warps: 100, 86, 85 and 90)
    const long long per = (long long)batch * L.n_kv_heads, tokens = in.max_pages * (long long)L.page_size;
    const int S = suggest_splits4(L, batch, (int)tokens, kSms);
    a.out.S = per > kSms / 4 ? (int)std::max<long long>(1, std::min({1024LL, 8LL * kSms / per, (tokens + 255) / 256})) : S;
    a.lse = lse;
    a.mass = mass;
    a.status = status;
    return launch(L, in, a, true, batch, st);
}

}  // namespace oscar
