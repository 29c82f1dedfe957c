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

// One wave of CTAs at first: of 16 warps, one an SM, or of 8, two an SM, by the tokens an SM gets (the
// latter takes 2.1 times as long a token of its split, and 500 tokens more).  A wave costs about 4.5 us, so
// only splits that are long in that wave (32K tokens, or 16K with 8 warps) are cut into more waves, which finish
// evenly: 8K tokens each, six waves at most.  Splits of at least 256 tokens (8 blocks): shorter ones cost more in the
// merge than they save.  8 heads, us: 1 x 100K 30.8 with 19 splits of 16 warps, 35.1 with 37 of 8; 4 x 131K 105
// with 9 splits (8 warps), 110 with 4 (16); 4 x 8K 16.9 and 15.9; 16 x 8K 34.8, 39, 44, 49 and 68 with 1, 2, 4, 7 and
// 14; 32 x 8K 64, 73, 75 and 89 with 1, 2, 4 and 7; lengths 22K to 32K, 32 requests: 213, 198, 182 and 187; 32 of
// 64K to 100K: 497, 494, 488, 493 and 497 with 5, 6, 7, 8 and 10.
int suggest_splits4(const oscar_layout_t &L, int batch, int max_hist, int sm_count) {
    const long long heads = (long long)batch * L.n_kv_heads, h = max_hist;
    const long long wide = sm_count / heads, narrow = std::max(1LL, 2LL * sm_count / heads);
    const bool is_wide = wide > 0 && 10 * h / wide <= 21 * h / narrow + 5000;
    long long want = is_wide ? wide : narrow;
    if (h > want * (is_wide ? 32768 : 16384)) want = std::max(want, std::min(h / 8192, 12LL * sm_count / heads));
    want = std::min(want, (h + 255) / 256);
    return (int)std::max(1LL, std::min(want, 1024LL));
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
    // no merge to pay for: CTAs of 16 warps, one an SM, where they fill nine SMs in ten; else of 4 warps, four an
    // SM, one wave, or two where that leaves splits of 1,200 tokens (8 heads, one and two waves: 4 x 32K 20.0 and
    // 23.3 us, 8 x 8K 12.8 and 15.9, 8 x 100K 97.6 and 90.0, 64 x 8K 78.9 and 68.6; 4 x 100K 49.5, of 8 warps 64.8)
    const long long heads = (long long)batch * L.n_kv_heads, tokens = in.max_pages * (long long)L.page_size;
    const long long wide = kSms / heads, wave = 4LL * kSms;
    long long want = 10 * wide * heads >= 9 * kSms ? wide : tokens * heads >= 2 * wave * 1200 ? 2 * wave / heads : wave / heads;
    want = std::min(want, (tokens + 255) / 256);
    a.out.S = (int)std::max(1LL, std::min(want, 1024LL));
    a.lse = lse;
    a.mass = mass;
    a.status = status;
    return launch(L, in, a, true, batch, st);
}

}  // namespace oscar
