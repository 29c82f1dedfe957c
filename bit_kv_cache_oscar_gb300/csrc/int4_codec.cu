// BF16 rows to 4 bits (demotion without a rotation) and back (promotion), over position ranges.
//
// Per group of g channels: lo = c·min, hi = c·max, zero = bf16(lo), scale = bf16((hi - lo)/15), code =
// nearest integer to (x - zero)/scale (ties to even) clamped to 0..15; value = zero + code·scale.
//
// Sixteen lanes take one (token, kv head): 8 channels of its key and of its value each (two 16-byte
// loads), so a row's codes are one 32-bit word a lane and key and value meet for the shared scale/zero
// record.  The grid is a fixed number of CTAs per request that stride over its range, because the
// ranges are device data: one token a step and a whole prompt are the same launch.

#include "int4.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerCta = kThreads / 16;

struct RangeArgs {
    Bf16PoolView bf;
    Int4PoolView i4;
    const int32_t *bpt, *ipt;
    int max_pages, page_size, n_kv;
    const int32_t *begin, *end;
    float cK, cV;
    int32_t *status;
};

// One row part of 8 channels -> the lane's word of codes; *sz gets scale | zero << 16.
template <int GROUP>
__device__ __forceinline__ uint32_t quantize8(uint4 w, float clip, uint32_t *sz) {
    float x[8];
    const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(p[e] << 16);
        x[2 * e + 1] = __uint_as_float(p[e] & 0xffff0000u);
    }
    float mn = x[0], mx = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        mn = fminf(mn, x[e]);
        mx = fmaxf(mx, x[e]);
    }
#pragma unroll
    for (int o = GROUP / 16; o; o >>= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    mn = __fadd_rn(mn, 0.0f);                       // a signed zero is read as +0
    mx = __fadd_rn(mx, 0.0f);
    const float lo = __fmul_rn(clip, mn), hi = __fmul_rn(clip, mx);
    const uint16_t zb = f32_to_bf16_rn(lo), sb = f32_to_bf16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float z = bf16_to_f32(zb), s = bf16_to_f32(sb);
    *sz = (uint32_t)sb | ((uint32_t)zb << 16);
    uint32_t code = 0;
    if (s != 0.0f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double r = rint(((double)x[e] - (double)z) / (double)s);
            code |= (uint32_t)(r >= 15.0 ? 15 : (r >= 0.0 ? (int)r : 0)) << (4 * e);
        }
    }
    return code;
}

// The range of request b: false when there is nothing to do; flags a bad one.
__device__ __forceinline__ bool read_range(const RangeArgs &a, int b, int &lo, int &n) {
    lo = a.begin[b];
    const int hi = a.end[b];
    if (lo < 0 || hi < lo || hi > a.max_pages * a.page_size) {
        if (threadIdx.x == 0 && blockIdx.x == 0) flag_status(a.status, OSCAR_DEV_BAD_LENGTH);
        return false;
    }
    n = hi - lo;
    return n > 0;
}

template <int GROUP>
__global__ void __launch_bounds__(kThreads) demote4_kernel(RangeArgs a) {
    const int b = blockIdx.y, hl = threadIdx.x & 15;
    int lo, n;
    if (!read_range(a, b, lo, n)) return;
    const long long items = (long long)n * a.n_kv;
    // whole warps stay in the loop: the two halves of a warp shuffle together
    for (long long w = (long long)blockIdx.x * kRowsPerCta; w < items; w += (long long)gridDim.x * kRowsPerCta) {
        const long long e = w + (threadIdx.x >> 4);
        const bool in = e < items;
        const int pos = lo + (int)((in ? e : 0) / a.n_kv), h = (int)((in ? e : 0) % a.n_kv);
        const int src = a.bpt[(size_t)b * a.max_pages + pos / a.page_size];
        const int dst = a.ipt[(size_t)b * a.max_pages + pos / a.page_size];
        const bool src_ok = src >= 0 && src < a.bf.n_pages, dst_ok = dst >= 0 && dst < a.i4.n_pages;
        if (hl == 0 && !src_ok) flag_status(a.status, OSCAR_DEV_BAD_BF16_PAGE);
        if (hl == 0 && !dst_ok) flag_status(a.status, OSCAR_DEV_BAD_INT4_PAGE);
        const bool on = in && src_ok && dst_ok;
        const size_t from = (((size_t)(on ? src : 0) * a.page_size + pos % a.page_size) * a.n_kv + h) * kHeadDim + 8 * hl;
        const uint4 kx = on ? *reinterpret_cast<const uint4 *>(a.bf.k + from) : make_uint4(0, 0, 0, 0);
        const uint4 vx = on ? *reinterpret_cast<const uint4 *>(a.bf.v + from) : make_uint4(0, 0, 0, 0);
        uint2 sz;
        const uint32_t kc = quantize8<GROUP>(kx, a.cK, &sz.x), vc = quantize8<GROUP>(vx, a.cV, &sz.y);
        if (on) {
            const size_t row = row4(dst, a.n_kv, h, a.page_size, pos % a.page_size);
            reinterpret_cast<uint32_t *>(a.i4.codes_k + row * kRow4)[hl] = kc;
            reinterpret_cast<uint32_t *>(a.i4.codes_v + row * kRow4)[hl] = vc;
            constexpr int LPG = GROUP / 8;          // lanes per group
            if (hl % LPG == 0) reinterpret_cast<uint2 *>(a.i4.scale_zero)[row * (kHeadDim / GROUP) + hl / LPG] = sz;
        }
    }
}

__device__ __forceinline__ uint4 restore8(uint32_t code, uint32_t sz) {
    const float s = __uint_as_float(sz << 16), z = __uint_as_float(sz & 0xffff0000u);
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float lo = fmaf((float)((code >> (8 * e)) & 15u), s, z), hi = fmaf((float)((code >> (8 * e + 4)) & 15u), s, z);
        o[e] = (uint32_t)f32_to_bf16_rn(lo) | ((uint32_t)f32_to_bf16_rn(hi) << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int GROUP>
__global__ void __launch_bounds__(kThreads) promote4_kernel(RangeArgs a) {
    const int b = blockIdx.y, hl = threadIdx.x & 15;
    int lo, n;
    if (!read_range(a, b, lo, n)) return;
    const long long items = (long long)n * a.n_kv;
    for (long long e = (long long)blockIdx.x * kRowsPerCta + (threadIdx.x >> 4); e < items;
         e += (long long)gridDim.x * kRowsPerCta) {
        const int pos = lo + (int)(e / a.n_kv), h = (int)(e % a.n_kv);
        const int src = a.ipt[(size_t)b * a.max_pages + pos / a.page_size];
        const int dst = a.bpt[(size_t)b * a.max_pages + pos / a.page_size];
        const bool src_ok = src >= 0 && src < a.i4.n_pages, dst_ok = dst >= 0 && dst < a.bf.n_pages;
        if (!src_ok || !dst_ok) {
            if (hl == 0) flag_status(a.status, (src_ok ? 0 : OSCAR_DEV_BAD_INT4_PAGE) | (dst_ok ? 0 : OSCAR_DEV_BAD_BF16_PAGE));
            continue;
        }
        const size_t row = row4(src, a.n_kv, h, a.page_size, pos % a.page_size);
        const uint32_t kc = reinterpret_cast<const uint32_t *>(a.i4.codes_k + row * kRow4)[hl];
        const uint32_t vc = reinterpret_cast<const uint32_t *>(a.i4.codes_v + row * kRow4)[hl];
        const uint2 sz = reinterpret_cast<const uint2 *>(a.i4.scale_zero)[row * (kHeadDim / GROUP) + hl / (GROUP / 8)];
        const size_t to = (((size_t)dst * a.page_size + pos % a.page_size) * a.n_kv + h) * kHeadDim + 8 * hl;
        *reinterpret_cast<uint4 *>(const_cast<uint16_t *>(a.bf.k) + to) = restore8(kc, sz.x);
        *reinterpret_cast<uint4 *>(const_cast<uint16_t *>(a.bf.v) + to) = restore8(vc, sz.y);
    }
}

// CTAs per request: together about eight a SM, no more than the longest possible range has rows for.
dim3 range_grid(const oscar_layout_t &L, int max_pages, int batch) {
    const long long most = ((long long)max_pages * L.page_size * L.n_kv_heads + kRowsPerCta - 1) / kRowsPerCta;
    const long long want = (8 * 152 + batch - 1) / batch;
    return dim3((unsigned)(want < most ? want : most), batch);
}

}  // namespace

cudaError_t launch_demote4(const oscar_layout_t &L, Bf16PoolView src, const int32_t *bpt, Int4PoolView dst,
                           const int32_t *ipt, int max_pages, int batch, const int32_t *begin, const int32_t *end,
                           float cK, float cV, int32_t *status, cudaStream_t st) {
    const RangeArgs a{src, dst, bpt, ipt, max_pages, L.page_size, L.n_kv_heads, begin, end, cK, cV, status};
    const dim3 grid = range_grid(L, max_pages, batch);
    switch (L.group) {
        case 32: demote4_kernel<32><<<grid, kThreads, 0, st>>>(a); break;
        case 64: demote4_kernel<64><<<grid, kThreads, 0, st>>>(a); break;
        default: demote4_kernel<128><<<grid, kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_promote4(const oscar_layout_t &L, Int4PoolView src, const int32_t *ipt, Bf16PoolView dst,
                            const int32_t *bpt, int max_pages, int batch, const int32_t *begin, const int32_t *end,
                            int32_t *status, cudaStream_t st) {
    const RangeArgs a{dst, src, bpt, ipt, max_pages, L.page_size, L.n_kv_heads, begin, end, 1.f, 1.f, status};
    const dim3 grid = range_grid(L, max_pages, batch);
    switch (L.group) {
        case 32: promote4_kernel<32><<<grid, kThreads, 0, st>>>(a); break;
        case 64: promote4_kernel<64><<<grid, kThreads, 0, st>>>(a); break;
        default: promote4_kernel<128><<<grid, kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace oscar
