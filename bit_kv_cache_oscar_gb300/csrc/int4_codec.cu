// BF16 rows to 4 bits (demotion without a rotation) and back (promotion), over position ranges.
//
// Per group of g channels: lo = c·min, hi = c·max, zero = bf16(lo), scale = bf16((hi - lo)/15), code =
// nearest integer to (x - zero)/scale (ties to even) clamped to 0..15; value = zero + code·scale.
//
// Bound by HBM in both directions (648 bytes per token and kv head at g = 128).  A half-warp takes one
// row: 8 channels a lane, one 16-byte access each for the key and the value, one 32-bit word of codes a
// lane; key and value go together because they share the scale/zero record.  A CTA takes one kv head and
// 16-token tiles of the range at absolute positions 16 i (inside one page: two table entries a tile, no
// division by the number of heads), so a tile's codes are 1 KB in a row; it loads a tile ahead.  The
// number of CTAs does not depend on the ranges, which are device data: one token a step and a whole
// prompt are the same launch.

#include <cuda_bf16.h>

#include "int4.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 256;

struct RangeArgs {
    Bf16PoolView bf;
    Int4PoolView i4;
    const int32_t *bpt, *ipt;
    int max_pages, page_size, n_kv;
    const int32_t *begin, *end;
    float cK, cV;
    int32_t *status;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t *>(&v); }

// The lane's 8 channels of a row -> its word of codes; *sz gets scale | zero << 16.
// The code is first rounded from u = (x - zero)·(1/(15 scale))·15 in fp32, off by at most 15·4·2^-24 <
// 4e-6; the saturating product is the clamp (and 0 for NaN).  Where u lies within 1e-4 of a border k + 1/2
// (one lane in a few hundred) the quotient is compared with it exactly: d = fl(x - zero) and its error e
// by a two-sum, (k + 1/2)·scale has 13 bits, d minus it is exact because they nearly cancel, and the sign
// of that plus e is the answer.  (Dividing in 64 bits there instead took 2.4 ms for a 100K prompt.)
template <int GROUP>
__device__ __forceinline__ uint32_t quantize8(uint4 w, float clip, uint32_t *sz) {
    const uint32_t p[4] = {w.x, w.y, w.z, w.w};
    // (min, -max) of the lane's values as one bf16 pair, then the least of both over the group's lanes
    const __nv_bfloat162 mn2 = __hmin2(__hmin2(as_bf2(w.x), as_bf2(w.y)), __hmin2(as_bf2(w.z), as_bf2(w.w)));
    const __nv_bfloat162 mx2 = __hmax2(__hmax2(as_bf2(w.x), as_bf2(w.y)), __hmax2(as_bf2(w.z), as_bf2(w.w)));
    __nv_bfloat162 r = __halves2bfloat162(__hmin(mn2.x, mn2.y), __hneg(__hmax(mx2.x, mx2.y)));
#pragma unroll
    for (int o = GROUP / 16; o; o >>= 1) r = __hmin2(r, as_bf2(__shfl_xor_sync(0xffffffffu, as_u32(r), o)));
    const float mn = __fadd_rn(lo16(as_u32(r)), 0.0f);                  // a signed zero is read as +0
    const float mx = __fadd_rn(-hi16(as_u32(r)), 0.0f);
    const float lo = __fmul_rn(clip, mn), hi = __fmul_rn(clip, mx);
    const uint16_t zb = f32_to_bf16_rn(lo), sb = f32_to_bf16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float z = bf16_to_f32(zb), s = bf16_to_f32(sb);
    *sz = (uint32_t)sb | ((uint32_t)zb << 16);
    if (s == 0.0f) return 0u;
    constexpr float kMagic = 12582912.0f;                               // 1.5·2^23: adding it rounds to an integer
    const float inv = __frcp_rn(s * 15.0f);
    uint32_t code = 0;
    float off = s < 1e-30f || s > 1e37f ? 1.0f : 0.0f;                  // 15 s or its inverse would leave fp32's range
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = e & 1 ? hi16(p[e >> 1]) : lo16(p[e >> 1]);
        const float u = __saturatef(__fmul_rn(__fsub_rn(x, z), inv));
        const float f = __fmaf_rn(u, 15.0f, kMagic);
        off = fmaxf(off, fabsf(__fmaf_rn(u, 15.0f, -__fsub_rn(f, kMagic))));
        code += (__float_as_uint(f) - 0x4B400000u) << (4 * e);
    }
    if (off > 0.4999f) {
        const float up = s < 1e-30f ? 0x1p64f : (s > 1e37f ? 0x1p-64f : 1.0f);
        const float zz = z * up, ss = s * up, iv = __frcp_rn(ss * 15.0f);
        code = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = (e & 1 ? hi16(p[e >> 1]) : lo16(p[e >> 1])) * up;
            const float d = __fsub_rn(x, zz), u = __saturatef(__fmul_rn(d, iv)) * 15.0f, k = floorf(u);
            float c = rintf(u);
            if (fabsf(u - k - 0.5f) < 1e-3f) {
                const float bb = __fsub_rn(d, x), err = __fadd_rn(__fsub_rn(x, __fsub_rn(d, bb)), __fsub_rn(-zz, bb));
                const float w = __fadd_rn(__fmaf_rn(-(k + 0.5f), ss, d), err);
                c = w > 0.0f ? k + 1.0f : (w < 0.0f ? k : 2.0f * rintf(0.5f * (k + 0.5f)));
            }
            code |= (uint32_t)c << (4 * e);
        }
    }
    return code;
}

__device__ __forceinline__ uint4 restore8(uint32_t code, uint32_t sz) {
    const float s = lo16(sz), z = hi16(sz);
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        // a code below 2^23 as the low bits of 2^23 + code
        const float a = __uint_as_float(0x4B000000u | ((code >> (8 * e)) & 15u)) - 8388608.0f;
        const float b = __uint_as_float(0x4B000000u | ((code >> (8 * e + 4)) & 15u)) - 8388608.0f;
        const __nv_bfloat162 v = __floats2bfloat162_rn(fmaf(a, s, z), fmaf(b, s, z));
        o[e] = as_u32(v);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The two pool slots of one (position, kv head): page ids checked, rows resolved.
struct Slot {
    bool on;
    size_t bf, i4;      // element offset of the lane's channels in the BF16 pool, row in the INT4 pool
};
__device__ __forceinline__ Slot find(const RangeArgs &a, int b, int h, int pos, int lo, int hi, int hl) {
    Slot s{false, 0, 0};
    if (pos < lo || pos >= hi) return s;
    const int pb = a.bpt[(size_t)b * a.max_pages + pos / a.page_size], p4 = a.ipt[(size_t)b * a.max_pages + pos / a.page_size];
    const bool okb = (uint32_t)pb < (uint32_t)a.bf.n_pages, ok4 = (uint32_t)p4 < (uint32_t)a.i4.n_pages;
    if (!(okb && ok4)) {
        if (hl == 0) flag_status(a.status, (okb ? 0 : OSCAR_DEV_BAD_BF16_PAGE) | (ok4 ? 0 : OSCAR_DEV_BAD_INT4_PAGE));
        return s;
    }
    const int slot = pos % a.page_size;
    s.on = true;
    s.bf = (((size_t)pb * a.page_size + slot) * a.n_kv + h) * kHeadDim + 8 * hl;
    s.i4 = row4(p4, a.n_kv, h, a.page_size, slot);
    return s;
}

// grid (X, Hkv, batch): CTA x takes tiles x, x + X, ... of its request's range for its kv head.
template <int GROUP, bool DEMOTE>
__global__ void __launch_bounds__(kThreads) codec4_kernel(RangeArgs a) {
    const int h = blockIdx.y, b = blockIdx.z, hl = threadIdx.x & 15, row = threadIdx.x >> 4;
    const int lo = a.begin[b], hi = a.end[b];
    if (lo < 0 || hi < lo || hi > a.max_pages * a.page_size) {
        if (threadIdx.x == 0 && blockIdx.x == 0) flag_status(a.status, OSCAR_DEV_BAD_LENGTH);
        return;
    }
    constexpr int G = kHeadDim / GROUP, LPG = GROUP / 8;        // groups a row, lanes a group
    const int step = gridDim.x * 16;
    const long long first = (lo & ~15) + (long long)blockIdx.x * 16;
    if (first >= hi) return;
    if constexpr (DEMOTE) {
        Slot s = find(a, b, h, (int)first + row, lo, hi, hl);
        uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
        if (s.on) {
            kx = *reinterpret_cast<const uint4 *>(a.bf.k + s.bf);
            vx = *reinterpret_cast<const uint4 *>(a.bf.v + s.bf);
        }
        for (long long p = first; p < hi; p += step) {
            const Slot cur = s;
            const uint4 k = kx, v = vx;
            s.on = false;
            if (p + step < hi) s = find(a, b, h, (int)(p + step) + row, lo, hi, hl);
            if (s.on) {
                kx = *reinterpret_cast<const uint4 *>(a.bf.k + s.bf);
                vx = *reinterpret_cast<const uint4 *>(a.bf.v + s.bf);
            }
            uint2 sz;
            const uint32_t kc = quantize8<GROUP>(k, a.cK, &sz.x), vc = quantize8<GROUP>(v, a.cV, &sz.y);
            if (cur.on) {
                reinterpret_cast<uint32_t *>(a.i4.codes_k + cur.i4 * kRow4)[hl] = kc;
                reinterpret_cast<uint32_t *>(a.i4.codes_v + cur.i4 * kRow4)[hl] = vc;
                if (hl % LPG == 0) reinterpret_cast<uint2 *>(a.i4.scale_zero)[cur.i4 * G + hl / LPG] = sz;
            }
        }
    } else {
        Slot s = find(a, b, h, (int)first + row, lo, hi, hl);
        uint32_t kc = 0, vc = 0;
        uint2 sz = make_uint2(0, 0);
        auto load = [&]() {
            kc = reinterpret_cast<const uint32_t *>(a.i4.codes_k + s.i4 * kRow4)[hl];
            vc = reinterpret_cast<const uint32_t *>(a.i4.codes_v + s.i4 * kRow4)[hl];
            sz = reinterpret_cast<const uint2 *>(a.i4.scale_zero)[s.i4 * G + hl / LPG];
        };
        if (s.on) load();
        for (long long p = first; p < hi; p += step) {
            const Slot cur = s;
            const uint32_t k = kc, v = vc;
            const uint2 z = sz;
            s.on = false;
            if (p + step < hi) s = find(a, b, h, (int)(p + step) + row, lo, hi, hl);
            if (s.on) load();
            if (cur.on) {
                *reinterpret_cast<uint4 *>(const_cast<uint16_t *>(a.bf.k) + cur.bf) = restore8(k, z.x);
                *reinterpret_cast<uint4 *>(const_cast<uint16_t *>(a.bf.v) + cur.bf) = restore8(v, z.y);
            }
        }
    }
}

template <bool DEMOTE>
cudaError_t launch(const oscar_layout_t &L, const RangeArgs &a, int batch, cudaStream_t st) {
    // about eight CTAs an SM over all (head, request) pairs, no more than the longest possible range has tiles
    const long long most = ((long long)a.max_pages * L.page_size + 15) / 16, pairs = (long long)batch * L.n_kv_heads;
    const long long want = (8 * 152 + pairs - 1) / pairs;
    const dim3 grid((unsigned)(want < most ? want : most), L.n_kv_heads, batch);
    switch (L.group) {
        case 32: codec4_kernel<32, DEMOTE><<<grid, kThreads, 0, st>>>(a); break;
        case 64: codec4_kernel<64, DEMOTE><<<grid, kThreads, 0, st>>>(a); break;
        default: codec4_kernel<128, DEMOTE><<<grid, kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_demote4(const oscar_layout_t &L, Bf16PoolView src, const int32_t *bpt, Int4PoolView dst,
                           const int32_t *ipt, int max_pages, int batch, const int32_t *begin, const int32_t *end,
                           float cK, float cV, int32_t *status, cudaStream_t st) {
    return launch<true>(L, {src, dst, bpt, ipt, max_pages, L.page_size, L.n_kv_heads, begin, end, cK, cV, status}, batch, st);
}

cudaError_t launch_promote4(const oscar_layout_t &L, Int4PoolView src, const int32_t *ipt, Bf16PoolView dst,
                            const int32_t *bpt, int max_pages, int batch, const int32_t *begin, const int32_t *end,
                            int32_t *status, cudaStream_t st) {
    return launch<false>(L, {dst, src, bpt, ipt, max_pages, L.page_size, L.n_kv_heads, begin, end, 1.f, 1.f, status}, batch, st);
}

}  // namespace oscar
