// BF16 rows to 4 bits (demotion without a rotation) and back (promotion), over position ranges.
//
// Per group of g channels: lo = c·min, hi = c·max, zero = bf16(lo), scale = bf16((hi - lo)/15), code =
// nearest integer to (x - zero)/scale (ties to even) clamped to 0..15; value = zero + code·scale.
//
// Bound by HBM in both directions (648 bytes per token and kv head at g = 128), and by the issue rate next
// to it: a half-warp takes one (token, kv head), eight lanes its key and eight its value with 16 channels
// each, so that what is done once a row (the range, scale and zero) is shared by 16 values, and the
// quantizer's steps run on packed fp32 pairs.  A CTA takes one kv head and 16-token tiles of the range at
// absolute positions 16 i (inside one page, so no division by the number of heads; a tile's codes are
// 1 KB in a row) and loads a tile ahead.  The number of CTAs does not depend on the ranges, which are
// device data: one token a step and a whole prompt are the same launch.  Measured, 100K tokens of 8 kv
// heads at g = 128: demotion 144 us = 3.6 TB/s (the ALU pipe: 310 instructions a warp and two rows),
// promotion 85 us = 6.1 TB/s.

#include <cuda_bf16.h>

#include "int4.cuh"
#include "ptx.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 256;

struct RangeArgs {
    Bf16PoolView bf;
    Int4PoolView i4;
    const int32_t *bpt, *ipt;
    int max_pages, page_shift, n_kv;
    const int32_t *begin, *end;
    float cK, cV;
    int32_t *status;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t *>(&v); }

// packed fp32 pairs
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// The lane's 16 channels (8 words of bf16 pairs) -> its two words of codes; *sz gets scale | zero << 16.
// bf16 values hit the border between two codes exactly about once in 300, so the border is decided exactly
// for every value: with u = (x - zero)/scale approximately (error below 1e-5), k = rint(u - 1/2) in 0..14
// (the saturating product is the clamp, and 0 for NaN) is the code or one below it whatever the error, and
// d - k·scale, which is exact, against scale/2 tells which: above it k + 1, below it k, on it the even one
// (its last bit is set where k is odd, which only then lifts it above scale/2).  d = x - zero is exact in
// fp32 unless one of the two is below 2^-15 of the other.  A zero that small shows in the group's range.  A
// value x that small lies within 2^-10 codes of -zero/scale, so it matters only where that is that near a
// border, which one group in 200 is.  Such groups add the error of d, by a two-sum, to the comparison.
template <int GROUP>
__device__ __forceinline__ uint2 quantize16(const uint32_t (&w)[8], float clip, uint32_t *sz) {
    // (min, -max) of the lane's values as one bf16 pair, then the least of both over the group's lanes
    __nv_bfloat162 mn2 = as_bf2(w[0]), mx2 = as_bf2(w[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        mn2 = __hmin2(mn2, as_bf2(w[i]));
        mx2 = __hmax2(mx2, as_bf2(w[i]));
    }
    __nv_bfloat162 r = __halves2bfloat162(__hmin(mn2.x, mn2.y), __hneg(__hmax(mx2.x, mx2.y)));
#pragma unroll
    for (int o = GROUP / 32; o; o >>= 1) r = __hmin2(r, as_bf2(__shfl_xor_sync(0xffffffffu, as_u32(r), o)));
    const float mn = __fadd_rn(lo16(as_u32(r)), 0.0f);                  // a signed zero is read as +0
    const float mx = __fadd_rn(-hi16(as_u32(r)), 0.0f);
    const float lo = __fmul_rn(clip, mn), hi = __fmul_rn(clip, mx);
    const uint16_t zb = f32_to_bf16_rn(lo), sb = f32_to_bf16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float z = bf16_to_f32(zb), s = bf16_to_f32(sb);
    *sz = (uint32_t)sb | ((uint32_t)zb << 16);
    if (s == 0.0f) return make_uint2(0u, 0u);
    // the arithmetic below leaves fp32's range for ranges near its ends: those are moved by 2^64
    const float up = s < 1e-30f ? 0x1p64f : (s > 1e36f ? 0x1p-64f : 1.0f);
    const float top = fmaxf(fabsf(mn), fabsf(mx)), az = fabsf(z);
    const float ss = s * up, iv = __fdividef(1.0f, ss * 14.0f), at0 = -z * up * (iv * 14.0f);     // the code position of x = 0
    const bool near0 = fabsf(at0 - floorf(at0) - 0.5f) < 0x1p-9f;
    uint32_t code[2] = {0u, 0u};
    if (up != 1.0f || near0 || (az < top * 0x1p-15f && az > 0.0f)) {
        const float zz = z * up;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float x = (e & 1 ? hi16(w[e >> 1]) : lo16(w[e >> 1])) * up;
            const float d = __fsub_rn(x, zz), bb = __fsub_rn(d, x);
            const float err = __fadd_rn(__fsub_rn(x, __fsub_rn(d, bb)), __fsub_rn(-zz, bb));
            const float k = rintf(__saturatef(__fmaf_rn(d, iv, -1.0f / 28.0f)) * 14.0f);
            const float t = __fadd_rn(__fmaf_rn(-(k + 0.5f), ss, d), err);
            const float c = t > 0.0f ? k + 1.0f : (t < 0.0f ? k : 2.0f * rintf(0.5f * (k + 0.5f)));
            code[e >> 3] |= (uint32_t)c << (4 * (e & 7));
        }
        return make_uint2(code[0], code[1]);
    }
    constexpr float kMagic = 12582912.0f;                               // 1.5·2^23: adding it rounds to an integer
    const float inv = iv, half = 0.5f * s;
    const uint64_t nz = pair(-z, -z), ns = pair(-s, -s), f14 = pair(14.0f, 14.0f), magic = pair(kMagic, kMagic),
                   down = pair(-kMagic, -kMagic);
#pragma unroll
    for (int i = 7; i >= 0; --i) {
        const uint64_t d = add2(pair(lo16(w[i]), hi16(w[i])), nz);
        float a, b, r0, r1, k0, k1;
        unpair(d, a, b);
        const uint64_t f = fma2(pair(__saturatef(__fmaf_rn(a, inv, -1.0f / 28.0f)), __saturatef(__fmaf_rn(b, inv, -1.0f / 28.0f))), f14,
                                magic);                                 // kMagic + k: k in the low bits
        unpair(fma2(add2(f, down), ns, d), r0, r1);                     // d - k·scale
        unpair(f, k0, k1);
        const uint32_t f0 = __float_as_uint(k0), f1 = __float_as_uint(k1);
        uint32_t &c = code[i >> 2];
        c = (c << 4) + f1 + (__uint_as_float(__float_as_uint(r1) | (f1 & 1u)) > half ? 1u : 0u);
        c = (c << 4) + f0 + (__uint_as_float(__float_as_uint(r0) | (f0 & 1u)) > half ? 1u : 0u);
    }
    // each term carried the bits of kMagic, 0x4B400000, eight times over: their sum shifted as the codes are
    constexpr uint32_t kSum = 0x4B400000u * 0x11111111u;
    code[0] -= kSum;
    code[1] -= kSum;
    return make_uint2(code[0], code[1]);
}

// Eight codes -> four words of bf16 pairs, zero + code·scale in one bf16 fused multiply-add (rounded once).
// A nibble below bits of value 128 in bf16 (0x4300) is 128 + code exactly; codes 4 channels apart share a
// word, so the results are put back in channel order.
__device__ __forceinline__ uint4 restore8(uint32_t code, uint32_t sz) {
    const __nv_bfloat162 s = as_bf2(__byte_perm(sz, 0, 0x1010)), z = as_bf2(__byte_perm(sz, 0, 0x3232));
    const __nv_bfloat162 off = as_bf2(0x43004300u);
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = as_u32(__hfma2(__hsub2(as_bf2(((code >> (4 * e)) & 0x000F000Fu) | 0x43004300u), off), s, z));
    return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                      __byte_perm(v[2], v[3], 0x7632));
}

// A row's two places: checked page ids, row indexes in both pools (the INT4 pool's is below 2^31).
struct Slot {
    bool on;
    long long bf;
    int i4;
};
__device__ __forceinline__ Slot find(const RangeArgs &a, size_t pt0, int h, int pos, int lo, int hi) {
    Slot s{false, 0, 0};
    if (pos < lo || pos >= hi) return s;
    const int pb = a.bpt[pt0 + (pos >> a.page_shift)], p4 = a.ipt[pt0 + (pos >> a.page_shift)];
    const bool okb = (uint32_t)pb < (uint32_t)a.bf.n_pages, ok4 = (uint32_t)p4 < (uint32_t)a.i4.n_pages;
    if (!(okb && ok4)) {
        if ((threadIdx.x & 15) == 0) flag_status(a.status, (okb ? 0 : OSCAR_DEV_BAD_BF16_PAGE) | (ok4 ? 0 : OSCAR_DEV_BAD_INT4_PAGE));
        return s;
    }
    const int slot = pos & ((1 << a.page_shift) - 1);
    s.on = true;
    s.bf = (((long long)pb << a.page_shift) + slot) * a.n_kv + h;
    s.i4 = ((p4 * a.n_kv + h) << a.page_shift) + slot;
    return s;
}

// grid (X, Hkv, batch): CTA x takes tiles x, x + X, ... of its request's range for its kv head.
template <int GROUP, bool DEMOTE>
__global__ void __launch_bounds__(kThreads) codec4_kernel(RangeArgs a) {
    const int h = blockIdx.y, b = blockIdx.z, hl = threadIdx.x & 7, row = threadIdx.x >> 4;
    const bool value = threadIdx.x & 8;
    pdl_wait();
    const int lo = a.begin[b], hi = a.end[b];
    if (lo < 0 || hi < lo || (long long)hi > ((long long)a.max_pages << a.page_shift)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) flag_status(a.status, OSCAR_DEV_BAD_LENGTH);
        return;
    }
    constexpr int G = kHeadDim / GROUP;                          // groups a row
    const int step = gridDim.x * 16;
    const long long first = (lo & ~15) + (long long)blockIdx.x * 16;
    if (first >= hi) return;
    const size_t pt0 = (size_t)b * a.max_pages;
    uint4 *rows = reinterpret_cast<uint4 *>(const_cast<uint16_t *>(value ? a.bf.v : a.bf.k));               // 16 uint4 a row
    uint32_t *codes = reinterpret_cast<uint32_t *>(value ? a.i4.codes_v : a.i4.codes_k);                    // 16 words a row
    uint32_t *recs = reinterpret_cast<uint32_t *>(a.i4.scale_zero) + value;                                 // 2 G words a row
    Slot s = find(a, pt0, h, (int)first + row, lo, hi);
    if constexpr (DEMOTE) {
        // chunks of 8 channels: a lane's two in one group.  One group a row: hl and hl + 8, so that eight
        // lanes read 128 bytes in a row; smaller groups: two neighbours.
        const int c0 = G == 1 ? hl : 2 * hl, c1 = G == 1 ? hl + 8 : 2 * hl + 1;
        const float clip = value ? a.cV : a.cK;
        uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
        if (s.on) {
            x0 = rows[s.bf * 16 + c0];
            x1 = rows[s.bf * 16 + c1];
        }
        for (long long p = first; p < hi; p += step) {
            const Slot cur = s;
            const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            s.on = false;
            if (p + step < hi) s = find(a, pt0, h, (int)(p + step) + row, lo, hi);
            if (s.on) {
                x0 = rows[s.bf * 16 + c0];
                x1 = rows[s.bf * 16 + c1];
            }
            uint32_t sz;
            const uint2 c = quantize16<GROUP>(w, clip, &sz);
            if (cur.on) {
                uint32_t *to = codes + (size_t)cur.i4 * 16;
                if (G == 1) {
                    to[c0] = c.x;
                    to[c1] = c.y;
                } else {
                    *reinterpret_cast<uint2 *>(to + c0) = c;
                }
                if (hl % (GROUP / 16) == 0) recs[(size_t)cur.i4 * 2 * G + 2 * (hl / (GROUP / 16))] = sz;
            }
        }
    } else {
        // chunks hl and hl + 8 whatever the group: eight lanes write 128 bytes in a row
        uint32_t c0 = 0, c1 = 0, z0 = 0, z1 = 0;
        auto fetch = [&]() {
            const uint32_t *from = codes + (size_t)s.i4 * 16, *rec = recs + (size_t)s.i4 * 2 * G;
            c0 = from[hl];
            c1 = from[hl + 8];
            z0 = rec[2 * (8 * hl / GROUP)];
            z1 = G == 1 ? z0 : rec[2 * ((64 + 8 * hl) / GROUP)];
        };
        if (s.on) fetch();
        for (long long p = first; p < hi; p += step) {
            const Slot cur = s;
            const uint32_t k0 = c0, k1 = c1, y0 = z0, y1 = z1;
            s.on = false;
            if (p + step < hi) s = find(a, pt0, h, (int)(p + step) + row, lo, hi);
            if (s.on) fetch();
            if (cur.on) {
                rows[cur.bf * 16 + hl] = restore8(k0, y0);
                rows[cur.bf * 16 + hl + 8] = restore8(k1, y1);
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
        case 32: return launch_ahead(codec4_kernel<32, DEMOTE>, grid, kThreads, 0, st, a);
        case 64: return launch_ahead(codec4_kernel<64, DEMOTE>, grid, kThreads, 0, st, a);
        default: return launch_ahead(codec4_kernel<128, DEMOTE>, grid, kThreads, 0, st, a);
    }
}

}  // namespace

cudaError_t launch_demote4(const oscar_layout_t &L, Bf16PoolView src, const int32_t *bpt, Int4PoolView dst,
                           const int32_t *ipt, int max_pages, int batch, const int32_t *begin, const int32_t *end,
                           float cK, float cV, int32_t *status, cudaStream_t st) {
    return launch<true>(L, {src, dst, bpt, ipt, max_pages, page_shift(L), L.n_kv_heads, begin, end, cK, cV, status}, batch, st);
}

cudaError_t launch_promote4(const oscar_layout_t &L, Int4PoolView src, const int32_t *ipt, Bf16PoolView dst,
                            const int32_t *bpt, int max_pages, int batch, const int32_t *begin, const int32_t *end,
                            int32_t *status, cudaStream_t st) {
    return launch<false>(L, {dst, src, bpt, ipt, max_pages, page_shift(L), L.n_kv_heads, begin, end, 1.f, 1.f, status}, batch, st);
}

}  // namespace oscar
