// BF16 rows to 4 bits (demotion without a rotation) and back (promotion), over position ranges.
//
// Per group of g channels: lo = c·min, hi = c·max, zero = bf16(lo), scale = bf16((hi - lo)/15), code =
// nearest integer to (x - zero)/scale (ties to even) clamped to 0..15; value = zero + code·scale.
//
// Bound by HBM in both directions (648 bytes per token and kv head at g = 128), and demotion by the issue rate
// next to it.  A half-warp takes one (token, kv head), eight lanes its key and eight its value with 16
// channels each; a warp two tokens a step.  Demotion takes runs of four steps: a group's range is known to
// all its lanes, and each forms the record (scale, zero, reciprocal) of one step only, which then goes
// round by shuffles; page ids are checked once a run, whose 8 tokens lie in one page; the quantizer's steps
// run on packed fp32 pairs; the next run's lines are asked into L2 meanwhile.  Promotion takes 16-token tiles
// a CTA and loads a tile ahead.  A CTA has one kv head, so there is no division by the number of heads, and
// the number of CTAs, as many as fit at once, does not depend on the ranges, which are device data: one token a
// step and a whole prompt are the same launch.  Measured, 100K tokens of 8 kv heads at g = 128: demotion
// 102 us = 5.1 TB/s (216 instructions a step; 144 us with every record formed by all lanes; 110 without the
// prefetch; 107 with three CTAs of 80 registers an SM, 104 with runs of eight steps), promotion 85 us = 6.1 TB/s.

#include <cuda_bf16.h>

#include <algorithm>

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

// (min, -max) of the group that the lane's 16 channels (8 words of bf16 pairs) belong to, as a bf16 pair.
template <int GROUP>
__device__ __forceinline__ uint32_t range16(const uint32_t (&w)[8]) {
    __nv_bfloat162 mn2 = as_bf2(w[0]), mx2 = as_bf2(w[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        mn2 = __hmin2(mn2, as_bf2(w[i]));
        mx2 = __hmax2(mx2, as_bf2(w[i]));
    }
    __nv_bfloat162 r = __halves2bfloat162(__hmin(mn2.x, mn2.y), __hneg(__hmax(mx2.x, mx2.y)));
#pragma unroll
    for (int o = GROUP / 32; o; o >>= 1) r = __hmin2(r, as_bf2(__shfl_xor_sync(0xffffffffu, as_u32(r), o)));
    return as_u32(r);
}

// A group's record, scale | zero << 16, and 1/(14 scale), which is below 0 where codes16 does not do.
//
// bf16 values hit the border between two codes exactly about once in 300, so the border is decided exactly
// for every value: with u = (x - zero)/scale approximately (error below 1e-5), k = rint(u - 1/2) in 0..14
// (the saturating product is the clamp, and 0 for NaN) is the code or one below it whatever the error, and
// d - k·scale, which is exact, against scale/2 tells which: above it k + 1, below it k, on it the even one
// (its last bit is set where k is odd, which only then lifts it above scale/2).  d = x - zero is exact in
// fp32 unless one of the two is below 2^-15 of the other.  A zero that small shows in the group's range.  A
// value x that small lies within 2^-10 codes of -zero/scale, so it matters only where that is that near a
// border, which one group in 200 is.  Such groups add the error of d, by a two-sum, to the comparison; so
// do ranges near fp32's ends.
__device__ __forceinline__ float record(uint32_t r, float clip, uint32_t *sz) {
    const float mn = __fadd_rn(lo16(r), 0.0f);                          // a signed zero is read as +0
    const float mx = __fadd_rn(-hi16(r), 0.0f);
    const float lo = __fmul_rn(clip, mn), hi = __fmul_rn(clip, mx);
    const uint16_t zb = f32_to_bf16_rn(lo), sb = f32_to_bf16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float z = bf16_to_f32(zb), s = bf16_to_f32(sb);
    *sz = (uint32_t)sb | ((uint32_t)zb << 16);
    if (s < 1e-30f || s > 1e36f) return -1.0f;
    const float top = fmaxf(fabsf(mn), fabsf(mx)), az = fabsf(z);
    const float iv = __fdividef(1.0f, s * 14.0f), at0 = -z * (iv * 14.0f);                 // the code position of x = 0
    const bool near0 = fabsf(at0 - floorf(at0) - 0.5f) < 0x1p-9f;
    return near0 || (az < top * 0x1p-15f && az > 0.0f) ? -1.0f : iv;
}

// The lane's 16 channels -> its two words of codes, for ordinary groups.
__device__ __forceinline__ uint2 codes16(const uint32_t (&w)[8], uint32_t sz, float inv) {
    constexpr float kMagic = 12582912.0f;                               // 1.5·2^23: adding it rounds to an integer
    const float s = lo16(sz), z = hi16(sz), half = 0.5f * s;
    const uint64_t nz = pair(-z, -z), ns = pair(-s, -s), f14 = pair(14.0f, 14.0f), magic = pair(kMagic, kMagic),
                   down = pair(-kMagic, -kMagic);
    // the codes are put together as integers in fp32: two channels of a word's four, then both pairs
    const uint64_t f256 = pair(256.0f, 256.0f);
    uint32_t code[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float v[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint64_t k2[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t x = w[4 * q + 2 * m + e];
                const uint64_t d = add2(pair(lo16(x), hi16(x)), nz);
                float a, b, r0, r1, f0, f1, k0, k1;
                unpair(d, a, b);
                const uint64_t f = fma2(pair(__saturatef(__fmaf_rn(a, inv, -1.0f / 28.0f)), __saturatef(__fmaf_rn(b, inv, -1.0f / 28.0f))),
                                        f14, magic);                    // kMagic + k: k in the low bits
                const uint64_t k = add2(f, down);
                unpair(fma2(k, ns, d), r0, r1);                         // d - k·scale
                unpair(f, f0, f1);
                unpair(k, k0, k1);
                if (__uint_as_float(__float_as_uint(r0) | (__float_as_uint(f0) & 1u)) > half) k0 += 1.0f;
                if (__uint_as_float(__float_as_uint(r1) | (__float_as_uint(f1) & 1u)) > half) k1 += 1.0f;
                k2[e] = pair(k0, k1);
            }
            float even, odd;
            unpair(fma2(k2[1], f256, k2[0]), even, odd);
            v[m] = __fmaf_rn(odd, 16.0f, even) + 0x1p23f;
        }
        code[q] = __byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x5410);
    }
    return make_uint2(code[0], code[1]);
}

// The same for every group: with the error of d, ranges near fp32's ends moved by 2^64.
__device__ __forceinline__ uint2 codes16_any(const uint32_t (&w)[8], uint32_t sz) {
    const float s = lo16(sz), z = hi16(sz);
    if (s == 0.0f) return make_uint2(0u, 0u);
    const float up = s < 1e-30f ? 0x1p64f : (s > 1e36f ? 0x1p-64f : 1.0f);
    const float ss = s * up, iv = __fdividef(1.0f, ss * 14.0f), zz = z * up;
    uint32_t code[2] = {0u, 0u};
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

// A position's two places for a kv head: checked page ids, row indexes in both pools (the INT4 pool's is below 2^31).
struct Slot {
    bool on;
    long long bf;
    int i4;
};
__device__ __forceinline__ Slot find(const RangeArgs &a, size_t pt0, int h, int pos, int lanes) {
    Slot s{false, 0, 0};
    const int pb = a.bpt[pt0 + (pos >> a.page_shift)], p4 = a.ipt[pt0 + (pos >> a.page_shift)];
    const bool okb = (uint32_t)pb < (uint32_t)a.bf.n_pages, ok4 = (uint32_t)p4 < (uint32_t)a.i4.n_pages;
    if (!(okb && ok4)) {
        if ((threadIdx.x & (lanes - 1)) == 0)
            flag_status(a.status, (okb ? 0 : OSCAR_DEV_BAD_BF16_PAGE) | (ok4 ? 0 : OSCAR_DEV_BAD_INT4_PAGE));
        return s;
    }
    const int slot = pos & ((1 << a.page_shift) - 1);
    s.on = true;
    s.bf = (((long long)pb << a.page_shift) + slot) * a.n_kv + h;
    s.i4 = ((p4 * a.n_kv + h) << a.page_shift) + slot;
    return s;
}

// The request's range, false if there is nothing to do.
__device__ __forceinline__ bool read_range(const RangeArgs &a, int b, int &lo, int &hi) {
    lo = a.begin[b], hi = a.end[b];
    const bool bad = lo < 0 || hi < lo || (long long)hi > ((long long)a.max_pages << a.page_shift);
    if (bad && threadIdx.x == 0 && blockIdx.x == 0) flag_status(a.status, OSCAR_DEV_BAD_LENGTH);
    return !bad && lo < hi;
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A warp's share of [lo, hi) of one request and kv head: runs of 2 STEPS positions (at 2 STEPS i: inside a
// page), two positions a step.  A run's rows are all read, being in the pool whether in the range or not.
template <int GROUP, int STEPS>
__device__ __forceinline__ void demote_range(const RangeArgs &a, int lo, int hi) {
    const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31, hl = lane & 7, tok = lane >> 4;
    const bool value = lane & 8;
    constexpr int G = kHeadDim / GROUP, kLanes = GROUP / 16;     // groups a row, lanes a group
    constexpr int kOwn = kLanes < STEPS ? kLanes : STEPS;        // of which the first kOwn form records: of steps own, own + kOwn, ...
    const int own = hl & (kOwn - 1);
    const int stride = gridDim.x * (kThreads / 32) * 2 * STEPS;
    long long p = (lo & ~(2 * STEPS - 1)) + ((long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * 2 * STEPS;
    if (p >= hi) return;
    const size_t pt0 = (size_t)b * a.max_pages;
    // chunks of 8 channels: a lane's two in one group.  One group a row: hl and hl + 8, so that eight
    // lanes read 128 bytes in a row; smaller groups: two neighbours.
    const int c0 = G == 1 ? hl : 2 * hl, c1 = G == 1 ? hl + 8 : 2 * hl + 1;
    const float clip = value ? a.cV : a.cK;
    const uint4 *rows = reinterpret_cast<const uint4 *>(value ? a.bf.v : a.bf.k) + c0;                       // 16 uint4 a row
    uint32_t *codes = reinterpret_cast<uint32_t *>(value ? a.i4.codes_v : a.i4.codes_k) + c0;               // 16 words a row
    uint32_t *recs = reinterpret_cast<uint32_t *>(a.i4.scale_zero) + value + 2 * (hl / kLanes);             // 2 G words a row
    const size_t two = (size_t)a.n_kv * 32;                                                                 // uint4s, two tokens
    const uint4 *line = rows - c0 + 8 * tok;
    Slot s = find(a, pt0, h, (int)p, 32);
    for (; p < hi; p += stride) {
        const Slot cur = s;
        const int first = lo - (int)p - tok, last = (int)(hi - p) - tok;     // row 2 j is in the range if in first .. last - 1
        const uint4 *from = rows + (cur.bf + tok * a.n_kv) * 16;
        uint32_t *to = codes + ((size_t)cur.i4 + tok) * 16, *rec = recs + ((size_t)cur.i4 + tok) * 2 * G;
        uint32_t w[STEPS][8];
        if (cur.on) {
#pragma unroll
            for (int j = 0; j < STEPS; ++j) {
                const uint4 x0 = from[j * two], x1 = from[j * two + c1 - c0];
                w[j][0] = x0.x, w[j][1] = x0.y, w[j][2] = x0.z, w[j][3] = x0.w;
                w[j][4] = x1.x, w[j][5] = x1.y, w[j][6] = x1.z, w[j][7] = x1.w;
            }
        }
        if (p + stride < hi) {
            s = find(a, pt0, h, (int)(p + stride), 32);
            // the next run's 32 lines of 128 bytes on their way to L2, one a lane
            if (STEPS == 4 && s.on) prefetch_l2(line + (s.bf + hl * a.n_kv) * 16);
        }
        if (!cur.on) continue;
        uint32_t r[STEPS];
#pragma unroll
        for (int j = 0; j < STEPS; ++j) r[j] = range16<GROUP>(w[j]);
        // the steps' records, each formed once or twice a group, not by all its lanes
        uint32_t sz[STEPS / kOwn];
        float iv[STEPS / kOwn];
        bool odd = false;
#pragma unroll
        for (int q = 0; q < STEPS / kOwn; ++q) {
            uint32_t x = r[q * kOwn];
#pragma unroll
            for (int j = 1; j < kOwn; ++j) x = own == j ? r[q * kOwn + j] : x;
            iv[q] = record(x, clip, &sz[q]);
            const int row = 2 * (q * kOwn + own);
            if (row >= first && row < last) {
                odd |= iv[q] < 0.0f;
                if ((hl & (kLanes - 1)) < kOwn) rec[row * 2 * G] = sz[q];
            }
        }
        const int lane0 = lane & ~(kLanes - 1);
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
            const uint32_t z = kOwn == 1 ? sz[j] : __shfl_sync(0xffffffffu, sz[j / kOwn], lane0 | (j % kOwn));
            const float inv = kOwn == 1 ? iv[j] : __shfl_sync(0xffffffffu, iv[j / kOwn], lane0 | (j % kOwn));
            uint2 c = codes16(w[j], z, inv);
            if (STEPS == 1 && odd) c = codes16_any(w[j], z);
            if (2 * j >= first && 2 * j < last) {
                if (G == 1) {
                    to[j * 32] = c.x;
                    to[j * 32 + 8] = c.y;
                } else {
                    *reinterpret_cast<uint2 *>(to + j * 32) = c;
                }
            }
        }
        if (STEPS > 1 && __any_sync(0xffffffffu, odd)) {          // groups that codes16 does not do: over again
#pragma unroll 1
            for (int j = 0; j < STEPS; ++j) {
                uint32_t z = sz[0];
                float inv = iv[0];
#pragma unroll
                for (int q = 1; q < STEPS / kOwn; ++q)
                    if (j / kOwn == q) z = sz[q], inv = iv[q];
                z = __shfl_sync(0xffffffffu, z, lane0 | (j % kOwn));
                inv = __shfl_sync(0xffffffffu, inv, lane0 | (j % kOwn));
                if (inv < 0.0f && 2 * j >= first && 2 * j < last) {
                    const uint4 x0 = from[j * two], x1 = from[j * two + c1 - c0];
                    const uint32_t x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                    const uint2 c = codes16_any(x, z);
                    to[j * 32] = c.x;
                    to[j * 32 + c1 - c0] = c.y;
                }
            }
        }
    }
}

// grid (X, Hkv, batch).  Ranges that the CTAs' warps cover with two steps each are done one step at a time, which
// is done sooner; four steps a run share more.  One and four, with the promotion after it: 32 requests of one
// token 8.3 and 9.0 us; 8 heads, 600 tokens 10.3 and 12.3 us, 1,200 11.5 and 12.4, 2,400 13.1 and 13.1, 4,800
// 22.6 and 19.3, 100K 274 and 187.
template <int GROUP>
__global__ void __launch_bounds__(kThreads, 2) demote4_kernel(RangeArgs a) {
    int lo, hi;
    pdl_wait();
    if (!read_range(a, blockIdx.z, lo, hi)) return;
    if (hi - lo <= (int)gridDim.x * (kThreads / 8)) demote_range<GROUP, 1>(a, lo, hi);
    else demote_range<GROUP, 4>(a, lo, hi);
}

// grid (X, Hkv, batch): CTA x takes 16-token tiles x, x + X, ... of its request's range for its kv head.
template <int GROUP>
__global__ void __launch_bounds__(kThreads) promote4_kernel(RangeArgs a) {
    const int h = blockIdx.y, b = blockIdx.z, hl = threadIdx.x & 7, row = threadIdx.x >> 4;
    const bool value = threadIdx.x & 8;
    int lo, hi;
    pdl_wait();
    if (!read_range(a, b, lo, hi)) return;
    constexpr int G = kHeadDim / GROUP;                          // groups a row
    const int step = gridDim.x * 16;
    const long long begin = (lo & ~15) + (long long)blockIdx.x * 16;
    if (begin >= hi) return;
    const size_t pt0 = (size_t)b * a.max_pages;
    uint4 *rows = reinterpret_cast<uint4 *>(const_cast<uint16_t *>(value ? a.bf.v : a.bf.k));               // 16 uint4 a row
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(value ? a.i4.codes_v : a.i4.codes_k);        // 16 words a row
    const uint32_t *recs = reinterpret_cast<const uint32_t *>(a.i4.scale_zero) + value;                     // 2 G words a row
    auto place = [&](long long tile) {
        const int pos = (int)tile + row;
        return pos >= lo && pos < hi ? find(a, pt0, h, pos, 16) : Slot{false, 0, 0};
    };
    // chunks hl and hl + 8 whatever the group: eight lanes write 128 bytes in a row
    uint32_t c0 = 0, c1 = 0, z0 = 0, z1 = 0;
    Slot s = place(begin);
    auto fetch = [&]() {
        const uint32_t *from = codes + (size_t)s.i4 * 16, *rec = recs + (size_t)s.i4 * 2 * G;
        c0 = from[hl];
        c1 = from[hl + 8];
        z0 = rec[2 * (8 * hl / GROUP)];
        z1 = G == 1 ? z0 : rec[2 * ((64 + 8 * hl) / GROUP)];
    };
    if (s.on) fetch();
    for (long long p = begin; p < hi; p += step) {
        const Slot cur = s;
        const uint32_t k0 = c0, k1 = c1, y0 = z0, y1 = z1;
        s.on = false;
        if (p + step < hi) s = place(p + step);
        if (s.on) fetch();
        if (cur.on) {
            rows[cur.bf * 16 + hl] = restore8(k0, y0);
            rows[cur.bf * 16 + hl + 8] = restore8(k1, y1);
        }
    }
}

template <bool DEMOTE>
cudaError_t launch(const oscar_layout_t &L, const RangeArgs &a, int batch, cudaStream_t st) {
    // the CTAs that fit at once over all (head, request) pairs, no more than the longest possible range has tiles
    constexpr int kTile = DEMOTE ? kThreads / 4 : kThreads / 16;
    const long long most = ((long long)a.max_pages * L.page_size + kTile - 1) / kTile, pairs = (long long)batch * L.n_kv_heads;
    const long long want = std::max(1LL, (DEMOTE ? 2 : 8) * 152 / pairs);
    const dim3 grid((unsigned)(want < most ? want : most), L.n_kv_heads, batch);
    auto go = [&](auto demote, auto promote) { return launch_ahead(DEMOTE ? demote : promote, grid, kThreads, 0, st, a); };
    switch (L.group) {
        case 32: return go(demote4_kernel<32>, promote4_kernel<32>);
        case 64: return go(demote4_kernel<64>, promote4_kernel<64>);
        default: return go(demote4_kernel<128>, promote4_kernel<128>);
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
