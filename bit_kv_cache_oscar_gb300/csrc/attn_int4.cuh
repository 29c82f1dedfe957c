// Decode attention over an INT4 history with BF16 sink and recent rows, and the attention weight each
// position received, on the tensor cores.
//
// With a row's 4-bit codes n_c, scale s and zero z per channel group, a logit is
//   sm·(s·sum_c q_c n_c + z·sum_c q_c)
// and an output sum_t p_t v_t = sum_t (p_t s_t) n_t + sum_t p_t z_t: both contractions meet the codes
// themselves, so the codes are the A operand of mma.sync m16n8k16 (f16 in, fp32 accumulate) and scales
// and zeros stay outside.  A nibble n in bits 0..3, 2..5, 4..7 or 6..9 of an f16 with no exponent bits is the
// subnormal n·2^-24 to n·2^-18, so unpacking eight codes is one or two shifts and four ANDs; the powers of two
// go into the other operand or the result.  q is bf16 and exact in f16 after a power-of-two scaling of
// each head (elements down to 2^-25 of its largest).  p·s goes in as two f16 parts, 22 bits together: codes are
// not centred, so the zero points cancel most of the sum, and what is lost of it counts hundreds of times over
// in the output of a long history.
// The parts are scaled by a power of two that follows the largest p·s met so far, not the largest s: a row
// whose scale is far above the others' and whose weight is far below must not push them out of f16's range.
// The contractions have 8 columns: the query heads of one kv head, twice for up to four heads, whose second
// four columns take the lower parts of p·s (and of the BF16 rows' p) in the same instructions.
//
// A CTA takes one kv head of one split; each of its warps takes every W-th block of 32 tokens on its own
// (2 KB of key codes, 2 KB of value codes, their scale/zero records) through a ring of stages that its
// lane 0 fills with bulk tensor copies (64-byte swizzle: conflict-free ldmatrix of key rows and
// ldmatrix.trans of value rows), so no warp waits for another before the end.  p moves from the logits'
// accumulator layout to the value product's B operand by movmatrix.  The running maximum is only
// raised when a logit passes it by 2^8: a rescale of the accumulators is rare.
// The BF16 rows are dealt out in tiles of 16 to the same warps, which work on them while their first
// blocks are on the way.  With counters, the last CTA of a (request, kv head) to finish merges all its
// slots, in slot order.
// W is 16 (one CTA an SM) when the launch has a CTA for each SM at most, else 8, or 4 for the weights, whose
// CTAs have no results to join: several CTAs an SM, so that one's start and end hide behind another's stream.
// Every wait is bounded: one that gives up sets OSCAR_DEV_WAIT_TIMEOUT.
//
// Measured (passes back to back, 32 query and 8 kv heads, group 128): 100K tokens 29.4 us: 8 us to the first
// block (lengths, page ids and the first copies of all warps at once), 16 to the loop's end (110 MB in all), 5 to
// join warps and splits; a ragged batch of 32, 64K to 100K, 528 us = 5.5 TB/s (0.82 of a copy's rate): issue slots
// (661 instructions a block) and HBM.  64 query heads and groups of 32, 4 x 131K: 176 us = 3.8 TB/s: issue slots, 928
// instructions a block.  What the value product's precision costs of that, with the bf16 outputs' distance from
// fp32 arithmetic: p·s in one part and one running sum 27.4, 486 and 141 us, 2.0, 2.1 and 2.1e-3 of their size; two
// parts and one running sum 28.4, 497 and 168 us, 1.6, 2.0 and 3.5e-3 (the sum's truncation, twice as often for eight
// heads); as it is 0.44, 0.50 and 0.54e-3.  Codes centred by one more operation each: 0.01, 0.17 and 0.08e-3, in 32,
// 605 and 192 us.  Weights, ragged batch of 8: 76 us = 5.4 TB/s.

#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstring>

#include "attn_int4_args.cuh"
#include "merge_math.cuh"
#include "ptx.cuh"
#include "tma.cuh"

namespace oscar {

namespace {

constexpr uint32_t kM0 = 0x000F000Fu, kM1 = 0x00F000F0u;                         // keys: codes n as n·2^-24 and 16n·2^-24
constexpr uint32_t kV0 = 0x003C003Cu, kV1 = 0x03C003C0u;                         // values: n·2^-22 and n·2^-18
constexpr float kVScale0 = 0x1p-22f, kVScale1 = 0x1p-18f;
constexpr int kResRow = kHeadDim + 4;           // floats of a result row: heads 2 t, t = 0..3, in different banks
constexpr float kNone = -1e30f;                  // running maximum before the first token
constexpr float kSlack = 8.f;                    // logits (base 2) may pass the running maximum by this
constexpr int kPShift = 11;                      // a new scaling brings the largest p·s into [2^11, 2^12); near 2^15 another is due
constexpr float kPMost = 0x1p110f;               // the largest scaling: that of sums that are still all zero
constexpr uint32_t kHighPart = 0xFFFFE000u;      // fp32 bits that f16 holds

// One stage of one warp: key codes [32][64 B], value codes, scale/zero records [32][NG][8 B].
template <int NG, bool MASS, int W>
struct Ring {
    static constexpr int codes = MASS ? 2048 : 4096;
    static constexpr int bytes = codes + kBlock * NG * 8;
    static constexpr int stride = (bytes + 511) & ~511;          // the swizzle pattern repeats every 512 bytes
    static constexpr int n = MASS ? 4 : (NG == 4 ? 2 : 3);        // as many as 16 warps an SM leave room for
    static constexpr int total = W * n * stride;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t *>(&v); }
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_b2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Heads of column c: up to four heads have their columns twice, for the two parts of p·s.
template <int G>
__device__ __forceinline__ int column_head(int c) { return G <= 4 ? c & 3 : c; }
__device__ __forceinline__ float high_part(float x) { return __uint_as_float(__float_as_uint(x) & kHighPart); }
__device__ __forceinline__ void add4(float (&a)[4], const float (&d)[4]) {       // in packed pairs
#pragma unroll
    for (int i = 0; i < 4; i += 2)
        asm("{\n.reg .b64 x, y;\nmov.b64 x, {%0, %1};\nmov.b64 y, {%2, %3};\nadd.rn.f32x2 x, x, y;\nmov.b64 {%0, %1}, x;\n}"
            : "+f"(a[i]), "+f"(a[i + 1])
            : "f"(d[i]), "f"(d[i + 1]));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ void tma_rows(uint32_t dst, const void *tmap, int row, uint32_t bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3}], [%4], %5;"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(row), "r"(bar), "l"(pol)
        : "memory");
}
__device__ __forceinline__ float col_sum(float x) {       // over the 8 lanes of a column
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}
__device__ __forceinline__ float col_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}

// What a warp holds of the G heads' partials when it is done: column c = 2 t + j is head c.
struct ColState {
    float m[2], l[2];
};

// The power of two that brings x > 0, 2^e <= x < 2^(e + 1), to 2^kPShift.
__device__ __forceinline__ float scaling(float x) {
    const int e = max((int)(__float_as_uint(x) >> 23) - 127, kPShift - 110);
    return __uint_as_float((uint32_t)(kPShift - e + 127) << 23);
}

// Limit of (logit - maximum) + log2 s, as the history's loop forms it, under this scaling: 2^15 for p·s·vinv, the 2^-7 of the
// sum's own rounding far below f16's end.
__device__ __forceinline__ float product_limit(float vinv) { return 65536.f + 127.f + 15.f - (float)((int)(__float_as_uint(vinv) >> 23) - 127); }

// ---- the BF16 rows: [0, min(sink, T)) and [hist_end, T), 16-token tiles dealt out to the warps ----------
struct Window {
    int n0, lo1, T, sink_tiles, rec0, tiles;
    __device__ __forceinline__ Window(int sink, int T_, int he) {
        T = T_;
        n0 = min(sink, T);
        lo1 = max(he, n0);
        sink_tiles = (n0 + 15) / 16;
        rec0 = lo1 / 16;
        tiles = sink_tiles + (lo1 < T ? (T + 15) / 16 - rec0 : 0);
    }
};

// The rows of tile k on their way to shared memory: 16 key rows of 256 bytes, then 16 value rows; value rows
// outside the tile's positions are zeroed.  False (and no copy) for a bad page.
struct WindowTile {
    int p0, lo, hi;
};
template <bool MASS>
__device__ __forceinline__ bool issue_tile(const Attn4Args &a, const Window &w, int k, int b, int h, int lane, uint8_t *dst, uint32_t bar,
                                           WindowTile &x) {
    const bool in_sink = k < w.sink_tiles;
    x.p0 = (in_sink ? k : w.rec0 + k - w.sink_tiles) * 16;
    x.lo = in_sink ? 0 : w.lo1;
    x.hi = in_sink ? w.n0 : w.T;
    const int page = a.bpt[(size_t)b * a.max_pages + (x.p0 >> a.page_shift)];
    if ((uint32_t)page >= (uint32_t)a.bf.n_pages) {
        if (lane == 0) flag_status(a.status, OSCAR_DEV_BAD_BF16_PAGE);
        return false;
    }
    const int rows = min(x.hi, x.p0 + 16) - max(x.lo, x.p0), r = lane & 15;
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)rows * 256 * (MASS ? 1 : 2));
    __syncwarp();
    if (!MASS || lane < 16) {
        uint8_t *to = dst + lane * 256;
        if (x.p0 + r >= x.lo && x.p0 + r < x.hi) {
            const size_t row = ((size_t)page << a.page_shift) + (x.p0 & ((1 << a.page_shift) - 1)) + r;
            tma_load_1d(saddr(to), (lane < 16 ? a.bf.k : a.bf.v) + (row * a.n_kv + h) * kHeadDim, 256, bar);
        } else if (lane >= 16) {
            for (int i = 0; i < 16; ++i) reinterpret_cast<uint4 *>(to)[i] = make_uint4(0, 0, 0, 0);
        }
    }
    return true;
}

// Fold the warp's tiles first, first + every, ... (the first is under way in buf, `ok` unless its page is bad).
// Leaves the running maxima and sums in cs, and the accumulators in the layout and scaling (vinv) that the
// history's loop goes on with.  Lane (g, t) reads channels 32 i + 8 t .. + 7 of tokens g and g + 8; value rows
// become the A operand through movmatrix (channels 32 c + 4 n + 2 j of eight tokens are an 8 x 8 matrix), p
// the B operand in two bf16 parts.
template <int G, bool MASS>
__device__ __forceinline__ void window_tiles(const Attn4Args &a, const Window &w, int b, int h, int first, int every, int lane,
                                             uint8_t *buf, uint32_t bar, bool ok, WindowTile &x, ColState &cs, float (&out)[4][2][4],
                                             float (&vinv)[2]) {
    const int g = lane >> 2, t = lane & 3, sh = a.page_shift, head = MASS ? g : column_head<G>(g);
    const bool lower = G <= 4 && t >= 2;                       // this lane's columns take the lower parts
    uint4 bq[4];
    const uint16_t *qr = a.q + ((size_t)b * a.n_kv * G + h * G + (head < G ? head : 0)) * kHeadDim + 8 * t;
#pragma unroll
    for (int i = 0; i < 4; ++i) bq[i] = head < G ? *reinterpret_cast<const uint4 *>(qr + 32 * i) : make_uint4(0, 0, 0, 0);
    uint32_t phase = 0;
#pragma unroll 1
    for (int k = first; k < w.tiles; k += every) {
        if (k != first) {
            fence_proxy_async_smem();                          // the tile before is read, its zeros are written
            __syncwarp();
            ok = issue_tile<MASS>(a, w, k, b, h, lane, buf, bar, x);
        }
        if (!ok) continue;
        if (!mbar_wait(bar, phase)) {
            if (lane == 0) flag_status(a.status, OSCAR_DEV_WAIT_TIMEOUT);
            mbar_wait(bar, phase);                             // its copies land before this memory is used again
            break;
        }
        phase ^= 1;
        __syncwarp();
        const uint4 *rows = reinterpret_cast<const uint4 *>(buf) + g * 16 + t;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 k0 = rows[4 * i], k1 = rows[4 * i + 128];
            mma16816_bf16(d, k0.x, k1.x, k0.y, k1.y, bq[i].x, bq[i].y);
            mma16816_bf16(d, k0.z, k1.z, k0.w, k1.w, bq[i].z, bq[i].w);
        }
        float s[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool in = x.p0 + 8 * r + g >= x.lo && x.p0 + 8 * r + g < x.hi;
#pragma unroll
            for (int j = 0; j < 2; ++j) s[r][j] = in ? d[2 * r + j] * a.scale2 : -INFINITY;
        }
        if (MASS) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float y = ex2_approx(s[r][0] - cs.m[0]) + ex2_approx(s[r][1] - cs.m[1]);
                y += __shfl_xor_sync(0xffffffffu, y, 1);
                y += __shfl_xor_sync(0xffffffffu, y, 2);
                const int p = x.p0 + 8 * r + g;
                if (t == 0 && p >= x.lo && p < x.hi) atomicAdd(a.mass + (((size_t)b * a.n_kv + h) * a.max_pages << sh) + p, y);
            }
            continue;
        }
        float al[2], pr[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float m = fmaxf(cs.m[j], col_max(fmaxf(s[0][j], s[1][j])));
            al[j] = ex2_approx(cs.m[j] - m);
            cs.m[j] = m;
            pr[0][j] = ex2_approx(s[0][j] - m);
            pr[1][j] = ex2_approx(s[1][j] - m);
            cs.l[j] = fmaf(cs.l[j], al[j], pr[0][j] + pr[1][j]);
        }
        uint32_t bh[2], bl[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t hi = pack_b2(pr[r][0], pr[r][1]), lo = pack_b2(pr[r][0] - lo16(hi), pr[r][1] - hi16(hi));
            bh[r] = movmatrix_trans(lower ? lo : hi);
            if (G > 4) bl[r] = movmatrix_trans(lo);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 v0 = rows[4 * c + 256], v1 = rows[4 * c + 384];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t m0 = movmatrix_trans(__byte_perm(j ? v0.y : v0.x, j ? v0.w : v0.z, 0x5410));
                const uint32_t m1 = movmatrix_trans(__byte_perm(j ? v0.y : v0.x, j ? v0.w : v0.z, 0x7632));
                const uint32_t m2 = movmatrix_trans(__byte_perm(j ? v1.y : v1.x, j ? v1.w : v1.z, 0x5410));
                const uint32_t m3 = movmatrix_trans(__byte_perm(j ? v1.y : v1.x, j ? v1.w : v1.z, 0x7632));
#pragma unroll
                for (int e = 0; e < 4; ++e) out[c][j][e] *= al[e & 1];
                mma16816_bf16(out[c][j], m0, m1, m2, m3, bh[0], bh[1]);
                if (G > 4) mma16816_bf16(out[c][j], m0, m1, m2, m3, bl[0], bl[1]);
            }
        }
    }
    if (MASS) return;
    float top[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) top[e & 1] = fmaxf(top[e & 1], fabsf(out[c][j][e]));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        top[j] = col_max(top[j]);
        if (G <= 4) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 2));     // both parts of a head alike
        vinv[j] = scaling(top[j]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) out[c][j][e] *= vinv[e & 1] * (e >> 1 ? kVScale1 : kVScale0);
}

// ---- the history -------------------------------------------------------------------------------
template <int G, int NG, bool MASS, int W>
__device__ __forceinline__ void history_warp(const Attn4Args &a, const CUtensorMap *tmk, const CUtensorMap *tmv, uint8_t *ring,
                                             uint32_t bars, int b, int h, int split, int T, int he, int warp, int lane, float *res) {
    using R = Ring<NG, MASS, W>;
    const int g = lane >> 2, t = lane & 3, sh = a.page_shift, S = a.out.S, head = MASS ? g : column_head<G>(g);
    const bool lower = G <= 4 && t >= 2;           // this lane's columns take the lower parts of p·s
    const int first = a.sink / kBlock, nb = he > a.sink ? (he + kBlock - 1) / kBlock - first : 0;
    const int lo = first + (int)((long long)split * nb / S) + warp, hi = first + (int)((long long)(split + 1) * nb / S);
    const int n = lo < hi ? (hi - lo + W - 1) / W : 0;      // blocks lo, lo + W, ...
    const int32_t *pt = a.ipt + (size_t)b * a.max_pages;
    const uint64_t pol = l2_evict_first_policy();

    int pg0 = -1, pg1 = -1;        // lane j: pages of the two 16-token halves of block lo + W (batch + j)
    uint32_t ok = 0;               // two bits per stage: halves that were loaded
    auto issue = [&](int i, int st) {
        if ((i & 31) == 0) {
            const int p = (lo + W * (i + lane)) * kBlock;
            pg0 = pg1 = -1;
            if (i + lane < n) {
                if (p + 16 > a.sink && p < he) pg0 = pt[p >> sh];
                if (p + kBlock > a.sink && p + 16 < he) pg1 = pt[(p + 16) >> sh];
                if ((p + 16 > a.sink && p < he && (uint32_t)pg0 >= (uint32_t)a.i4_pages) ||
                    (p + kBlock > a.sink && p + 16 < he && (uint32_t)pg1 >= (uint32_t)a.i4_pages))
                    flag_status(a.status, OSCAR_DEV_BAD_INT4_PAGE);
            }
        }
        const int a0 = __shfl_sync(0xffffffffu, pg0, i & 31), a1 = __shfl_sync(0xffffffffu, pg1, i & 31);
        const bool ok0 = (uint32_t)a0 < (uint32_t)a.i4_pages, ok1 = (uint32_t)a1 < (uint32_t)a.i4_pages;
        ok = (ok & ~(3u << (2 * st))) | ((ok0 ? 1u : 0u) | (ok1 ? 2u : 0u)) << (2 * st);
        if (lane == 0) {
            const int p = (lo + W * i) * kBlock;
            const uint32_t dst = saddr(ring + st * R::stride), bar = bars + 8 * st;
            // pages of 32 or more: one box of 32 rows; pages of 16: a box a half
            const int rows = sh >= 5 ? kBlock : 16;
            const bool l0 = sh >= 5 ? ok0 || ok1 : ok0, l1 = sh >= 5 ? false : ok1;
            mbar_arrive_expect_tx(bar, (uint32_t)(l0 + l1) * rows * (R::bytes / kBlock));
            const int page[2] = {ok0 ? a0 : a1, a1};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!(half ? l1 : l0)) continue;
                const int row = ((page[half] * a.n_kv + h) << sh) + ((p + 16 * half) & ((1 << sh) - 1));
                tma_rows(dst + half * 1024, tmk, row, bar, pol);
                if (!MASS) tma_rows(dst + 2048 + half * 1024, tmv, row, bar, pol);
                tma_load_1d(dst + R::codes + half * 16 * NG * 8, a.sz + (size_t)row * NG * 4, (uint32_t)rows * NG * 8, bar, pol);
            }
        }
    };
    // The warp's first tile of BF16 rows, ahead of its blocks in the memory queues: it takes the first two
    // stages, so the blocks start in the third (in a ring of two: when the tiles are done).
    const Window win(a.sink, T, he);
    const int tile0 = warp * S + split, wbar = R::n;
    const bool has_tile = tile0 < win.tiles;
    WindowTile wt;
    bool tile_ok = false;
    if (has_tile) tile_ok = issue_tile<MASS>(a, win, tile0, b, h, lane, ring, bars + 8 * wbar, wt);
    const int st0 = has_tile ? 2 % R::n : 0, ahead = has_tile ? R::n - 2 : R::n;
    for (int i = 0; i < ahead && i < n; ++i) issue(i, (st0 + i) % R::n);

    ColState cs;
    float zs[NG][2], acc[4][2][4];
    float vinv[2] = {kPMost, kPMost};              // what this lane's columns' p·s are multiplied by, powers of two
#pragma unroll
    for (int i = 0; i < NG; ++i) zs[i][0] = zs[i][1] = 0.f;
    cs.m[0] = cs.m[1] = kNone;
    cs.l[0] = cs.l[1] = 0.f;
    if (MASS) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float l = 2 * t + j < G ? a.lse[(size_t)b * a.n_kv * G + h * G + 2 * t + j] : -INFINITY;
            cs.m[j] = l == -INFINITY ? INFINITY : l * kLog2e;
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][j][e] = 0.f;
    if (has_tile) {
        window_tiles<G, MASS>(a, win, b, h, tile0, S * W, lane, ring, bars + 8 * wbar, tile_ok, wt, cs, acc, vinv);
        fence_proxy_async_smem();
        __syncwarp();
        for (int i = ahead; i < R::n && i < n; ++i) issue(i, (st0 + i) % R::n);
    }

    // B operand of the logits: column g = its query head, channels 32 i + 8 t + e of chunk i; the odd
    // nibbles meet q/16.  fac undoes the scalings, qz is the zero's factor, per column and group.
    uint32_t bq[4][4];
    float fac[2], qz[NG][2];
    {
        uint4 w[4];
        const uint16_t *qr = a.q + ((size_t)b * a.n_kv * G + h * G + (head < G ? head : 0)) * kHeadDim + 8 * t;
        float mx = 0.f, qs[NG];
#pragma unroll
        for (int j = 0; j < NG; ++j) qs[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = head < G ? *reinterpret_cast<const uint4 *>(qr + 32 * i) : make_uint4(0, 0, 0, 0);
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mx = fmaxf(mx, fmaxf(fabsf(lo16(x[e])), fabsf(hi16(x[e]))));
                qs[i * NG / 4] += lo16(x[e]) + hi16(x[e]);
            }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int ex = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 117);   // |q| < 2^(ex + 1)
        const float mul = __uint_as_float((uint32_t)(14 - ex + 127) << 23), mul16 = mul * 0.0625f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bq[i][0] = pack_h2(lo16(w[i].x) * mul, lo16(w[i].z) * mul);
            bq[i][1] = pack_h2(hi16(w[i].x) * mul16, hi16(w[i].z) * mul16);
            bq[i][2] = pack_h2(lo16(w[i].y) * mul, lo16(w[i].w) * mul);
            bq[i][3] = pack_h2(hi16(w[i].y) * mul16, hi16(w[i].w) * mul16);
        }
        const float f = a.scale2 * __uint_as_float((uint32_t)(10 + ex + 127) << 23);   // 2^24 / mul
#pragma unroll
        for (int j = 0; j < 2; ++j) fac[j] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + j));
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            qs[k] += __shfl_xor_sync(0xffffffffu, qs[k], 1);
            qs[k] += __shfl_xor_sync(0xffffffffu, qs[k], 2);
#pragma unroll
            for (int j = 0; j < 2; ++j) qz[k][j] = __shfl_sync(0xffffffffu, qs[k] * a.scale2, 4 * (2 * t + j));
        }
    }
    float most[2] = {product_limit(vinv[0]), product_limit(vinv[1])};
    for (int i = 0, st = st0, round = 0, phase = 0; i < n; ++i) {
        if (!mbar_wait(bars + 8 * st, phase)) {
            if (lane == 0) flag_status(a.status, OSCAR_DEV_WAIT_TIMEOUT);
            // the copies still under way land before this memory is used again
            for (int k = i + 1; k < i + R::n && k < n; ++k) mbar_wait(bars + 8 * ((st0 + k) % R::n), (k / R::n) & 1);
            break;
        }
        const uint8_t *stage = ring + st * R::stride;
        const uint32_t sb = saddr(stage);
        const int p0 = (lo + W * i) * kBlock;
        const uint32_t okb = (ok >> (2 * st)) & 3u;
        const bool full = okb == 3u && p0 >= a.sink && p0 + kBlock <= he;

        float s[2][2][2];                            // [tile][row g, g + 8][column]
        uint32_t vw[2][2][NG];                       // value scale | zero of those rows
#pragma unroll
        for (int tl = 0; tl < 2; ++tl) {
            uint32_t w[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = tl * 16 + r * 8 + (lane & 7);
                ldmatrix_x4(sb + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4), w[r][0], w[r][1], w[r][2], w[r][3]);
            }
            float d[NG][4];
#pragma unroll
            for (int k = 0; k < NG; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[k][e] = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t x = w[0][c], y = w[1][c], x8 = x >> 8, y8 = y >> 8;
                mma16816_nv(d[c * NG / 4], x & kM0, y & kM0, x & kM1, y & kM1, bq[c][0], bq[c][1]);
                mma16816_nv(d[c * NG / 4], x8 & kM0, y8 & kM0, x8 & kM1, y8 & kM1, bq[c][2], bq[c][3]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = tl * 16 + r * 8 + g;
                const uint2 *rec = reinterpret_cast<const uint2 *>(stage + R::codes) + row * NG;
                float s0, s1, z0, z1;
#pragma unroll
                for (int k = 0; k < NG; ++k) {
                    const uint2 z = rec[k];
                    const float ks = lo16(z.x), kz = hi16(z.x);
                    s0 = k ? fmaf(ks, d[k][2 * r], s0) : ks * d[k][2 * r];
                    s1 = k ? fmaf(ks, d[k][2 * r + 1], s1) : ks * d[k][2 * r + 1];
                    z0 = k ? fmaf(kz, qz[k][0], z0) : kz * qz[k][0];
                    z1 = k ? fmaf(kz, qz[k][1], z1) : kz * qz[k][1];
                    vw[tl][r][k] = z.y;
                }
                s[tl][r][0] = fmaf(s0, fac[0], z0);
                s[tl][r][1] = fmaf(s1, fac[1], z1);
            }
        }
        if (!full) {
#pragma unroll
            for (int tl = 0; tl < 2; ++tl)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int p = p0 + tl * 16 + r * 8 + g;
                    if (p < a.sink || p >= he || !((okb >> tl) & 1u)) {
                        s[tl][r][0] = s[tl][r][1] = -INFINITY;
#pragma unroll
                        for (int k = 0; k < NG; ++k) vw[tl][r][k] = 0u;
                    }
                }
        }
        if (MASS) {
            float add = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float x = ex2_approx(s[u >> 1][u & 1][0] - cs.m[0]) + ex2_approx(s[u >> 1][u & 1][1] - cs.m[1]);
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (t == u) add = x;
            }
            const int p = p0 + 8 * t + g;
            if (p >= a.sink && p < he && ((okb >> (t >> 1)) & 1u))
                atomicAdd(a.mass + (((size_t)b * a.n_kv + h) * a.max_pages << sh) + p, add);
        } else {
            // Raise the running maximum when a block passes it, change the scaling when a p·s might pass f16's range:
            // looked at only where the lane's largest logit with its largest scale would, rows apart or not.  log2 s
            // is at most 0.09 above its exponent and fraction read as one number, bits/128 - 127.
            float top[2], over[2], far[2];                               // largest logit, that less the maximum, that with log2 s
            __nv_bfloat162 v2 = as_bf2(vw[0][0][0]);                     // scales in the low halves (never negative)
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int k = 0; k < NG; ++k) v2 = __hmax2(v2, as_bf2(vw[u >> 1][u & 1][k]));
            const float bits = __uint_as_float(__byte_perm(as_u32(v2), 0x4B000000u, 0x7610));       // 2^23 + the scale's 16 bits
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                top[j] = fmaxf(fmaxf(s[0][0][j], s[0][1][j]), fmaxf(s[1][0][j], s[1][1][j]));
                over[j] = top[j] - cs.m[j];                              // as for p: exact where it matters
                far[j] = fmaf(bits, 0x1p-7f, over[j]);                   // 2^16 + 127 + log2(p·s)
            }
            if (__any_sync(0xffffffffu, fmaxf(over[0], over[1]) > kSlack || far[0] > most[0] || far[1] > most[1])) {
                float f[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float m = fmaxf(cs.m[j], col_max(top[j])), al = ex2_approx(cs.m[j] - m);
                    // what was summed shrinks by al, so the scaling may grow by as much (by 2^100 at most)
                    const float up = __uint_as_float((uint32_t)(__float2int_rn(fminf(m - cs.m[j], 100.f)) + 127) << 23), old = vinv[j];
                    cs.m[j] = m;
                    cs.l[j] *= al;
#pragma unroll
                    for (int k = 0; k < NG; ++k) zs[k][j] *= al;
                    float x = 0.f;
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int k = 0; k < NG; ++k) x = fmaxf(x, ex2_approx(s[u >> 1][u & 1][j] - m) * lo16(vw[u >> 1][u & 1][k]));
                    x = col_max(x);
                    vinv[j] = fminf(old * up, kPMost);
                    if (x * vinv[j] > 0x1p14f) vinv[j] = scaling(x);
                    f[j] = al * (vinv[j] / old);                         // both powers of two
                    most[j] = product_limit(vinv[j]);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[c][j][e] *= f[e & 1];
            }
            float w[4][2], z4[NG][2];                            // p·vinv of rows g, g + 8 of both tiles; the zeros' part of the block
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float p = ex2_approx(s[u >> 1][u & 1][j] - cs.m[j]);
                    cs.l[j] += p;
#pragma unroll
                    for (int k = 0; k < NG; ++k) {
                        const float z = hi16(vw[u >> 1][u & 1][k]);
                        z4[k][j] = u ? fmaf(p, z, z4[k][j]) : p * z;
                    }
                    w[u][j] = p * vinv[j];
                }
#pragma unroll
            for (int k = 0; k < NG; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) zs[k][j] += z4[k][j];
            // 32 channels at a time.  A block's products are summed on their own, then added: the tensor cores truncate
            // their sums, and a running one of codes that are never negative would drift by a bit each time.  Products
            // keep 25 bits below the largest one's exponents, for which a subnormal's is 2^-14: codes are moved up, to
            // 2^-22 and 2^-18 a unit, so that weights 2^-7 and 2^-11 of their tile's largest still lose nothing.
            uint32_t bp[4], bl[4], vc[2][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c % 2 == 0)
#pragma unroll
                    for (int tl = 0; tl < 2; ++tl) {
                        const int row = tl * 16 + (lane & 15);
                        ldmatrix_x4_trans(sb + 2048 + row * 64 + (((c + (lane >> 4)) ^ ((row >> 1) & 3)) << 4), vc[tl][0], vc[tl][1], vc[tl][2],
                                          vc[tl][3]);
                    }
                const int k = c * NG / 4;
                if (c * NG % 4 == 0)                             // a new group
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float v = lo16(vw[u >> 1][u & 1][k]), y0 = w[u][0] * v, y1 = w[u][1] * v, h0 = high_part(y0), h1 = high_part(y1);
                        if (G <= 4) {
                            bp[u] = movmatrix_trans(pack_h2(lower ? y0 - h0 : h0, lower ? y1 - h1 : h1));
                        } else {
                            bp[u] = movmatrix_trans(pack_h2(h0, h1));
                            bl[u] = movmatrix_trans(pack_h2(y0 - h0, y1 - h1));
                        }
                    }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int tl = 0; tl < 2; ++tl) {
                        const uint32_t a0 = vc[tl][2 * (c & 1)], a1 = vc[tl][2 * (c & 1) + 1], x = j ? a0 >> 6 : a0 << 2, y = j ? a1 >> 6 : a1 << 2;
                        if (G > 4) mma16816_nv(d, x & kV0, x & kV1, y & kV0, y & kV1, bl[2 * tl], bl[2 * tl + 1]);
                        mma16816_nv(d, x & kV0, x & kV1, y & kV0, y & kV1, bp[2 * tl], bp[2 * tl + 1]);
                    }
                    add4(acc[c][j], d);
                }
            }
        }
        __syncwarp();
        if (i + R::n < n) issue(i + R::n, st);
        if (++st == R::n) st = 0;
        if (++round == R::n) {                           // every stage once more
            round = 0;
            phase ^= 1;
        }
    }
    if (MASS) return;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        cs.l[j] = col_sum(cs.l[j]);
#pragma unroll
        for (int k = 0; k < NG; ++k) zs[k][j] = col_sum(zs[k][j]);
    }
    __syncthreads();                                 // every warp is done with its ring: results take its place
    float *wm = res, *wl = res + W * 8, *wa = res + 2 * W * 8 + warp * G * kResRow;
    if (g == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            wm[warp * 8 + 2 * t + j] = cs.l[j] > 0.f ? cs.m[j] : -INFINITY;
            wl[warp * 8 + 2 * t + j] = cs.l[j];
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {                // head 2 t + e, channels 32 c + 4 g .. + 3
            const float up = 1.f / vinv[e], z = zs[c * NG / 4][e];
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = acc[c][i >> 1][2 * (i & 1) + e] * (i & 1 ? 1.f / kVScale1 : 1.f / kVScale0) * up;
                if (G <= 4) x[i] += __shfl_xor_sync(0xffffffffu, x[i], 2);       // the upper parts' sum and the lower ones'
            }
            if (2 * t + e < G)
                *reinterpret_cast<float4 *>(wa + (2 * t + e) * kResRow + 32 * c + 4 * g) = make_float4(x[0] + z, x[1] + z, x[2] + z, x[3] + z);
        }
}

// One channel of a merged row: sum A over weight L, maximum M (oscar_merge's last steps).
__device__ __forceinline__ void write_out(const Attn4Args &a, size_t orow, int d, float A, float L, float M) {
    const bool on = L > 0.f;
    const float r = on ? __fdiv_rn(A, L) : 0.f;
    if (a.of) a.of[orow * kHeadDim + d] = r;
    if (a.o) a.o[orow * kHeadDim + d] = f32_to_bf16_rn(r);
    if (a.o_lse && d == 0) a.o_lse[orow] = on ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

// The merge of one kv head's G query heads over the S splits (slot S is empty), in oscar_merge's order and
// arithmetic.  A warp takes 32 channels of a head, 32 splits at a time: their rows are on their way while
// the lanes form the weights, a split each, and half of them always is while the other half is added up.
template <int G, int W>
__device__ __forceinline__ void merge_head(const Attn4Args &a, int b, int h) {
    constexpr int kHalf = 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, S = a.out.S;
    for (int item = warp; item < 4 * G; item += W) {
        const int hh = item >> 2, d = (item & 3) * 32 + lane;
        const size_t orow = ((size_t)b * a.n_kv + h) * G + hh, row0 = orow * (S + 1);
        const float *m = a.out.m + row0, *l = a.out.l + row0, *acc = a.out.acc + row0 * kHeadDim + d;
        float x[2][kHalf];
        auto load = [&](float (&r)[kHalf], int s0) {
#pragma unroll
            for (int i = 0; i < kHalf; ++i) r[i] = s0 + i < S ? __ldcg(acc + (size_t)(s0 + i) * kHeadDim) : 0.f;
        };
        load(x[0], 0);
        load(x[1], kHalf);
        float l1 = lane < S ? __ldcg(l + lane) : 0.f, m1 = lane < S ? __ldcg(m + lane) : 0.f;
        float M = l1 > 0.f ? m1 : -INFINITY;
        for (int i = 32 + lane; i < S; i += 32) {
            const float li = __ldcg(l + i), mi = __ldcg(m + i);
            if (li > 0.f) M = fmaxf(M, mi);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float L = 0.f, A = 0.f;
        for (int s0 = 0; s0 < S; s0 += 32) {
            const float li = l1, wi = li > 0.f ? exp2_taylor(__fsub_rn(m1, M)) : 0.f;
            const bool more = s0 + 32 + lane < S;
            l1 = more ? __ldcg(l + s0 + 32 + lane) : 0.f;
            m1 = more ? __ldcg(m + s0 + 32 + lane) : 0.f;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    if (s0 + p * kHalf + i >= S) break;
                    const float lw = __shfl_sync(0xffffffffu, li, p * kHalf + i), w = __shfl_sync(0xffffffffu, wi, p * kHalf + i);
                    L = lw > 0.f ? __fmaf_rn(lw, w, L) : L;
                    A = lw > 0.f ? __fmaf_rn(x[p][i], w, A) : A;
                }
                load(x[p], s0 + 32 + p * kHalf);
            }
        }
        write_out(a, orow, d, A, L, M);
    }
}

// grid (S, Hkv, batch): CTA x takes split x; the first of each (request, kv head) also writes slot S, empty.
template <int G, int NG, bool MASS, int W>
__global__ void __launch_bounds__(W * 32, 16 / W)
    attn4_kernel(Attn4Args a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using R = Ring<NG, MASS, W>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[W * (R::n + 1)];           // a warp's stages, then its tile of BF16 rows
    __shared__ int last;
    __shared__ float wf[W * 8], wM[8];
    uint8_t *smem = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
    const int h = blockIdx.y, b = blockIdx.z, S = a.out.S, slot = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
        for (int i = 0; i <= R::n; ++i) mbar_init(saddr(&bars[warp * (R::n + 1) + i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    pdl_wait();
    int T, he;
    read_lengths(a.seq_len, a.hist_end, b, a.sink, a.max_pages << a.page_shift, a.status, T, he);
    float *res = reinterpret_cast<float *>(smem);
    history_warp<G, NG, MASS, W>(a, &tmk, &tmv, smem + warp * R::n * R::stride, saddr(&bars[warp * (R::n + 1)]), b, h, slot, T, he, warp,
                                 lane, res);
    if (MASS) return;
    __syncthreads();
    const size_t S1 = (size_t)S + 1, row0 = ((size_t)b * a.n_kv * G + h * G) * S1;
    // every warp's weight 2^(m - M) once, then the sums
    const float *wm = res, *wl = res + W * 8, *wa = res + 2 * W * 8;
    if (threadIdx.x < W * 8) {
        const int hh = threadIdx.x & 7;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, wm[w * 8 + hh]);
        wf[threadIdx.x] = M != -INFINITY ? exp2f(wm[threadIdx.x] - M) : 0.f;
        if (threadIdx.x < 8) wM[hh] = M;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < G * kHeadDim; e += W * 32) {
        const int hh = e / kHeadDim, d = e % kHeadDim;
        const float M = wM[hh];
        float L = 0.f, A = 0.f;
#pragma unroll 4
        for (int w = 0; w < W; ++w) {
            const float f = wf[w * 8 + hh], x = wa[(w * G + hh) * kResRow + d];
            L = fmaf(wl[w * 8 + hh], f, L);
            A = fmaf(f > 0.f ? x : 0.f, f, A);
        }
        const size_t row = row0 + hh * S1 + slot;
        a.out.acc[row * kHeadDim + d] = A;
        if (d == 0) {
            a.out.m[row] = M;
            a.out.l[row] = L;
        }
        if (slot == 0) {
            a.out.acc[(row + S) * kHeadDim + d] = 0.f;
            if (d == 0) {
                a.out.m[row + S] = -INFINITY;
                a.out.l[row + S] = 0.f;
            }
        }
        if (S == 1 && a.counters) write_out(a, ((size_t)b * a.n_kv + h) * G + hh, d, A, L, M);   // weight 2^0: merged
    }
    if (!a.counters || S == 1) return;
    __syncthreads();                                  // the slot is written; the count releases it
    if (threadIdx.x == 0) {
        int32_t *c = a.counters + (size_t)b * a.n_kv + h;
        int32_t n;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(n) : "l"(c) : "memory");
        last = n == S - 1;
        if (last) *c = 0;
    }
    __syncthreads();
    if (last) merge_head<G, W>(a, b, h);
}

template <int G, int NG, bool MASS, int W>
cudaError_t launch_one(const Attn4Args &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int batch, cudaStream_t st) {
    const int combine = (2 * W * 8 + W * G * kResRow) * 4;
    int smem = Ring<NG, MASS, W>::total;
    if (!MASS && smem < combine) smem = combine;
    smem += 1024;
    auto kern = attn4_kernel<G, NG, MASS, W>;
    if (cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(kern), smem)) return e;
    return launch_ahead(kern, dim3(a.out.S, a.n_kv, batch), W * 32, smem, st, a, tmk, tmv);
}

template <int G, bool MASS, int W>
cudaError_t launch_group(const Attn4Args &a, int group, const CUtensorMap &tmk, const CUtensorMap &tmv, int batch, cudaStream_t st) {
    switch (group) {
        case 32: return launch_one<G, 4, MASS, W>(a, tmk, tmv, batch, st);
        case 64: return launch_one<G, 2, MASS, W>(a, tmk, tmv, batch, st);
        default: return launch_one<G, 1, MASS, W>(a, tmk, tmv, batch, st);
    }
}

}  // namespace

template <int G>
cudaError_t launch_attn4(const Attn4Args &a, int group, bool mass, const CUtensorMap &tmk, const CUtensorMap &tmv, int batch,
                         cudaStream_t st) {
    const bool wide = (long long)a.out.S * a.n_kv * batch <= kSms;       // a CTA for each SM at most: 16 warps each
    if (mass) return wide ? launch_group<G, true, 16>(a, group, tmk, tmv, batch, st) : launch_group<G, true, 4>(a, group, tmk, tmv, batch, st);
    return wide ? launch_group<G, false, 16>(a, group, tmk, tmv, batch, st) : launch_group<G, false, 8>(a, group, tmk, tmv, batch, st);
}

}  // namespace oscar
