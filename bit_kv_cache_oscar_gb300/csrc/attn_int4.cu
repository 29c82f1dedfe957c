// Decode attention over an INT4 history with BF16 sink and recent rows, and the attention weight each
// position received, on the tensor cores.
//
// With a row's 4-bit codes n_c, scale s and zero z per channel group, a logit is
//   sm·(s·sum_c q_c n_c + z·sum_c q_c)
// and an output sum_t p_t v_t = sum_t (p_t s_t) n_t + sum_t p_t z_t: both contractions meet the codes
// themselves, so the codes are the A operand of mma.sync m16n8k16 (f16 in, fp32 accumulate) and scales
// and zeros stay outside.  A nibble n in bits 0..3 or 4..7 of an f16 with no exponent bits is the
// subnormal n·2^-24 or 16n·2^-24, so unpacking eight codes is one shift and four ANDs; the powers of two
// go into the other operand or the result.  q is bf16 and exact in f16 after a power-of-two scaling of
// each head; p·s is rounded to f16 (2^-11 relative), scaled by a power of two that follows the value
// scales.  The contractions have 8 columns: the query heads of one kv head.
//
// A CTA takes one kv head of one split; each of its 8 warps takes every 8th block of 32 tokens on its
// own (2 KB of key codes, 2 KB of value codes, their scale/zero records) through a ring of stages that
// its lane 0 fills with bulk tensor copies (64-byte swizzle: conflict-free ldmatrix of key rows and
// ldmatrix.trans of value rows), so no warp waits for another before the end.  p moves from the logits'
// accumulator layout to the value product's B operand by movmatrix.  The running maximum is only
// raised when a logit passes it by 2^8: a rescale of the accumulators is rare.
// The BF16 rows are CTA 0 of each (request, kv head).  With counters, the last CTA of a (request, kv
// head) to finish merges all its slots, in slot order.
// Every wait is bounded: one that gives up sets OSCAR_DEV_WAIT_TIMEOUT.

#include <cuda.h>
#include <cuda_fp16.h>
#include <cstring>

#include "int4.cuh"
#include "merge_math.cuh"
#include "ptx.cuh"
#include "tma.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kBlock = 32;                       // tokens of one stage
constexpr uint32_t kM0 = 0x000F000Fu, kM1 = 0x00F000F0u;
constexpr float kNone = -1e30f;                  // running maximum before the first token
constexpr float kSlack = 8.f;                    // logits (base 2) may pass the running maximum by this
constexpr int kPShift = 6;                       // p·s is held at 2^6 below 2^(kSlack + 1): at most 2^15

// One stage of one warp: key codes [32][64 B], value codes, scale/zero records [32][NG][8 B].
template <int NG, bool MASS>
struct Ring {
    static constexpr int codes = MASS ? 2048 : 4096;
    static constexpr int bytes = codes + kBlock * NG * 8;
    static constexpr int stride = (bytes + 511) & ~511;          // the swizzle pattern repeats every 512 bytes
    static constexpr int n = MASS ? 4 : (NG == 4 ? 2 : 3);        // as many as two CTAs an SM leave room for
    static constexpr int total = kWarps * n * stride;
};

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
    int smem_bytes;            // from the aligned base on
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
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

// ---- the history -------------------------------------------------------------------------------
template <int G, int NG, bool MASS>
__device__ __forceinline__ void history_warp(const Attn4Args &a, const CUtensorMap *tmk, const CUtensorMap *tmv, uint8_t *ring,
                                             uint32_t bars, int b, int h, int split, int he, int warp, int lane, float *res) {
    using R = Ring<NG, MASS>;
    const int g = lane >> 2, t = lane & 3, sh = a.page_shift, S = a.out.S;
    const int first = a.sink / kBlock, nb = he > a.sink ? (he + kBlock - 1) / kBlock - first : 0;
    const int lo = first + (int)((long long)split * nb / S) + warp, hi = first + (int)((long long)(split + 1) * nb / S);
    const int n = lo < hi ? (hi - lo + kWarps - 1) / kWarps : 0;      // blocks lo, lo + 8, ...
    const int32_t *pt = a.ipt + (size_t)b * a.max_pages;
    const uint64_t pol = l2_evict_first_policy();

    int pg0 = -1, pg1 = -1;        // lane j: pages of the two 16-token halves of block lo + 8 (batch + j)
    uint32_t ok = 0;               // two bits per stage: halves that were loaded
    auto issue = [&](int i, int st) {
        if ((i & 31) == 0) {
            const int p = (lo + kWarps * (i + lane)) * kBlock;
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
            const int p = (lo + kWarps * i) * kBlock;
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
    for (int i = 0; i < R::n && i < n; ++i) issue(i, i);

    // B operand of the logits: column g = query head g, channels 32 i + 8 t + e of chunk i; the odd
    // nibbles meet q/16.  fac undoes the scalings, qz is the zero's factor, per column and group.
    uint32_t bq[4][4];
    float fac[2], qz[NG][2];
    {
        uint4 w[4];
        const uint16_t *qr = a.q + ((size_t)b * a.n_kv * G + h * G + (g < G ? g : 0)) * kHeadDim + 8 * t;
        float mx = 0.f, qs[NG];
#pragma unroll
        for (int j = 0; j < NG; ++j) qs[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = g < G ? *reinterpret_cast<const uint4 *>(qr + 32 * i) : make_uint4(0, 0, 0, 0);
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

    ColState cs;
    float zs[NG][2], acc[4][2][4];
    float vmax = 0.f, vinv = 1.f;                  // value scales seen are at most vmax = 2^(e + 1); vinv = 2^(kPShift - e)
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
    for (int i = 0; i < NG; ++i) zs[i][0] = zs[i][1] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;

    for (int i = 0, st = 0, phase = 0; i < n; ++i) {
        if (!mbar_wait(bars + 8 * st, phase)) {
            if (lane == 0) flag_status(a.status, OSCAR_DEV_WAIT_TIMEOUT);
            // the copies still under way land before this memory is used again
            for (int k = i + 1; k < i + R::n && k < n; ++k) mbar_wait(bars + 8 * (k % R::n), (k / R::n) & 1);
            break;
        }
        const uint8_t *stage = ring + st * R::stride;
        const uint32_t sb = saddr(stage);
        const int p0 = (lo + kWarps * i) * kBlock;
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
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int k = 0; k < NG; ++k) {
                    const uint2 z = rec[k];
                    const float ks = lo16(z.x), kz = hi16(z.x);
                    s0 += fmaf(ks, d[k][2 * r] * fac[0], kz * qz[k][0]);
                    s1 += fmaf(ks, d[k][2 * r + 1] * fac[1], kz * qz[k][1]);
                    vw[tl][r][k] = z.y;
                }
                s[tl][r][0] = s0;
                s[tl][r][1] = s1;
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
            // raise the running maximum, or the bound on the value scales, when a block passes it
            float top0 = fmaxf(fmaxf(s[0][0][0], s[0][1][0]), fmaxf(s[1][0][0], s[1][1][0]));
            float top1 = fmaxf(fmaxf(s[0][0][1], s[0][1][1]), fmaxf(s[1][0][1], s[1][1][1]));
            float vs = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int k = 0; k < NG; ++k) vs = fmaxf(vs, fabsf(lo16(vw[u >> 1][u & 1][k])));
            if (__any_sync(0xffffffffu, top0 > cs.m[0] + kSlack || top1 > cs.m[1] + kSlack || vs > vmax)) {
                const float m0 = fmaxf(cs.m[0], col_max(top0)), m1 = fmaxf(cs.m[1], col_max(top1));
                const float al0 = ex2_approx(cs.m[0] - m0), al1 = ex2_approx(cs.m[1] - m1);
                cs.m[0] = m0;
                cs.m[1] = m1;
                cs.l[0] *= al0;
                cs.l[1] *= al1;
#pragma unroll
                for (int k = 0; k < NG; ++k) {
                    zs[k][0] *= al0;
                    zs[k][1] *= al1;
                }
                const uint32_t vb = __reduce_max_sync(0xffffffffu, __float_as_uint(vs));
                float down = 1.f;
                if (__uint_as_float(vb) > vmax) {
                    const int e = max((int)(vb >> 23) - 127, -100);
                    const float nv = __uint_as_float((uint32_t)(kPShift - e + 127) << 23);
                    down = vmax > 0.f ? nv / vinv : 0.f;         // a power of two (nothing but zeros was summed before)
                    vinv = nv;
                    vmax = e >= 126 ? INFINITY : __uint_as_float((uint32_t)(e + 1 + 127) << 23);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[c][j][e] *= (e & 1 ? al1 : al0) * down;
            }
#pragma unroll
            for (int tl = 0; tl < 2; ++tl) {
                uint32_t bp[NG][2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float q0 = ex2_approx(s[tl][r][0] - cs.m[0]), q1 = ex2_approx(s[tl][r][1] - cs.m[1]);
                    cs.l[0] += q0;
                    cs.l[1] += q1;
#pragma unroll
                    for (int k = 0; k < NG; ++k) {
                        const float v = lo16(vw[tl][r][k]) * vinv, z = hi16(vw[tl][r][k]);
                        zs[k][0] = fmaf(q0, z, zs[k][0]);
                        zs[k][1] = fmaf(q1, z, zs[k][1]);
                        bp[k][r] = movmatrix_trans(pack_h2(q0 * v, q1 * v));
                    }
                }
                const int row = tl * 16 + (lane & 15);
#pragma unroll
                for (int c = 0; c < 4; c += 2) {
                    uint32_t r0, r1, r2, r3;
                    ldmatrix_x4_trans(sb + 2048 + row * 64 + (((c + (lane >> 4)) ^ ((row >> 1) & 3)) << 4), r0, r1, r2, r3);
                    const int k0 = c * NG / 4, k1 = (c + 1) * NG / 4;
                    mma16816_nv(acc[c][0], r0 & kM0, r0 & kM1, r1 & kM0, r1 & kM1, bp[k0][0], bp[k0][1]);
                    mma16816_nv(acc[c + 1][0], r2 & kM0, r2 & kM1, r3 & kM0, r3 & kM1, bp[k1][0], bp[k1][1]);
                    r0 >>= 8; r1 >>= 8; r2 >>= 8; r3 >>= 8;
                    mma16816_nv(acc[c][1], r0 & kM0, r0 & kM1, r1 & kM0, r1 & kM1, bp[k0][0], bp[k0][1]);
                    mma16816_nv(acc[c + 1][1], r2 & kM0, r2 & kM1, r3 & kM0, r3 & kM1, bp[k1][0], bp[k1][1]);
                }
            }
        }
        __syncwarp();
        if (i + R::n < n) issue(i + R::n, st);
        if (++st == R::n) {
            st = 0;
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
    float *wm = res, *wl = res + kWarps * 8, *wa = res + 2 * kWarps * 8 + warp * G * kHeadDim;
    if (g == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            wm[warp * 8 + 2 * t + j] = cs.l[j] > 0.f ? cs.m[j] : -INFINITY;
            wl[warp * 8 + 2 * t + j] = cs.l[j];
        }
    }
    const float up = 1.f / vinv;                     // a power of two
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int head = 2 * t + (e & 1), ch = 32 * c + 4 * g + 2 * j + (e >> 1);
                if (head < G) wa[head * kHeadDim + ch] = acc[c][j][e] * (e >> 1 ? 1048576.f : 16777216.f) * up + zs[c * NG / 4][e & 1];
            }
}

// ---- the BF16 rows: [0, min(sink, T)) and [hist_end, T), 16-token tiles dealt out to the warps -----
template <int G, bool MASS>
__device__ __forceinline__ void window_warp(const Attn4Args &a, int b, int h, int T, int he, int warp, int lane, float *res) {
    const int g = lane >> 2, t = lane & 3, sh = a.page_shift;
    const int n0 = min(a.sink, T), lo1 = max(he, n0);
    const int sink_tiles = (n0 + 15) / 16, rec0 = lo1 / 16, tiles = sink_tiles + (lo1 < T ? (T + 15) / 16 - rec0 : 0);
    const int32_t *pt = a.bpt + (size_t)b * a.max_pages;
    uint4 bq[4];
    const uint16_t *qr = a.q + ((size_t)b * a.n_kv * G + h * G + (g < G ? g : 0)) * kHeadDim + 8 * t;
#pragma unroll
    for (int i = 0; i < 4; ++i) bq[i] = g < G ? *reinterpret_cast<const uint4 *>(qr + 32 * i) : make_uint4(0, 0, 0, 0);
    ColState cs;
    cs.m[0] = cs.m[1] = kNone;
    cs.l[0] = cs.l[1] = 0.f;
    if (MASS) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float l = 2 * t + j < G ? a.lse[(size_t)b * a.n_kv * G + h * G + 2 * t + j] : -INFINITY;
            cs.m[j] = l == -INFINITY ? INFINITY : l * kLog2e;
        }
    }
    float acc[G][4];                                 // lane: channels 4 lane .. 4 lane + 3
#pragma unroll
    for (int hh = 0; hh < G; ++hh)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[hh][e] = 0.f;

    int pages = -1;                                  // lane j: page of the warp's tile j of this batch of 32
    for (int k = warp, j = 0; k < tiles; k += kWarps, ++j) {
        auto tile_pos = [&](int kk) { return (kk < sink_tiles ? kk : rec0 + kk - sink_tiles) * 16; };
        if ((j & 31) == 0) {
            const int kk = k + kWarps * lane;
            pages = kk < tiles ? pt[tile_pos(kk) >> sh] : -1;
            // the rows of the first few of them start on their way to L2: a 128-byte line a lane, keys then values
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int pg = __shfl_sync(0xffffffffu, pages, u), kk2 = k + kWarps * u;
                if (kk2 < tiles && (uint32_t)pg < (uint32_t)a.bf.n_pages) {
                    const size_t row = ((size_t)pg << sh) + (tile_pos(kk2) & ((1 << sh) - 1)) + (lane >> 1);
                    const size_t at = (row * a.n_kv + h) * kHeadDim + 64 * (lane & 1);
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.bf.k + at));
                    if (!MASS) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.bf.v + at));
                }
            }
        }
        const bool in_sink = k < sink_tiles;
        const int p0 = tile_pos(k);
        const int lo = in_sink ? 0 : lo1, hi = in_sink ? n0 : T;
        const int page = __shfl_sync(0xffffffffu, pages, j & 31);
        if ((uint32_t)page >= (uint32_t)a.bf.n_pages) {
            if (lane == 0) flag_status(a.status, OSCAR_DEV_BAD_BF16_PAGE);
            continue;
        }
        const size_t row0 = ((size_t)page << sh) + (p0 & ((1 << sh) - 1));
        uint4 kx[2][4];
        uint2 vx[16];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool in = p0 + 8 * r + g >= lo && p0 + 8 * r + g < hi;
            const uint4 *src = reinterpret_cast<const uint4 *>(a.bf.k + ((row0 + 8 * r + g) * a.n_kv + h) * kHeadDim) + t;
#pragma unroll
            for (int i = 0; i < 4; ++i) kx[r][i] = in ? src[4 * i] : make_uint4(0, 0, 0, 0);
        }
        if (!MASS) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
                vx[r] = p0 + r >= lo && p0 + r < hi
                            ? reinterpret_cast<const uint2 *>(a.bf.v + ((row0 + r) * a.n_kv + h) * kHeadDim)[lane]
                            : make_uint2(0, 0);
        }
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mma16816_bf16(d, kx[0][i].x, kx[1][i].x, kx[0][i].y, kx[1][i].y, bq[i].x, bq[i].y);
            mma16816_bf16(d, kx[0][i].z, kx[1][i].z, kx[0][i].w, kx[1][i].w, bq[i].z, bq[i].w);
        }
        float s[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool in = p0 + 8 * r + g >= lo && p0 + 8 * r + g < hi;
#pragma unroll
            for (int j = 0; j < 2; ++j) s[r][j] = in ? d[2 * r + j] * a.scale2 : -INFINITY;
        }
        if (MASS) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = ex2_approx(s[r][0] - cs.m[0]) + ex2_approx(s[r][1] - cs.m[1]);
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                const int p = p0 + 8 * r + g;
                if (t == 0 && p >= lo && p < hi) atomicAdd(a.mass + (((size_t)b * a.n_kv + h) * a.max_pages << sh) + p, x);
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
#pragma unroll
        for (int hh = 0; hh < G; ++hh) {
            const float f = __shfl_sync(0xffffffffu, al[hh & 1], hh >> 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[hh][e] *= f;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float p = __shfl_sync(0xffffffffu, pr[r >> 3][hh & 1], 4 * (r & 7) + (hh >> 1));
                acc[hh][0] = fmaf(p, lo16(vx[r].x), acc[hh][0]);
                acc[hh][1] = fmaf(p, hi16(vx[r].x), acc[hh][1]);
                acc[hh][2] = fmaf(p, lo16(vx[r].y), acc[hh][2]);
                acc[hh][3] = fmaf(p, hi16(vx[r].y), acc[hh][3]);
            }
        }
    }
    if (MASS) return;
    cs.l[0] = col_sum(cs.l[0]);
    cs.l[1] = col_sum(cs.l[1]);
    float *wm = res, *wl = res + kWarps * 8, *wa = res + 2 * kWarps * 8 + warp * G * kHeadDim;
    if (g == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            wm[warp * 8 + 2 * t + j] = cs.l[j] > 0.f ? cs.m[j] : -INFINITY;
            wl[warp * 8 + 2 * t + j] = cs.l[j];
        }
    }
#pragma unroll
    for (int hh = 0; hh < G; ++hh)
        *reinterpret_cast<float4 *>(wa + hh * kHeadDim + 4 * lane) = make_float4(acc[hh][0], acc[hh][1], acc[hh][2], acc[hh][3]);
}

// The merge of all S + 1 slots of one kv head's G query heads, in oscar_merge's order and arithmetic.
// The accumulator rows come through shared memory, as many slots at a time as fit, all their 16-byte
// copies in flight at once and under way while the weights are formed.
template <int G>
__device__ __forceinline__ void merge_head(const Attn4Args &a, int b, int h, float *scratch, int scratch_bytes) {
    const int S1 = a.out.S + 1;
    const size_t row0 = ((size_t)b * a.n_kv * G + h * G) * S1;
    float *ws = scratch, *ls = scratch + G * S1, *ms = ls + G * S1;
    float *rows = scratch + ((2 * G * S1 + G + 3) & ~3);
    const int chunk = min(S1, (scratch_bytes - (int)((rows - scratch) * 4)) / (G * kHeadDim * 4));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto load = [&](int s0) {                          // slots [s0, s0 + chunk) of every head: [head][slot][128]
        const int n = min(chunk, S1 - s0);
        for (int e = threadIdx.x; e < G * n * 32; e += kThreads) {
            const int hh = e / (n * 32), r = e - hh * n * 32;
            cp_async16(saddr(rows + (size_t)hh * chunk * kHeadDim) + r * 16,
                       a.out.acc + (row0 + (size_t)hh * S1 + s0) * kHeadDim + r * 4);
        }
    };
    load(0);
    for (int i = threadIdx.x; i < G * S1; i += kThreads) {
        ls[i] = __ldcg(a.out.l + row0 + i);
        ws[i] = __ldcg(a.out.m + row0 + i);
    }
    __syncthreads();
    if (warp < G) {
        float M = -INFINITY;
        for (int i = lane; i < S1; i += 32)
            if (ls[warp * S1 + i] > 0.f) M = fmaxf(M, ws[warp * S1 + i]);
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (lane == 0) ms[warp] = M;
        for (int i = lane; i < S1; i += 32)
            ws[warp * S1 + i] = ls[warp * S1 + i] > 0.f ? exp2_taylor(__fsub_rn(ws[warp * S1 + i], M)) : 0.f;
    }
    constexpr int kPart = G * kHeadDim / kThreads > 0 ? G * kHeadDim / kThreads : 1;
    float L[kPart], A[kPart];
#pragma unroll
    for (int u = 0; u < kPart; ++u) L[u] = A[u] = 0.f;
    for (int s0 = 0; s0 < S1; s0 += chunk) {
        if (s0 > 0) {
            __syncthreads();                           // the previous chunk is consumed
            load(s0);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        const int n = min(chunk, S1 - s0);
#pragma unroll
        for (int u = 0; u < kPart; ++u) {
            const int e = threadIdx.x + u * kThreads, hh = e / kHeadDim, d = e % kHeadDim;
            if (hh >= G) continue;
            const float *x = rows + (size_t)hh * chunk * kHeadDim + d, *w = ws + hh * S1 + s0, *l = ls + hh * S1 + s0;
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                const bool on = l[i] > 0.f;
                L[u] = on ? __fmaf_rn(l[i], w[i], L[u]) : L[u];
                A[u] = on ? __fmaf_rn(x[i * kHeadDim], w[i], A[u]) : A[u];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kPart; ++u) {
        const int e = threadIdx.x + u * kThreads, hh = e / kHeadDim, d = e % kHeadDim;
        if (hh >= G) continue;
        const bool on = L[u] > 0.f;
        const float r = on ? __fdiv_rn(A[u], L[u]) : 0.f;
        const size_t orow = (size_t)b * a.n_kv * G + h * G + hh;
        if (a.of) a.of[orow * kHeadDim + d] = r;
        if (a.o) a.o[orow * kHeadDim + d] = f32_to_bf16_rn(r);
        if (a.o_lse && d == 0) a.o_lse[orow] = on ? (ms[hh] + log2f(L[u])) * 0.6931471805599453f : -INFINITY;
    }
}

// grid (S + 1, Hkv, batch): x = 0 the BF16 rows (slot S), x > 0 history split x - 1.
template <int G, int NG, bool MASS>
__global__ void __launch_bounds__(kThreads, 2)
    attn4_kernel(Attn4Args a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using R = Ring<NG, MASS>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[kWarps * R::n];
    __shared__ int last;
    uint8_t *smem = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
    const int h = blockIdx.y, b = blockIdx.z, S = a.out.S, slot = blockIdx.x == 0 ? S : (int)blockIdx.x - 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < kWarps * R::n) mbar_init(saddr(&bars[threadIdx.x]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    int T, he;
    read_lengths(a.seq_len, a.hist_end, b, a.sink, a.max_pages << a.page_shift, a.status, T, he);
    float *res = reinterpret_cast<float *>(smem);
    if (slot == S)
        window_warp<G, MASS>(a, b, h, T, he, warp, lane, res);
    else
        history_warp<G, NG, MASS>(a, &tmk, &tmv, smem + warp * R::n * R::stride, saddr(&bars[warp * R::n]), b, h, slot, he, warp,
                                  lane, res);
    if (MASS) return;
    __syncthreads();
    const float *wm = res, *wl = res + kWarps * 8, *wa = res + 2 * kWarps * 8;
    for (int e = threadIdx.x; e < G * kHeadDim; e += kThreads) {
        const int hh = e / kHeadDim, d = e % kHeadDim;
        float M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * 8 + hh]);
        if (M != -INFINITY) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2f(wm[w * 8 + hh] - M);
                L = fmaf(wl[w * 8 + hh], f, L);
                if (f > 0.f) A = fmaf(wa[(w * G + hh) * kHeadDim + d], f, A);
            }
        }
        const size_t row = ((size_t)b * a.n_kv * G + h * G + hh) * (S + 1) + slot;
        a.out.acc[row * kHeadDim + d] = A;
        if (d == 0) {
            a.out.m[row] = M;
            a.out.l[row] = L;
        }
    }
    if (!a.counters) return;
    __threadfence();                                  // this thread's part of the slot, before the count
    __syncthreads();
    if (threadIdx.x == 0) {
        int32_t *c = a.counters + (size_t)b * a.n_kv + h;
        last = atomicAdd(c, 1) == S;
        if (last) *c = 0;
        __threadfence();
    }
    __syncthreads();
    if (last) merge_head<G>(a, b, h, res, a.smem_bytes);
}

bool rows_tensor_map(CUtensorMap *tm, const uint8_t *base, long long rows, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {kRow4, (cuuint64_t)rows}, strides[1] = {kRow4};
    const cuuint32_t box[2] = {kRow4, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int G, int NG, bool MASS>
cudaError_t launch_one(Attn4Args a, const CUtensorMap &tmk, const CUtensorMap &tmv, dim3 grid, cudaStream_t st) {
    // the merge: weights of every slot, and room for one slot's rows at least
    const int merge = (((2 * G * (a.out.S + 1) + G + 3) & ~3) + G * kHeadDim) * 4, combine = (2 * kWarps * 8 + kWarps * G * kHeadDim) * 4;
    int smem = Ring<NG, MASS>::total;
    if (!MASS && smem < combine) smem = combine;
    if (!MASS && a.counters && smem < merge) smem = merge;
    a.smem_bytes = smem;
    smem += 1024;
    auto kern = attn4_kernel<G, NG, MASS>;
    if (cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(kern), smem)) return e;
    kern<<<grid, kThreads, smem, st>>>(a, tmk, tmv);
    return cudaGetLastError();
}

template <int G, bool MASS>
cudaError_t launch_group(const Attn4Args &a, int group, const CUtensorMap &tmk, const CUtensorMap &tmv, dim3 grid, cudaStream_t st) {
    switch (group) {
        case 32: return launch_one<G, 4, MASS>(a, tmk, tmv, grid, st);
        case 64: return launch_one<G, 2, MASS>(a, tmk, tmv, grid, st);
        default: return launch_one<G, 1, MASS>(a, tmk, tmv, grid, st);
    }
}

template <bool MASS>
cudaError_t launch(const oscar_layout_t &L, const Attn4Input &in, Attn4Args a, int batch, cudaStream_t st) {
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
    const dim3 grid(a.out.S + 1, L.n_kv_heads, batch);
    switch (L.gqa) {
        case 1: return launch_group<1, MASS>(a, L.group, tmk, tmv, grid, st);
        case 2: return launch_group<2, MASS>(a, L.group, tmk, tmv, grid, st);
        case 4: return launch_group<4, MASS>(a, L.group, tmk, tmv, grid, st);
        default: return launch_group<8, MASS>(a, L.group, tmk, tmv, grid, st);
    }
}

}  // namespace

// Two CTAs an SM: one wave of them when the batch's heads fit, else about four, so that requests of
// different lengths finish evenly.  At least 8 blocks of 32 tokens (one a warp) for each split.
int suggest_splits4(const oscar_layout_t &L, int batch, int max_hist, int sm_count) {
    const long long per = (long long)batch * L.n_kv_heads, slots = 2LL * sm_count;
    long long want = per * 8 <= slots ? slots / per - 1 : (4 * slots + per - 1) / per;
    const long long most = ((long long)max_hist + kWarps * kBlock - 1) / (kWarps * kBlock);
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
    if (cudaError_t e = launch<false>(L, in, a, batch, st)) return e;
    return merge && !counters ? launch_merge(L, out, nullptr, batch, o, of, lse, st) : cudaSuccess;
}

cudaError_t launch_mass4(const oscar_layout_t &L, const Attn4Input &in, int batch, const float *lse, float *mass,
                         int32_t *status, cudaStream_t st) {
    Attn4Args a{};
    a.out.S = suggest_splits4(L, batch, in.max_pages * L.page_size, 152);
    a.lse = lse;
    a.mass = mass;
    a.status = status;
    return launch<true>(L, in, a, batch, st);
}

}  // namespace oscar
