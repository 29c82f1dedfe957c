// Attention of a tree of drafted tokens over an INT4 history with BF16 sink and recent rows: tiles of 16 query rows
// (node, query head of one kv head) on mma.sync, the BF16 rows with the nodes' mask, and the merge of the splits.
//
// As for one token (attn_int4.cuh), with a row's codes n, scale s and zero z per channel group, a logit is
// sm (s sum_c q_c n_c + z sum_c q_c), and the products meet the codes as f16 subnormals.  Here the 16 query rows are the A
// operand of m16n8k16 and eight keys the B operand, so that a pair of logit accumulators is the A operand of the value product
// as it lies (no movement between lanes), and a code is unpacked once for 16 rows.  The value product is
//   sum_t p_t v_t = sum_t (p_t s_t) (n_t - 8) + sum_t p_t (z_t + 8 s_t)
// with centred codes, normal f16 numbers at one operation more a pair: uncentred the two sums cancel most of each other, which
// would ask for p s in two parts and for sums that are not truncated (the accumulators of mma.sync are).  p s is one f16
// number, 2^-11 relative.  p = 2^(logit - M) with a reference M per row that is raised, in whole steps, whenever a p s passes 2^15
// (then brought to about 2^8) or p passes 2^100: the largest p s so far, not the largest p, sits near the top of f16's range.
//
// A CTA takes (split, 16 query rows, kv head, request); each of its W warps takes every W-th block of 32 tokens through a ring
// of bulk tensor copies of its own, and they join at the end.  W is 12 where the launch has about a CTA an SM, else 8, two CTAs
// an SM (group 128; smaller groups need the registers of one).  Slot S of the partials is the BF16 rows': the last CTA of a
// row tile, whose warps take 16 positions at a time straight from global memory.  With one split, a CTA takes both, one after the
// other, and writes the result: no partials, no merge.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "merge_math.cuh"
#include "tma.cuh"
#include "tree_window.cuh"

namespace oscar {
namespace {

constexpr int kWide = kSms + 8;                  // CTAs of a launch up to which each gets an SM (or nearly)
constexpr float kMostP = 0x1p100f;               // of the sum of a lane's p in a block
constexpr float kNewW = 8.f, kNewP = 80.f;       // a new reference brings p·s to 2^8 at most, p to 2^80

template <int NG, int W>
struct Ring {
    static constexpr int bytes = 4096 + kBlock4 * NG * 8;
    static constexpr int stride = (bytes + 511) & ~511;
    static constexpr int n = NG == 4 ? 2 : 3;                    // as many as leave room for two CTAs on an SM
    static constexpr int total = W * n * stride;
};

__device__ __forceinline__ void tma_rows(uint32_t dst, const void *tmap, int row, uint32_t bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3}], [%4], %5;"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(row), "r"(bar), "l"(pol)
        : "memory");
}

// ---- the history -----------------------------------------------------------------------------------
template <int NG, int W>
__device__ __forceinline__ void history_warp(const TreeArgs &a, const CUtensorMap *tmk, const CUtensorMap *tmv, uint8_t *ring, uint32_t bars,
                                             const TreeRequest &rq, int b, int h, int row0, int rows, int split, uint4 *frag, int warp, int lane, Rows &x) {
    using R = Ring<NG, W>;
    const int t = lane & 3, sh = a.page_shift, S = a.part.S, he = rq.he;
    const int first = a.sink / kBlock4, nb = he > a.sink ? (he + kBlock4 - 1) / kBlock4 - first : 0;
    const int lo = first + (int)((long long)split * nb / S) + warp, hi = first + (int)((long long)(split + 1) * nb / S);
    const int n = lo < hi ? (hi - lo + W - 1) / W : 0;        // blocks lo, lo + W, ...
    const int32_t *pt = a.ipt + (size_t)b * a.max_pages;
    const uint64_t pol = l2_evict_first_policy();

    int pg0 = -1, pg1 = -1;        // lane j: pages of the two 16-token halves of block lo + W (batch + j)
    uint32_t ok = 0;               // two bits per stage: halves that were loaded
    auto issue = [&](int i, int st) {
        if ((i & 31) == 0) {
            const int p = (lo + W * (i + lane)) * kBlock4;
            pg0 = pg1 = -1;
            if (i + lane < n) {
                const bool in0 = p + 16 > a.sink && p < he, in1 = p + kBlock4 > a.sink && p + 16 < he;
                if (in0) pg0 = pt[p >> sh];
                if (in1) pg1 = pt[(p + 16) >> sh];
                if ((in0 && (uint32_t)pg0 >= (uint32_t)a.i4_pages) || (in1 && (uint32_t)pg1 >= (uint32_t)a.i4_pages))
                    flag_status(a.status, OSCAR_DEV_BAD_INT4_PAGE);
            }
        }
        const int a0 = __shfl_sync(0xffffffffu, pg0, i & 31), a1 = __shfl_sync(0xffffffffu, pg1, i & 31);
        const bool ok0 = (uint32_t)a0 < (uint32_t)a.i4_pages, ok1 = (uint32_t)a1 < (uint32_t)a.i4_pages;
        ok = (ok & ~(3u << (2 * st))) | ((ok0 ? 1u : 0u) | (ok1 ? 2u : 0u)) << (2 * st);
        if (lane == 0) {
            const int p = (lo + W * i) * kBlock4;
            const uint32_t dst = saddr(ring + st * R::stride), bar = bars + 8 * st;
            // pages of 32 or more: one box of 32 rows; pages of 16: a box a half
            const int box = sh >= 5 ? kBlock4 : 16;
            const bool l0 = sh >= 5 ? ok0 || ok1 : ok0, l1 = sh >= 5 ? false : ok1;
            mbar_arrive_expect_tx(bar, (uint32_t)(l0 + l1) * box * (R::bytes / kBlock4));
            const int page[2] = {ok0 ? a0 : a1, a1};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!(half ? l1 : l0)) continue;
                const int row = ((page[half] * a.n_kv + h) << sh) + ((p + 16 * half) & ((1 << sh) - 1));
                tma_rows(dst + half * 1024, tmk, row, bar, pol);
                tma_rows(dst + 2048 + half * 1024, tmv, row, bar, pol);
                tma_load_1d(dst + 4096 + half * 16 * NG * 8, a.sz + (size_t)row * NG * 4, (uint32_t)box * NG * 8, bar, pol);
            }
        }
    };
    for (int i = 0; i < R::n && i < n; ++i) issue(i, i);

    // A operand of the logits, for all warps (fragment 2 i + e of lane l at 32 (2 i + e) + l): channels 32 i + 8 t .. of chunk i,
    // the odd nibbles' against 1/16 of the query; fac undoes the scalings, qz is the zero's factor before it, per row and group.
    float fac[2], qz[NG][2];
    {
        float mul[2], qs[2][NG];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float mx = 0.f;
#pragma unroll
            for (int k = 0; k < NG; ++k) qs[r][k] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 q = query_piece(a, rq, h, row0, rows, r, i, lane);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mx = fmaxf(mx, fmaxf(fabsf(lo16(w[e])), fabsf(hi16(w[e]))));
                    qs[r][i * NG / 4] += lo16(w[e]) + hi16(w[e]);
                }
            }
            mx = row_max(mx);
            const int ex = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 117);      // |q| < 2^(ex + 1)
            mul[r] = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
            fac[r] = a.scale2 * __uint_as_float((uint32_t)(10 + ex + 127) << 23);              // 2^24 / mul
#pragma unroll
            for (int k = 0; k < NG; ++k) qz[k][r] = row_sum(qs[r][k]) * (mul[r] * 0x1p-24f);   // (fac's units)
        }
        for (int i = warp; i < 4; i += W) {
            uint32_t f[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint4 w = query_piece(a, rq, h, row0, rows, r, i, lane);
                const float m0 = mul[r], m1 = mul[r] * 0.0625f;
                f[0][r] = pack_h2(lo16(w.x) * m0, lo16(w.z) * m0);
                f[0][2 + r] = pack_h2(hi16(w.x) * m1, hi16(w.z) * m1);
                f[1][r] = pack_h2(lo16(w.y) * m0, lo16(w.w) * m0);
                f[1][2 + r] = pack_h2(hi16(w.y) * m1, hi16(w.w) * m1);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) frag[64 * i + 32 * e + lane] = make_uint4(f[e][0], f[e][1], f[e][2], f[e][3]);
        }
    }
    __syncthreads();
    for (int i = 0, st = 0, phase = 0; i < n; ++i) {
        if (!mbar_wait(bars + 8 * st, phase)) {
            if (lane == 0) flag_status(a.status, OSCAR_DEV_WAIT_TIMEOUT);
            // the copies still under way land before this memory is used again
            for (int k = i; k < i + R::n && k < n; ++k) mbar_wait(bars + 8 * (k % R::n), (k / R::n) & 1);
            break;
        }
        const uint8_t *stage = ring + st * R::stride;
        const uint32_t sb = saddr(stage);
        const int p0 = (lo + W * i) * kBlock4;
        const uint32_t okb = (ok >> (2 * st)) & 3u;
        const bool full = okb == 3u && p0 >= a.sink && p0 + kBlock4 <= he;

        f2 s[4][2];                                  // keys 8 u + 2 t, + 1 of row g + 8 r: the logits before fac
        uint32_t vw[4][2][NG];                       // value scale | zero of those keys
        {
            uint32_t w[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int row = 8 * u + (lane & 7);
                ldmatrix_x4(sb + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4), w[u][0], w[u][1], w[u][2], w[u][3]);
            }
#pragma unroll
            for (int k = 0; k < NG; ++k) {
                float d[4][4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[u][e] = 0.f;
#pragma unroll
                for (int c = 4 * k / NG; c < 4 * (k + 1) / NG; ++c) {
                    const uint4 x0 = frag[64 * c + lane], x1 = frag[64 * c + 32 + lane];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t y = w[u][c], y8 = y >> 8;
                        mma16816_nv(d[u], x0.x, x0.y, x0.z, x0.w, y & kM0, y & kM1);
                        mma16816_nv(d[u], x1.x, x1.y, x1.z, x1.w, y8 & kM0, y8 & kM1);
                    }
                }
                // sum over groups of ks d + kz qz
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint2 *rec = reinterpret_cast<const uint2 *>(stage + 4096) + (8 * u + 2 * t) * NG + k;
                    const uint2 z0 = rec[0], z1 = rec[NG];
                    vw[u][0][k] = z0.y;
                    vw[u][1][k] = z1.y;
                    const f2 ks = pair(lo16(z0.x), lo16(z1.x)), kz = pair(hi16(z0.x), hi16(z1.x));
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const f2 qk = pair(qz[k][r], qz[k][r]);
                        s[u][r] = fma2(ks, pair(d[u][2 * r], d[u][2 * r + 1]), k ? fma2(kz, qk, s[u][r]) : mul2(kz, qk));
                    }
                }
            }
        }
        uint32_t usable = 0xffu;                     // bit 2 u + e
        if (!full) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int p = p0 + 8 * u + 2 * t + e;
                    if (p < a.sink || p >= he || !((okb >> (u >> 1)) & 1u)) {
                        usable &= ~(1u << (2 * u + e));
#pragma unroll
                        for (int k = 0; k < NG; ++k) vw[u][e][k] = 0u;
                    }
                }
        }
        f2 p[4][2];                                  // 2^(logit - M)
        float l[2];
        for (int again = 0;; ++again) {              // once, or twice where a reference was due
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const f2 fr = pair(fac[r], fac[r]), mr = pair(-x.m[r], -x.m[r]);
                f2 l2 = 0ull;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float e0, e1;
                    unpair(fma2(s[u][r], fr, mr), e0, e1);
                    if (!full) {
                        if (!((usable >> (2 * u)) & 1)) e0 = -INFINITY;
                        if (!((usable >> (2 * u + 1)) & 1)) e1 = -INFINITY;
                    }
                    p[u][r] = pair(ex2_approx(e0), ex2_approx(e1));
                    l2 = add2(l2, p[u][r]);
                }
                float l0, l1;
                unpair(l2, l0, l1);
                l[r] = l0 + l1;
            }
            // looked at closer where the rows' sums with the largest of the lane's scales would pass f16's range, together or not
            __nv_bfloat162 v2 = as_bf2(vw[0][0][0]);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int k = 0; k < NG; ++k) v2 = __hmax2(v2, as_bf2(vw[u][e][k]));        // scales in the low halves
            const float both = fmaxf(l[0], l[1]);
            if (!__any_sync(0xffffffffu, both * __low2float(v2) >= 0x1p15f || both >= kMostP) || again) break;
#pragma unroll 1
            for (int r = 0; r < 2; ++r) {
                float top = -INFINITY, topw = -INFINITY;                   // largest logit, largest logit + log2 s
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float e[2];
                    unpair(mul2(r ? s[u][1] : s[u][0], pair(r ? fac[1] : fac[0], r ? fac[1] : fac[0])), e[0], e[1]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (!((usable >> (2 * u + j)) & 1)) continue;
                        top = fmaxf(top, e[j]);
#pragma unroll
                        for (int k = 0; k < NG; ++k) topw = fmaxf(topw, e[j] + __log2f(lo16(vw[u][j][k])));
                    }
                }
                top = row_max(top);
                topw = row_max(topw);
                const float M = r ? x.m[1] : x.m[0];
                float to = M;
                // kept where it will do: the check above is for sums of eight and scales apart
                if (topw - M >= 11.9f || top - M >= 90.f) {
                    const float want = ceilf(fmaxf(topw - kNewW, top - kNewP));
                    to = M == kNone ? want : fmaxf(M, want);
                }
                const int down = __float2int_rn(M - to);                   // (whole, or far below)
                const float f = down < -126 ? 0.f : __uint_as_float((uint32_t)(down + 127) << 23);
                if (r) x.m[1] = to;
                else x.m[0] = to;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float fq = q == r ? f : 1.f;
                    x.l[q] *= fq;
#pragma unroll
                    for (int k = 0; k < NG; ++k) x.z[k][q] *= fq;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) x.out[c][j][2 * q + e] *= fq;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) x.l[r] += l[r];
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            f2 z2[2] = {0ull, 0ull};
#pragma unroll
            for (int u = 0; u < 4; ++u) {            // zero of the centred codes
                const f2 vs = pair(lo16(vw[u][0][k]), lo16(vw[u][1][k])), zc = fma2(pair(8.f, 8.f), vs, pair(hi16(vw[u][0][k]), hi16(vw[u][1][k])));
#pragma unroll
                for (int r = 0; r < 2; ++r) z2[r] = fma2(p[u][r], zc, z2[r]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float z0, z1;
                unpair(z2[r], z0, z1);
                x.z[k][r] += z0 + z1;
            }
        }
        uint32_t ap[2][4], vc[2][4];
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
            if (c * NG % 4 == 0)                     // a new group
#pragma unroll
                for (int tl = 0; tl < 2; ++tl)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int u = 2 * tl + (v >> 1), r = v & 1;
                        float w0, w1;
                        unpair(mul2(p[u][r], pair(lo16(vw[u][0][k]), lo16(vw[u][1][k]))), w0, w1);
                        ap[tl][v] = pack_h2(w0, w1);
                    }
#pragma unroll
            for (int tl = 0; tl < 2; ++tl) {
                const uint32_t y0 = vc[tl][2 * (c & 1)], y1 = vc[tl][2 * (c & 1) + 1], z0 = y0 >> 8, z1 = y1 >> 8;
                mma16816_nv(x.out[c][0], ap[tl][0], ap[tl][1], ap[tl][2], ap[tl][3], centred_low(y0), centred_low(y1));
                mma16816_nv(x.out[c][1], ap[tl][0], ap[tl][1], ap[tl][2], ap[tl][3], centred_high(y0), centred_high(y1));
                mma16816_nv(x.out[c][2], ap[tl][0], ap[tl][1], ap[tl][2], ap[tl][3], centred_low(z0), centred_low(z1));
                mma16816_nv(x.out[c][3], ap[tl][0], ap[tl][1], ap[tl][2], ap[tl][3], centred_high(z0), centred_high(z1));
            }
        }
        __syncwarp();
        if (i + R::n < n) issue(i + R::n, st);
        if (++st == R::n) {
            st = 0;
            phase ^= 1;
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            const float z = row_sum(x.z[k][r]);
#pragma unroll
            for (int c = k * 4 / NG; c < (k + 1) * 4 / NG; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) x.out[c][j][2 * r + e] += z;
        }
    }
}

// grid (slots x row tiles, Hkv, batch), slots 0 .. S, the row tiles of a slot next to each other: they read the same rows; S = 1:
// the row tiles, all of it by one CTA each.
template <int NG, int W>
__global__ void __launch_bounds__(W * 32, NG == 1 && W == 8 ? 2 : 1)
    tree_kernel(TreeArgs a, int tiles, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using R = Ring<NG, W>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[W * R::n];
    uint8_t *smem = smem_raw + ((512u - (saddr(smem_raw) & 511u)) & 511u);          // the swizzle pattern repeats every 512 bytes
    uint4 *frag = reinterpret_cast<uint4 *>(smem + R::total);
    const int slot = blockIdx.x / tiles, row0 = blockIdx.x % tiles * kTile, h = blockIdx.y, b = blockIdx.z, S = a.part.S;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
        for (int i = 0; i < R::n; ++i) mbar_init(saddr(&bars[warp * R::n + i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    const bool whole = S == 1;
    pdl_wait();
    const TreeRequest rq(a, b);
    const int rows = min(kTile, rq.n * a.G - row0);
    if (rows <= 0) return;
    Rows x;
    clear(x);
    if (slot < S)
        history_warp<NG, W>(a, &tmk, &tmv, smem + warp * R::n * R::stride, saddr(&bars[warp * R::n]), rq, b, h, row0, rows, slot, frag, warp, lane, x);
    if (whole) __syncthreads();                      // frag is read
    if (slot == S || whole) window_warp<W>(a, rq, b, h, row0, rows, frag, reinterpret_cast<uint4 *>(smem + warp * R::n * R::stride), 0, warp, lane, x);
    __syncthreads();                                 // every warp is done with its ring: results take its place
    join_warps<W>(a, rq, h, row0, rows, slot, whole, smem, 0, threadIdx.x, warp, lane, x);
}

// A warp takes a (node row, query head): its slots in ascending order, four channels a lane, eight slots on their way.
__global__ void __launch_bounds__(128) tree_merge_kernel(TreeArgs a) {
    pdl_wait();
    const TreeRequest rq(a, blockIdx.y);
    const int Hq = a.n_kv * a.G, lane = threadIdx.x & 31, S1 = a.part.S + 1;
    const int item = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (item >= rq.n * Hq) return;
    const size_t orow = (size_t)rq.first * Hq + item, row0 = orow * S1;
    const float4 *acc = reinterpret_cast<const float4 *>(a.part.acc + row0 * kHeadDim) + lane;
    float M = -INFINITY;
    for (int i = lane; i < S1; i += 32) M = fmaxf(M, a.part.m[row0 + i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < S1; s0 += 32) {
        const bool in = s0 + lane < S1;
        const float li = in ? a.part.l[row0 + s0 + lane] : 0.f, mi = in ? a.part.m[row0 + s0 + lane] : -INFINITY;
        const float wi = mi != mi ? mi : mi != -INFINITY ? exp2_taylor(__fsub_rn(mi, M)) : 0.f;
        for (int i0 = 0; i0 < 32 && s0 + i0 < S1; i0 += 8) {
            float4 y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (s0 + i0 + i < S1) y[i] = __ldcg(acc + (size_t)(s0 + i0 + i) * (kHeadDim / 4));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float l = __shfl_sync(0xffffffffu, li, (i0 + i) & 31), w = __shfl_sync(0xffffffffu, wi, (i0 + i) & 31);
                if (s0 + i0 + i < S1 && w != 0.f) {
                    L = __fmaf_rn(l, w, L);
                    A = make_float4(__fmaf_rn(y[i].x, w, A.x), __fmaf_rn(y[i].y, w, A.y), __fmaf_rn(y[i].z, w, A.z), __fmaf_rn(y[i].w, w, A.w));
                }
            }
        }
    }
    const bool on = L > 0.f || L != L;
    const float o0 = on ? __fdiv_rn(A.x, L) : 0.f, o1 = on ? __fdiv_rn(A.y, L) : 0.f, o2 = on ? __fdiv_rn(A.z, L) : 0.f,
                o3 = on ? __fdiv_rn(A.w, L) : 0.f;
    *reinterpret_cast<uint2 *>(a.o + orow * kHeadDim + 4 * lane) = make_uint2(pack_b2(o0, o1), pack_b2(o2, o3));
    if (a.lse && lane == 0) a.lse[orow] = on ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
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

template <int NG, int W>
cudaError_t launch_rows(const TreeArgs &a, int tiles, const CUtensorMap &tmk, const CUtensorMap &tmv, int batch, cudaStream_t st) {
    const int smem = std::max(Ring<NG, W>::total + 4096, join_bytes<W>()) + 512;
    auto kern = tree_kernel<NG, W>;
    if (cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(kern), smem)) return e;
    return launch_ahead(kern, dim3((a.part.S == 1 ? 1 : a.part.S + 1) * tiles, a.n_kv, batch), W * 32, smem, st, a, tiles, tmk, tmv);
}

}  // namespace

// Which kernel takes the history: 128 query rows a CTA on tcgen05 (group 128), or 16 on mma.sync.  The former takes 8.2 ns a tile
// of 128 positions and 128 rows, the whole GPU, the latter 5.2 ns for 16 rows; the former's launches cost 7 us more, and its CTAs of
// the BF16 rows, one an SM, 0.1 us each beyond those that find an SM at once.  With 8 kv heads, tcgen05 and mma.sync, us: 32 rows,
// 1 x 100K 60 and 71, 1 x 4K 20 and 15, 64 x 4K 224 and 214, 64 x 8K 317 and 366, 128 x 2K 327 and 264; 64 rows, 16 ragged of 100K
// 735 and 1,069, 1 x 4K 23 and 18, 64 x 4K 319 and 409.
// tokens: the longest history's, one number for the splits and for the launch.  By the tables' width instead (128K), 8 nodes, 1 x 4K
// and 1 x 1K took what tcgen05 takes: 20 us for 15, 20 for 13.
static bool on_tcgen05(const oscar_layout_t &L, int batch, int max_nodes, long long tokens) {
    const long long rows = (long long)max_nodes * L.gqa, heads = (long long)batch * L.n_kv_heads, tiles = heads * (tokens / 128 + 1);
    const long long gain = tiles * (52 * ((rows + 15) / 16) - 82 * ((rows + 127) / 128));
    return L.group == 128 && rows > 16 && gain > 70000 + 1000 * std::max(0LL, heads * ((rows + 31) / 32) - kSms);
}

// On tcgen05: one CTA an SM in one wave that leaves some SMs to the BF16 rows, or, where splits would pass 16K positions, splits of 8K,
// which finish evenly (16 ragged of 100K, 64 rows: 858 us with one split, 735 with 12) and keep long sums short.  On mma.sync: one wave, the
// BF16 rows' CTAs among it, of 12 warps and one CTA an SM where that leaves three splits, else (and for groups of 32 and 64) of 8
// warps, two CTAs an SM (one); splits of 8K where they would pass 32K.  4 rows a kv head, us, 12 and 8 warps: 1 x 100K 40 and 50 (18
// splits), 64 x 4K 125 and 120 (one), 8 x 8K 43 and 42 (3), 16 ragged of 100K 420 and 442 (12).
int suggest_splits_tree(const oscar_layout_t &L, int batch, int max_nodes, int max_hist, int sm_count) {
    const bool tc = on_tcgen05(L, batch, max_nodes, max_hist);
    const long long rows = max_nodes * (long long)L.gqa, tile = tc ? 128 : kTile;
    const long long units = (long long)batch * L.n_kv_heads * ((rows + tile - 1) / tile);
    long long want = tc ? (sm_count - 8) / units : sm_count / units - 1;
    if (!tc && want < 3 && L.group == 128) want = 2LL * sm_count / units - 1;
    want = std::max(want, 1LL);
    if (max_hist > want * (tc ? 16384 : 32768)) want = std::max(want, std::min(max_hist / 8192LL, 12LL * sm_count / units));
    want = std::min(want, (max_hist + 511LL) / 512);
    return (int)std::max(1LL, std::min(want, 1024LL));
}

cudaError_t launch_tree_attention(const oscar_layout_t &L, const Attn4Input &in, const TreeInput &t, const int32_t *mask, int mask_words,
                                  int max_hist, int batch, PartialsView part, uint16_t *out, float *lse, int32_t *status, cudaStream_t st) {
    TreeArgs a{in.q, t, mask, mask_words, in.bf, in.bpt, in.i4.codes_k, in.i4.codes_v, in.i4.scale_zero, in.i4.n_pages, in.ipt, in.max_pages, page_shift(L), L.n_kv_heads, L.gqa,
               L.sink, in.seq_len, in.hist_end, in.sm_scale * kLog2e, part, out, lse, status};
    const int tiles = (t.max_nodes * L.gqa + kTile - 1) / kTile;
    if (on_tcgen05(L, batch, t.max_nodes, max_hist) && tree_tc_fits(a, t.max_nodes * L.gqa, batch)) {
        if (cudaError_t e = launch_tree_tc(a, t.max_nodes * L.gqa, batch, st)) return e;
    } else {
        CUtensorMap tmk, tmv;
        const long long rows = (long long)in.i4.n_pages * L.n_kv_heads * L.page_size;
        const int box = L.page_size < kBlock4 ? L.page_size : kBlock4;
        if (!rows_tensor_map(&tmk, in.i4.codes_k, rows, box) || !rows_tensor_map(&tmv, in.i4.codes_v, rows, box)) return cudaErrorInvalidValue;
        const bool wide = (long long)(part.S + 1) * tiles * L.n_kv_heads * batch <= kWide;
        cudaError_t e;
        switch (L.group) {
            case 32: e = launch_rows<4, 8>(a, tiles, tmk, tmv, batch, st); break;
            case 64: e = launch_rows<2, 8>(a, tiles, tmk, tmv, batch, st); break;
            default: e = wide ? launch_rows<1, 12>(a, tiles, tmk, tmv, batch, st) : launch_rows<1, 8>(a, tiles, tmk, tmv, batch, st);
        }
        if (e || part.S == 1) return e;
    }
    return launch_ahead(tree_merge_kernel, dim3((t.max_nodes * L.n_kv_heads * L.gqa + 3) / 4, batch), 128, 0, st, a);
}

}  // namespace oscar
