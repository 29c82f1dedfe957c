// New tokens into the BF16 cache: per-head RMS norm, rotary position and the paged write in one pass.
//
// y = x / sqrt(mean(x^2) + eps) * w over a head's 128 channels, then the rotation of the first
// rot_dim channels by the token's angles, (a, b) -> (a cos - b sin, b cos + a sin); fp32 throughout,
// one rounding to bf16.  Queries go to q_out, keys and values to their slots of the BF16 pool.
//
// Bound by HBM (a row is read and written once).  A head's row is 256 bytes: 16 lanes with 8 channels each
// (one 16-byte load and store a lane), so the sum of squares is a 4-step shuffle and a rotation partner is
// either in the lane (channels 2j, 2j+1) or rot_dim/16 lanes away.  A warp takes a run of row pairs of one
// token, reads the token's angles once, and keeps four rows a half-warp in flight: each row's registers
// are refilled as soon as it is computed.  Measured: 8,115 tokens of 32 query and 8 kv heads 43.7 us = 4.7 TB/s
// (latency: half the issue slots are used, 16 warps an SM); one token 2.7 us a call in a stream.

#include <cuda_bf16.h>

#include <algorithm>

#include "int4.cuh"
#include "ptx.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 8;

struct AppendArgs {
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    int n, n_q, n_kv;
    int per, runs;                 // row pairs of a warp, warps of a token
    const uint16_t *wq, *wk;
    float eps;
    const float *rope;
    int rope_rows, rot;
    Bf16PoolView pool;
    const int32_t *pt;
    int max_pages, page_shift, batch;
    const int32_t *req, *pos, *rope_pos;
    uint16_t *q_out;
    int32_t *status;
};

// packed fp32 pairs
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// the two bf16 of a word as an fp32 pair
__device__ __forceinline__ uint64_t widen(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ void widen8(uint4 w, uint64_t (&x)[4]) {
    x[0] = widen(w.x);
    x[1] = widen(w.y);
    x[2] = widen(w.z);
    x[3] = widen(w.w);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

constexpr int kAhead = 4;

template <bool PAIRS>
__global__ void __launch_bounds__(kWarps * 32, 2) append_kernel(AppendArgs a) {
    const int lane = threadIdx.x & 31, half = lane >> 4, hl = lane & 15;
    const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5);       // below 2^32: n * runs is (launch_append)
    const int i = (int)(w / (uint32_t)a.runs);
    pdl_wait();
    if (i >= a.n) return;
    const int rows = a.n_q + 2 * a.n_kv, pair0 = (int)(w - (uint32_t)i * a.runs) * a.per;
    const int pairs = min(a.per, (rows + 1) / 2 - pair0);
    const uint16_t *q = a.q + i * a.q_stride + 8 * hl, *k = a.k + i * a.k_stride - (long long)a.n_q * kHeadDim + 8 * hl;
    const uint16_t *v = a.v + i * a.v_stride - (long long)(a.n_q + a.n_kv) * kHeadDim + 8 * hl;
    auto load = [&](int j) {                       // row 2 (pair0 + j) + half
        const int r = 2 * (pair0 + j) + half;
        if (j >= pairs || r >= rows) return make_uint4(0, 0, 0, 0);
        return *reinterpret_cast<const uint4 *>((r < a.n_q ? q : r < a.n_q + a.n_kv ? k : v) + (long long)r * kHeadDim);
    };
    uint4 x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) x[u] = load(u);
    const int pos = a.pos[i], b = a.req[i];
    if (pos == -1) return;                                        // padding
    const int rp = a.rope_pos ? a.rope_pos[i] : pos;
    if (b < 0 || b >= a.batch || pos < 0 || (pos >> a.page_shift) >= a.max_pages ||
        (a.rope && (rp < 0 || rp >= a.rope_rows))) {
        if (lane == 0) flag_status(a.status, OSCAR_DEV_BAD_LENGTH);
        return;
    }
    const int page = a.pt[(size_t)b * a.max_pages + (pos >> a.page_shift)];

    // this lane's angles: pair 4 hl + e (channels 2j, 2j + 1), or those of channels 8 hl + e of either half
    const int rl = a.rot >> 4;                                    // lanes per rotated half
    const bool turns = a.rope && 8 * hl < a.rot;
    // channel pairs (8 hl + 2e, + 1) as fp32 pairs; what lanes that do not turn get of them is not used
    uint64_t cs[4], sn[4];
    {
        float c[8], z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            c[e] = 1.f;
            z[e] = 0.f;
        }
        if (turns) {
            const float *t = a.rope + (size_t)rp * kHeadDim + (PAIRS ? 4 * hl : 8 * (hl < rl ? hl : hl - rl));
#pragma unroll
            for (int e = 0; e < (PAIRS ? 4 : 8); e += 4) {
                const float4 cc = *reinterpret_cast<const float4 *>(t + e), ss = *reinterpret_cast<const float4 *>(t + 64 + e);
                c[e] = cc.x; c[e + 1] = cc.y; c[e + 2] = cc.z; c[e + 3] = cc.w;
                z[e] = ss.x; z[e + 1] = ss.y; z[e + 2] = ss.z; z[e + 3] = ss.w;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (PAIRS) {                                          // (a, b)·cos + (b, a)·(-sin, sin)
                cs[e] = pair(c[e], c[e]);
                sn[e] = pair(-z[e], z[e]);
            } else {
                const float sg = hl < rl ? -1.f : 1.f;
                cs[e] = pair(c[2 * e], c[2 * e + 1]);
                sn[e] = pair(sg * z[2 * e], sg * z[2 * e + 1]);
            }
        }
    }
    const int partner = (lane & 16) | (turns ? (hl < rl ? hl + rl : hl - rl) : hl);
    const bool page_ok = (uint32_t)page < (uint32_t)a.pool.n_pages;
    if (!page_ok && lane == 0) flag_status(a.status, OSCAR_DEV_BAD_BF16_PAGE);
    const long long slot = (((long long)(page_ok ? page : 0) << a.page_shift) + (pos & ((1 << a.page_shift) - 1))) * a.n_kv;
    uint16_t *qo = a.q_out + (size_t)i * a.n_q * kHeadDim + 8 * hl;
    uint16_t *ko = const_cast<uint16_t *>(a.pool.k) + (slot - a.n_q) * kHeadDim + 8 * hl;
    uint16_t *vo = const_cast<uint16_t *>(a.pool.v) + (slot - a.n_q - a.n_kv) * kHeadDim + 8 * hl;

    // Two row pairs at a time: their reductions, roots and shuffles overlap.
    const uint16_t *held = nullptr;                               // the norm weights now in wv
    uint64_t wv[4];
    for (int j0 = 0; j0 < pairs; j0 += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; u += 2) {
            const int r0 = 2 * (pair0 + j0 + u) + half;
            const uint4 raw[2] = {x[u], x[u + 1]};
            x[u] = load(j0 + u + kAhead);
            x[u + 1] = load(j0 + u + 1 + kAhead);
            if (j0 + u >= pairs) continue;                        // the whole warp
            const int in_warp = min(rows, 2 * (pair0 + pairs));   // rows from here on are another warp's, or none
            if (r0 - half >= a.n_q + a.n_kv) {                    // values: moved as they are
#pragma unroll
                for (int v2 = 0; v2 < 2; ++v2)
                    if (page_ok && r0 + 2 * v2 < in_warp) *reinterpret_cast<uint4 *>(vo + (long long)(r0 + 2 * v2) * kHeadDim) = raw[v2];
                continue;
            }
            uint64_t y[2][4];
            float ss[2];
#pragma unroll
            for (int v2 = 0; v2 < 2; ++v2) {
                widen8(raw[v2], y[v2]);
                uint64_t sq = mul2(y[v2][0], y[v2][0]);
#pragma unroll
                for (int e = 1; e < 4; ++e) sq = fma2(y[v2][e], y[v2][e], sq);
                float s0, s1;
                unpair(sq, s0, s1);
                ss[v2] = s0 + s1;
            }
#pragma unroll
            for (int o = 8; o; o >>= 1) {
                const float t0 = __shfl_xor_sync(0xffffffffu, ss[0], o), t1 = __shfl_xor_sync(0xffffffffu, ss[1], o);
                ss[0] += t0;
                ss[1] += t1;
            }
#pragma unroll
            for (int v2 = 0; v2 < 2; ++v2) {
                const uint16_t *wt = r0 + 2 * v2 < a.n_q ? a.wq : a.wk;
                if (wt != held) {
                    held = wt;
                    if (wt) widen8(__ldg(reinterpret_cast<const uint4 *>(wt) + hl), wv);
                }
                if (wt) {
                    const float inv = rsqrtf(fmaf(ss[v2], 1.f / kHeadDim, a.eps));
                    const uint64_t inv2 = pair(inv, inv);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[v2][e] = mul2(mul2(y[v2][e], inv2), wv[e]);
                }
            }
            uint32_t o[2][4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int v2 = 0; v2 < 2; ++v2) {
                    float p, q2;
                    unpair(y[v2][e], p, q2);
                    const uint64_t z = PAIRS ? pair(q2, p)
                                             : pair(__shfl_sync(0xffffffffu, p, partner), __shfl_sync(0xffffffffu, q2, partner));
                    unpair(fma2(y[v2][e], cs[e], mul2(z, sn[e])), p, q2);
                    o[v2][e] = pack2(p, q2);
                }
            if (!turns) {                                         // normalised at most, else moved as they are
#pragma unroll
                for (int v2 = 0; v2 < 2; ++v2) {
                    const bool normed = (r0 + 2 * v2 < a.n_q ? a.wq : a.wk) != nullptr;
                    const uint32_t as_read[4] = {raw[v2].x, raw[v2].y, raw[v2].z, raw[v2].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float p, q2;
                        unpair(y[v2][e], p, q2);
                        o[v2][e] = normed ? pack2(p, q2) : as_read[e];
                    }
                }
            }
#pragma unroll
            for (int v2 = 0; v2 < 2; ++v2) {
                const int r = r0 + 2 * v2;
                const bool is_q = r < a.n_q, is_v = r >= a.n_q + a.n_kv;
                if (r < in_warp && (is_q || page_ok))
                    *reinterpret_cast<uint4 *>((is_q ? qo : is_v ? vo : ko) + (long long)r * kHeadDim) =
                        is_v ? raw[v2] : make_uint4(o[v2][0], o[v2][1], o[v2][2], o[v2][3]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_append(const oscar_layout_t &L, const AppendInput &in, int n, const uint16_t *wq, const uint16_t *wk,
                          float eps, const float *rope, int rope_rows, int rot, bool pairs_interleaved, Bf16PoolView pool,
                          const int32_t *pt, int max_pages, int batch, const int32_t *req, const int32_t *pos,
                          const int32_t *rope_pos, uint16_t *q_out, int32_t *status, cudaStream_t st) {
    const int n_q = in.q ? L.n_kv_heads * L.gqa : 0;
    const int pairs = (n_q + 2 * L.n_kv_heads + 1) / 2;
    // A token's row pairs go to equal runs of as many warps as the SMs hold at once (16 each), one pair a warp at
    // least, and to one warp where there are more tokens than that.  (32 query and 8 kv heads: 300 tokens 6.3 us,
    // 1,024 10.0, 2,048 15.4, 4,000 26.0; twice the warps: 8.3, 10.4, 17.5, 26.0; half: 6.2, 11.6, 15.4, 26.0.)
    const int most = (int)std::max(1LL, std::min((long long)pairs, 16LL * 152 / n));
    const int per = (pairs + most - 1) / most, runs = (pairs + per - 1) / per;
    const AppendArgs a{in.q, in.k, in.v, in.q_stride, in.k_stride, in.v_stride, n, n_q, L.n_kv_heads, per, runs, wq, wk, eps,
                       rope, rope_rows, rot, pool, pt, max_pages, page_shift(L), batch, req, pos, rope_pos, q_out, status};
    const unsigned blocks = (unsigned)(((long long)n * runs + kWarps - 1) / kWarps);
    return launch_ahead(pairs_interleaved ? append_kernel<true> : append_kernel<false>, dim3(blocks), kWarps * 32, 0, st, a);
}

}  // namespace oscar
