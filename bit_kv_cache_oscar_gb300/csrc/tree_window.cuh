// The BF16 rows of tree attention, 16 query rows a CTA, and the join of a CTA's warps: run by the mma.sync kernel, and by CTAs of the
// tcgen05 kernel's launch.
#pragma once

#include <cuda_bf16.h>

#include "tree_args.cuh"

namespace oscar {

constexpr int kTile = 16;                        // query rows of a CTA
constexpr int kResRow = kHeadDim + 4;
constexpr float kNone = -1e30f;                  // reference before the first token

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); }
__device__ __forceinline__ uint32_t pack_b2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// The W warps that share a tile of query rows: the CTA, or a part of it with a barrier of its own.
template <int W, bool PART>
__device__ __forceinline__ void tile_sync(int barrier) {
    if (PART) asm volatile("bar.sync %0, %1;" ::"r"(barrier), "n"(W * 32) : "memory");
    else __syncthreads();
}
// Over the four lanes of a row.
__device__ __forceinline__ float row_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float row_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
// What a warp holds of its 16 rows: lane (g, t) has rows g and g + 8 (index r); out[c][i][2 r + e] is channel
// 32 c + 8 t + 4 e + i of row g + 8 r.
struct Rows {
    float m[2], l[2], z[4][2], out[4][4][4];
};

__device__ __forceinline__ void clear(Rows &x) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        x.m[r] = kNone;
        x.l[r] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) x.z[k][r] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) x.out[c][i][e] = 0.f;
}

// Channels 32 i + 8 t .. + 7 of query row g + 8 r of the tile, t = lane % 4.
__device__ __forceinline__ uint4 query_piece(const TreeArgs &a, const TreeRequest &rq, int h, int row0, int rows, int r, int i, int lane) {
    const int row = (lane >> 2) + 8 * r;
    if (row >= rows) return make_uint4(0, 0, 0, 0);
    return *reinterpret_cast<const uint4 *>(a.q + tree_row(a, rq, h, row0 + row) * kHeadDim + 32 * i + 8 * (lane & 3));
}

// ---- the BF16 rows ---------------------------------------------------------------------------------
// Positions [0, min(sink, T)), [max(hist_end, those), T) and the nodes' [T, T + n), in tiles of 16.  frag: 4 KB of the W warps' shared
// memory, stage: 8 KB of this warp's, a tile's values and keys: both are on their way at once, and a lane copies the pieces that it
// reads itself.  (Keys and values through registers: 64 x 4K, 16 nodes on tcgen05 343 us, so 318; one node on mma.sync 136 and 128.)
template <int W, bool PART = false>
__device__ __forceinline__ void window_warp(const TreeArgs &a, const TreeRequest &rq, int b, int h, int row0, int rows, uint4 *frag, uint4 *stage, int barrier,
                                            int warp, int lane, Rows &x) {
    const int g = lane >> 2, t = lane & 3, sh = a.page_shift, T = rq.T, end = T + rq.n;
    const int n0 = min(a.sink, T), lo1 = max(rq.he, n0), sink_tiles = (n0 + 15) / 16, rec0 = lo1 / 16;
    const int tiles = sink_tiles + (end + 15) / 16 - rec0;
    // the A operand of the logits, as it lies, for all warps: fragment 2 i + e of lane l at 32 (2 i + e) + l
    for (int k = warp; k < 4; k += W) {
        const uint4 x = query_piece(a, rq, h, row0, rows, 0, k, lane), y = query_piece(a, rq, h, row0, rows, 1, k, lane);
        frag[64 * k + lane] = make_uint4(x.x, y.x, x.y, y.y);
        frag[64 * k + 32 + lane] = make_uint4(x.z, y.z, x.w, y.w);
    }
    tile_sync<W, PART>(barrier);
    int node[2];                                     // of the lane's rows
#pragma unroll
    for (int r = 0; r < 2; ++r) node[r] = (row0 + min(g + 8 * r, rows - 1)) / a.G;
#pragma unroll 1
    for (int k = warp; k < tiles; k += W) {
        const bool in_sink = k < sink_tiles;
        const int p0 = (in_sink ? k : rec0 + k - sink_tiles) * 16, lo = in_sink ? 0 : lo1, hi = in_sink ? n0 : end;
        const int page = a.bpt[(size_t)b * a.max_pages + (p0 >> sh)];
        if ((uint32_t)page >= (uint32_t)a.bf.n_pages) {
            if (lane == 0) flag_status(a.status, OSCAR_DEV_BAD_BF16_PAGE);
            continue;
        }
        // lane (g, t): channels 32 i + 8 t .. + 7 of tokens g and g + 8
        const bool in0 = p0 + g >= lo && p0 + g < hi, in1 = p0 + g + 8 >= lo && p0 + g + 8 < hi;
        const size_t at = ((((size_t)page << sh) + ((p0 + g) & ((1 << sh) - 1))) * a.n_kv + h) * kHeadDim + 8 * t, far = (size_t)8 * a.n_kv * kHeadDim;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (in0) cp_async16(saddr(stage + 256 + 64 * c + lane), a.bf.k + at + 32 * c);
            if (in1) cp_async16(saddr(stage + 288 + 64 * c + lane), a.bf.k + at + far + 32 * c);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (in0) cp_async16(saddr(stage + 64 * c + lane), a.bf.v + at + 32 * c);
            if (in1) cp_async16(saddr(stage + 64 * c + 32 + lane), a.bf.v + at + far + 32 * c);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        float s[2][4];                               // [keys 8 u + 2 t + e][2 r + e]
#pragma unroll
        for (int u = 0; u < 2; ++u) s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 x = frag[64 * i + lane], y = frag[64 * i + 32 + lane];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint4 kk = (u ? in1 : in0) ? stage[256 + 32 * u + 64 * i + lane] : make_uint4(0, 0, 0, 0);
                mma16816_bf16(s[u], x.x, x.y, x.z, x.w, kk.x, kk.y);
                mma16816_bf16(s[u], y.x, y.y, y.z, y.w, kk.z, kk.w);
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int p = p0 + 8 * u + 2 * t + (e & 1), r = e >> 1;
                bool sees = p >= lo && p < hi;
                if (sees && p >= T) {
                    const int j = p - T;
                    sees = a.mask ? (a.mask[(size_t)(rq.first + node[r]) * a.mask_words + (j >> 5)] >> (j & 31)) & 1 : j <= node[r];
                }
                s[u][e] = sees ? s[u][e] * a.scale2 : -INFINITY;
            }
        float al[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float m = fmaxf(x.m[r], row_max(fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]))));
            al[r] = ex2_approx(x.m[r] - m);
            x.m[r] = m;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) s[u][2 * r + e] = ex2_approx(s[u][2 * r + e] - m);
            x.l[r] = fmaf(x.l[r], al[r], (s[0][2 * r] + s[0][2 * r + 1]) + (s[1][2 * r] + s[1][2 * r + 1]));
        }
        uint32_t ph[4], pl[4];                       // A operand: rows g, g + 8 of keys 2 t + e, then of keys 8 + 2 t + e
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t hi2 = pack_b2(s[u][2 * r], s[u][2 * r + 1]);
                ph[2 * u + r] = hi2;
                pl[2 * u + r] = pack_b2(s[u][2 * r] - lo16(hi2), s[u][2 * r + 1] - hi16(hi2));
            }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 v0 = in0 ? stage[64 * c + lane] : make_uint4(0, 0, 0, 0), v1 = in1 ? stage[64 * c + 32 + lane] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) x.out[c][i][e] *= al[e >> 1];
            // infinities and NaN among the values: rows that do not see them must not meet them in a product
            // (their product with 0 is NaN, all others' a zero of some sign)
            const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            __nv_bfloat162 zeros = as_bf2(0u);
#pragma unroll
            for (int e = 0; e < 8; ++e) zeros = __hfma2(as_bf2(w[e]), as_bf2(0u), zeros);
            if (__any_sync(0xffffffffu, (*reinterpret_cast<const uint32_t *>(&zeros) & 0x7fff7fffu) != 0)) {
                // one key at a time, only where it has weight
#pragma unroll 1
                for (int key = 0; key < 16; ++key) {
                    const int u = key >> 3, from = (lane & ~3) | ((key & 7) >> 1), p = p0 + key;
                    if (p < lo || p >= hi) continue;
                    float pr[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float first = __shfl_sync(0xffffffffu, u ? s[1][2 * r] : s[0][2 * r], from);
                        const float second = __shfl_sync(0xffffffffu, u ? s[1][2 * r + 1] : s[0][2 * r + 1], from);
                        pr[r] = key & 1 ? second : first;
                    }
                    const uint16_t *v = a.bf.v + ((((size_t)page << sh) + (p & ((1 << sh) - 1))) * a.n_kv + h) * kHeadDim + 8 * t + 32 * c;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (pr[e >> 1] != 0.f) x.out[c][i][e] = fmaf(pr[e >> 1], bf16_to_f32(v[4 * (e & 1) + i]), x.out[c][i][e]);
                }
                continue;
            }
            // channels 32 c + 4 n + 2 j + e of eight tokens are an 8 x 8 matrix of 16 bits: transposed, the B operand
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t sel = e ? 0x7632 : 0x5410;
                    const uint32_t b0 = movmatrix_trans(__byte_perm(j ? v0.y : v0.x, j ? v0.w : v0.z, sel));
                    const uint32_t b1 = movmatrix_trans(__byte_perm(j ? v1.y : v1.x, j ? v1.w : v1.z, sel));
                    mma16816_bf16(x.out[c][2 * j + e], pl[0], pl[1], pl[2], pl[3], b0, b1);
                    mma16816_bf16(x.out[c][2 * j + e], ph[0], ph[1], ph[2], ph[3], b0, b1);
                }
        }
    }
}

// ---- the join --------------------------------------------------------------------------------------
// The rows of W warps, each under references of its own, joined through shared memory (join_bytes<W>()): to the slot of the
// partials, or, with whole, as the result.
template <int W>
constexpr int join_bytes() { return (3 * W * kTile + kTile + W * kTile * kResRow) * 4; }

template <int W, bool PART = false>
__device__ __forceinline__ void join_warps(const TreeArgs &a, const TreeRequest &rq, int h, int row0, int rows, int slot, bool whole, uint8_t *smem, int barrier,
                                           int tid, int warp, int lane, Rows &x) {
    const int S = a.part.S;
    float *wm = reinterpret_cast<float *>(smem), *wl = wm + W * kTile, *wa = wl + W * kTile + warp * kTile * kResRow;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = g + 8 * r;
        const float l = row_sum(x.l[r]);
        if (t == 0) {
            wm[warp * kTile + row] = l > 0.f ? x.m[r] : l != l ? l : -INFINITY;       // (NaN where a logit was: it has to reach the row)
            wl[warp * kTile + row] = l;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float4 *>(wa + row * kResRow + 32 * c + 8 * t + 4 * e) =
                    make_float4(x.out[c][0][2 * r + e], x.out[c][1][2 * r + e], x.out[c][2][2 * r + e], x.out[c][3][2 * r + e]);
    }
    tile_sync<W, PART>(barrier);
    // every warp's weight 2^(m - M) once, then the sums
    const float *sum = wl + W * kTile;
    float *wf = wl + W * kTile + W * kTile * kResRow, *wM = wf + W * kTile;
    if (tid < W * kTile) {
        const int row = tid % kTile;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, wm[w * kTile + row]);
        wf[tid] = wm[tid] != -INFINITY ? exp2f(wm[tid] - M) : 0.f;
        if (tid < kTile) wM[row] = M;
    }
    tile_sync<W, PART>(barrier);
    for (int e = tid; e < rows * (kHeadDim / 4); e += W * 32) {
        const int row = e / (kHeadDim / 4), d = 4 * (e % (kHeadDim / 4));
        float L = 0.f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = wf[w * kTile + row];
            if (f == 0.f) continue;
            const float4 y = *reinterpret_cast<const float4 *>(sum + (w * kTile + row) * kResRow + d);
            L = fmaf(wl[w * kTile + row], f, L);
            A = make_float4(fmaf(y.x, f, A.x), fmaf(y.y, f, A.y), fmaf(y.z, f, A.z), fmaf(y.w, f, A.w));
        }
        const size_t orow = tree_row(a, rq, h, row0 + row), at = orow * (S + 1) + slot;
        if (whole) {
            const bool on = L > 0.f || L != L;
            const float o0 = on ? __fdiv_rn(A.x, L) : 0.f, o1 = on ? __fdiv_rn(A.y, L) : 0.f, o2 = on ? __fdiv_rn(A.z, L) : 0.f,
                        o3 = on ? __fdiv_rn(A.w, L) : 0.f;
            *reinterpret_cast<uint2 *>(a.o + orow * kHeadDim + d) = make_uint2(pack_b2(o0, o1), pack_b2(o2, o3));
            if (a.lse && d == 0) a.lse[orow] = on ? (wM[row] + log2f(L)) * 0.6931471805599453f : -INFINITY;
            continue;
        }
        *reinterpret_cast<float4 *>(a.part.acc + at * kHeadDim + d) = A;
        if (d == 0) {
            a.part.m[at] = L != L ? L : wM[row];
            a.part.l[at] = L;
        }
    }
}

}  // namespace oscar
