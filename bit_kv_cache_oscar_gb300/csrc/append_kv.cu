// New tokens into the BF16 cache: per-head RMS norm, rotary position and the paged write in one pass.
//
// y = x / sqrt(mean(x^2) + eps) * w over a head's 128 channels, then the rotation of the first
// rot_dim channels by the token's angles, (a, b) -> (a cos - b sin, b cos + a sin); fp32 throughout,
// one rounding to bf16.  Queries go to q_out, keys and values to their slots of the BF16 pool.
//
// A head's row is 256 bytes: 16 lanes with 8 channels each (one 16-byte load and store a lane), so
// the sum of squares is a 4-step shuffle and a rotation partner is either in the lane (channels 2j,
// 2j+1) or rot_dim/16 lanes away.  A warp takes 2·U rows of one token and loads them all before it
// needs the first; the token's angles are read once for all of them.

#include "oscar_internal.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 8;

struct AppendArgs {
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    int n, n_q, n_kv, chunks;      // chunks: warps per token
    const uint16_t *wq, *wk;
    float eps;
    const float *rope;
    int rope_rows, rot;
    Bf16PoolView pool;
    const int32_t *pt;
    int max_pages, page_size, batch;
    const int32_t *req, *pos, *rope_pos;
    uint16_t *q_out;
    int32_t *status;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
    x[0] = lo16(w.x); x[1] = hi16(w.x); x[2] = lo16(w.y); x[3] = hi16(w.y);
    x[4] = lo16(w.z); x[5] = hi16(w.z); x[6] = lo16(w.w); x[7] = hi16(w.w);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return (uint32_t)f32_to_bf16_rn(a) | ((uint32_t)f32_to_bf16_rn(b) << 16);
}

template <int U, bool PAIRS>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(AppendArgs a) {
    const int lane = threadIdx.x & 31, half = lane >> 4, hl = lane & 15;
    const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5);       // below 2^32: n * chunks is (launch_append)
    const int i = (int)(w / (uint32_t)a.chunks);
    if (i >= a.n) return;
    const int row0 = (int)(w - (uint32_t)i * a.chunks) * 2 * U + half;
    const int rows = a.n_q + 2 * a.n_kv;

    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = row0 + 2 * u;
        const uint16_t *src = r < a.n_q            ? a.q + i * a.q_stride + (long long)r * kHeadDim
                              : r < a.n_q + a.n_kv ? a.k + i * a.k_stride + (long long)(r - a.n_q) * kHeadDim
                                                   : a.v + i * a.v_stride + (long long)(r - a.n_q - a.n_kv) * kHeadDim;
        x[u] = r < rows ? *reinterpret_cast<const uint4 *>(src + 8 * hl) : make_uint4(0, 0, 0, 0);
    }
    const int pos = a.pos[i], b = a.req[i];
    if (pos == -1) return;                                        // padding
    const int rp = a.rope_pos ? a.rope_pos[i] : pos;
    if (b < 0 || b >= a.batch || pos < 0 || pos / a.page_size >= a.max_pages ||
        (a.rope && (rp < 0 || rp >= a.rope_rows))) {
        if (lane == 0) flag_status(a.status, OSCAR_DEV_BAD_LENGTH);
        return;
    }
    const int page = a.pt[(size_t)b * a.max_pages + pos / a.page_size];
    const bool page_ok = page >= 0 && page < a.pool.n_pages;
    if (!page_ok && lane == 0) flag_status(a.status, OSCAR_DEV_BAD_BF16_PAGE);
    const size_t slot = ((size_t)(page_ok ? page : 0) * a.page_size + pos % a.page_size) * a.n_kv;

    // this lane's angles: pair j0 + e (channels 2j, 2j+1), or channels 8 hl + e of either half
    const int rl = a.rot >> 4;                                    // lanes per rotated half
    const bool turns = a.rope && 8 * hl < a.rot;
    float cs[8], sn[8];
    if (turns) {
        const float *t = a.rope + (size_t)rp * kHeadDim + (PAIRS ? 4 * hl : 8 * (hl < rl ? hl : hl - rl));
#pragma unroll
        for (int e = 0; e < (PAIRS ? 4 : 8); e += 4) {
            const float4 c = *reinterpret_cast<const float4 *>(t + e), s = *reinterpret_cast<const float4 *>(t + 64 + e);
            cs[e] = c.x; cs[e + 1] = c.y; cs[e + 2] = c.z; cs[e + 3] = c.w;
            sn[e] = s.x; sn[e + 1] = s.y; sn[e + 2] = s.z; sn[e + 3] = s.w;
        }
    }
    const int partner = (lane & 16) | (turns ? (hl < rl ? hl + rl : hl - rl) : hl);

#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = row0 + 2 * u;
        const bool is_q = r < a.n_q, is_v = r >= a.n_q + a.n_kv;
        float y[8];
        unpack8(x[u], y);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
        for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const uint16_t *wt = is_q ? a.wq : a.wk;
        if (wt && !is_v) {
            const float inv = rsqrtf(fmaf(ss, 1.f / kHeadDim, a.eps));
            float wv[8];
            unpack8(__ldg(reinterpret_cast<const uint4 *>(wt) + hl), wv);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * wv[e];
        }
        uint4 out = x[u];
        if constexpr (PAIRS) {
            if (turns) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = y[2 * e], s = y[2 * e + 1];
                    y[2 * e] = fmaf(p, cs[e], -s * sn[e]);
                    y[2 * e + 1] = fmaf(s, cs[e], p * sn[e]);
                }
            }
        } else {
            float z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = __shfl_sync(0xffffffffu, y[e], partner);
            if (turns) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], cs[e], hl < rl ? -z[e] * sn[e] : z[e] * sn[e]);
            }
        }
        if (!is_v) out = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
        if (r >= rows || (!is_q && !page_ok)) continue;
        uint16_t *dst = is_q ? a.q_out + ((size_t)i * a.n_q + r) * kHeadDim
                        : is_v ? const_cast<uint16_t *>(a.pool.v) + (slot + r - a.n_q - a.n_kv) * kHeadDim
                               : const_cast<uint16_t *>(a.pool.k) + (slot + r - a.n_q) * kHeadDim;
        *reinterpret_cast<uint4 *>(dst + 8 * hl) = out;
    }
}

}  // namespace

cudaError_t launch_append(const oscar_layout_t &L, const AppendInput &in, int n, const uint16_t *wq, const uint16_t *wk,
                          float eps, const float *rope, int rope_rows, int rot, bool pairs, Bf16PoolView pool,
                          const int32_t *pt, int max_pages, int batch, const int32_t *req, const int32_t *pos,
                          const int32_t *rope_pos, uint16_t *q_out, int32_t *status, cudaStream_t st) {
    const int n_q = in.q ? L.n_kv_heads * L.gqa : 0;
    AppendArgs a{in.q, in.k, in.v, in.q_stride, in.k_stride, in.v_stride, n, n_q, L.n_kv_heads, 0, wq, wk, eps, rope,
                 rope_rows, rot, pool, pt, max_pages, L.page_size, batch, req, pos, rope_pos, q_out, status};
    const int rows = n_q + 2 * L.n_kv_heads;
    auto run = [&](auto kern, int U) {
        a.chunks = (rows + 2 * U - 1) / (2 * U);
        const long long blocks = ((long long)n * a.chunks + kWarps - 1) / kWarps;
        kern<<<(unsigned)blocks, kWarps * 32, 0, st>>>(a);
        return cudaGetLastError();
    };
    // Few tokens: one row a half-warp, so that a step's rows are all in flight on as many warps as there
    // are.  Once four rows each still fill every SM with 32 warps, fewer warps with more loads each.
    const bool many = (long long)n * ((rows + 7) / 8) >= 152 * 32;
    if (pairs) return many ? run(append_kernel<4, true>, 4) : run(append_kernel<1, true>, 1);
    return many ? run(append_kernel<4, false>, 4) : run(append_kernel<1, false>, 1);
}

}  // namespace oscar
