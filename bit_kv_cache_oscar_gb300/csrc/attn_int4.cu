// Decode attention over an INT4 history with BF16 sink and recent rows, and the attention weight each
// position received (CUDA cores: the form every faster one is checked against).
//
// One CTA = (split, kv head, request); split S is the BF16 rows.  A warp takes a token at a time, a lane
// four channels of it; the head's G queries share each row.  Online softmax in base 2.

#include "int4.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 4, kBlock = 32;

struct Attn4Args {
    const uint16_t *q;
    Bf16PoolView bf;
    const int32_t *bpt;
    Int4PoolView i4;
    const int32_t *ipt;
    int max_pages, page_size, n_kv, group, sink;
    const int32_t *seq_len, *hist_end;
    float scale2;
    PartialsView out;
    const float *lse;          // mass only
    float *mass;
    int32_t *status;
};

__device__ __forceinline__ void row_bf16(const uint16_t *p, int lane, float (&x)[4]) {
    const uint2 w = reinterpret_cast<const uint2 *>(p)[lane];
    x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ void row_int4(const uint8_t *codes, const uint16_t *sz, size_t row, int group, int lane, float (&x)[4]) {
    const uint32_t c = reinterpret_cast<const uint16_t *>(codes + row * kRow4)[lane];
    const uint32_t w = *reinterpret_cast<const uint32_t *>(sz + (row * (kHeadDim / group) + 4 * lane / group) * 4);
    const float s = __uint_as_float(w << 16), z = __uint_as_float(w & 0xffff0000u);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fmaf((float)((c >> (4 * e)) & 15u), s, z);
}

template <int G, bool MASS>
__global__ void __launch_bounds__(kWarps * 32) attn4_kernel(Attn4Args a) {
    __shared__ float sm_m[kWarps][G], sm_l[kWarps][G], sm_acc[kWarps][G][kHeadDim];
    const int s = blockIdx.x, h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int Hq = a.n_kv * G, S = a.out.S;
    int T, he;
    read_lengths(a.seq_len, a.hist_end, b, a.sink, a.max_pages * a.page_size, a.status, T, he);
    const bool window = s == S;
    const int n0 = min(a.sink, T), lo1 = max(he, n0);
    int lo, hi;                                        // token range, or window index range
    if (window) {
        lo = 0;
        hi = n0 + T - lo1;
    } else {
        const int first = a.sink / kBlock, nb = he > a.sink ? (he + kBlock - 1) / kBlock - first : 0;
        lo = max(a.sink, (first + (int)((long long)s * nb / S)) * kBlock);
        hi = min(he, (first + (int)((long long)(s + 1) * nb / S)) * kBlock);
    }
    float q[G][4], m[G], l[G], acc[G][4];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        row_bf16(a.q + ((size_t)b * Hq + h * G + g) * kHeadDim, lane, q[g]);
        m[g] = MASS ? a.lse[(size_t)b * Hq + h * G + g] * kLog2e : -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[g][c] = 0.f;
    }
    for (int i = lo + warp; i < hi; i += kWarps) {
        const int p = window ? (i < n0 ? i : lo1 + i - n0) : i;
        const int page = (window ? a.bpt : a.ipt)[(size_t)b * a.max_pages + p / a.page_size];
        if (page < 0 || page >= (window ? a.bf.n_pages : a.i4.n_pages)) {
            if (lane == 0) flag_status(a.status, window ? OSCAR_DEV_BAD_BF16_PAGE : OSCAR_DEV_BAD_INT4_PAGE);
            continue;
        }
        float k[4], v[4];
        const size_t rb = (((size_t)page * a.page_size + p % a.page_size) * a.n_kv + h) * kHeadDim;
        const size_t r4 = row4(page, a.n_kv, h, a.page_size, p % a.page_size);
        if (window) row_bf16(a.bf.k + rb, lane, k);
        else row_int4(a.i4.codes_k, a.i4.scale_zero, r4, a.group, lane, k);
        if (!MASS) {
            if (window) row_bf16(a.bf.v + rb, lane, v);
            else row_int4(a.i4.codes_v, a.i4.scale_zero + 2, r4, a.group, lane, v);
        }
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float t = q[g][0] * k[0];
#pragma unroll
            for (int c = 1; c < 4; ++c) t = fmaf(q[g][c], k[c], t);
#pragma unroll
            for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            t *= a.scale2;
            if (MASS) {
                if (m[g] != -INFINITY) sum += exp2f(t - m[g]);
            } else {
                const float mn = fmaxf(m[g], t), al = exp2f(m[g] - mn), pr = exp2f(t - mn);
                l[g] = fmaf(l[g], al, pr);
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[g][c] = fmaf(acc[g][c], al, pr * v[c]);
                m[g] = mn;
            }
        }
        if (MASS && lane == 0) a.mass[((size_t)b * a.n_kv + h) * a.max_pages * a.page_size + p] += sum;
    }
    if (MASS) return;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        if (lane == 0) {
            sm_m[warp][g] = m[g];
            sm_l[warp][g] = l[g];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) sm_acc[warp][g][4 * lane + c] = acc[g][c];
    }
    __syncthreads();
    const int d = threadIdx.x;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float M = -INFINITY, L = 0.f, A = 0.f;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][g]);
        if (M != -INFINITY)
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2f(sm_m[w][g] - M);
                L = fmaf(sm_l[w][g], f, L);
                A = fmaf(sm_acc[w][g][d], f, A);
            }
        const size_t row = ((size_t)b * Hq + h * G + g) * (S + 1) + s;
        a.out.acc[row * kHeadDim + d] = A;
        if (d == 0) {
            a.out.m[row] = M;
            a.out.l[row] = L;
        }
    }
}

template <bool MASS>
cudaError_t launch(const Attn4Args &a, int gqa, dim3 grid, cudaStream_t st) {
    switch (gqa) {
        case 1: attn4_kernel<1, MASS><<<grid, kWarps * 32, 0, st>>>(a); break;
        case 2: attn4_kernel<2, MASS><<<grid, kWarps * 32, 0, st>>>(a); break;
        case 4: attn4_kernel<4, MASS><<<grid, kWarps * 32, 0, st>>>(a); break;
        default: attn4_kernel<8, MASS><<<grid, kWarps * 32, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

int suggest_splits4(const oscar_layout_t &L, int batch, int max_hist, int sm_count) {
    const long long per = (long long)batch * L.n_kv_heads, blocks = ((long long)max_hist + kBlock - 1) / kBlock;
    long long want = (16LL * sm_count + per - 1) / per;
    if (want > blocks) want = blocks;
    return (int)(want < 1 ? 1 : want > 1024 ? 1024 : want);
}

cudaError_t launch_decode4(const oscar_layout_t &L, const Attn4Input &in, int batch, PartialsView out, uint16_t *o,
                           float *of, float *lse, int32_t *counters, int32_t *status, cudaStream_t st) {
    const Attn4Args a{in.q, in.bf, in.bpt, in.i4, in.ipt, in.max_pages, L.page_size, L.n_kv_heads, L.group, L.sink,
                      in.seq_len, in.hist_end, in.sm_scale * kLog2e, out, nullptr, nullptr, status};
    if (cudaError_t e = launch<false>(a, L.gqa, dim3(out.S + 1, L.n_kv_heads, batch), st)) return e;
    if (!o && !of) return cudaSuccess;
    return launch_merge(L, out, nullptr, batch, o, of, lse, st);
}

cudaError_t launch_mass4(const oscar_layout_t &L, const Attn4Input &in, int batch, const float *lse, float *mass,
                         int32_t *status, cudaStream_t st) {
    const int S = suggest_splits4(L, batch, in.max_pages * L.page_size, 152);
    const Attn4Args a{in.q, in.bf, in.bpt, in.i4, in.ipt, in.max_pages, L.page_size, L.n_kv_heads, L.group, L.sink,
                      in.seq_len, in.hist_end, in.sm_scale * kLog2e, PartialsView{nullptr, nullptr, nullptr, S}, lse, mass, status};
    return launch<true>(a, L.gqa, dim3(S + 1, L.n_kv_heads, batch), st);
}

}  // namespace oscar
