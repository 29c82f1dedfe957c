// Eviction from the INT4 history by accumulated weight: which positions stay, and the move of their rows.
//
// For each (request, kv head) the `keep` positions of largest weight in [sink, hist_end) are kept, ties
// going to the lowest position.  The weights are mapped to integers of the same order and the keep-th
// largest is found digit by digit from the top (histogram of the digit among the values that match the
// digits found so far, then the bin where the count from above reaches keep).  A position stays if its
// value is above that threshold, or equal to it and among the first `keep - above` equal ones.  A second
// kernel copies the kept rows to their new pages.

#include "int4.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

struct EvictArgs {
    Int4PoolView src, dst;
    const int32_t *spt, *dpt;
    int max_pages, page_size, n_kv, group, sink;
    const int32_t *seq_len, *hist_end, *keep;
    const float *mass;
    float *mass_out;
    int32_t *kept;
    int kept_stride;
    int32_t *status;
};

// Larger weight, larger key; -0 as +0, NaN above all.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// History length n and number kept k of request b; false if it is left alone.  Every thread of both
// kernels decides alike.
__device__ __forceinline__ bool read_request(const EvictArgs &a, int b, int &T, int &he, int &n, int &k, bool flag) {
    k = a.keep[b];
    if (k == -1) return false;
    read_lengths(a.seq_len, a.hist_end, b, a.sink, a.max_pages * a.page_size, a.status, T, he);
    n = he > a.sink ? he - a.sink : 0;
    if (k < 0 || k > n || k > a.kept_stride) {
        if (flag) flag_status(a.status, OSCAR_DEV_BAD_LENGTH);
        return false;
    }
    return true;
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int cnt_gt[kWarps], cnt_eq[kWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int T, he, n, k;
    if (!read_request(a, b, T, he, n, k, threadIdx.x == 0 && h == 0)) return;
    if (k == 0) return;
    const float *m = a.mass + ((size_t)b * a.n_kv + h) * a.max_pages * a.page_size + a.sink;
    uint32_t prefix = 0;
    int left = k;                                     // still to find among the values that match the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint32_t key = order_key(m[i]);
            if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int d = 255, sum = 0;
            while (sum + hist[d] < left) sum += hist[d--];
            s_prefix = prefix | ((uint32_t)d << shift);
            s_left = left - sum;
        }
        __syncthreads();
        prefix = s_prefix;
        left = s_left;
    }
    // warp w takes the positions [w n / W, (w + 1) n / W): counts first, then its places in the list
    const int lo = (int)((long long)warp * n / kWarps), hi = (int)((long long)(warp + 1) * n / kWarps);
    int gt = 0, eq = 0;
    for (int i = lo; i < hi; i += 32) {
        const uint32_t key = i + lane < hi ? order_key(m[i + lane]) : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, i + lane < hi && key > prefix));
        eq += __popc(__ballot_sync(0xffffffffu, i + lane < hi && key == prefix));
    }
    if (lane == 0) {
        cnt_gt[warp] = gt;
        cnt_eq[warp] = eq;
    }
    __syncthreads();
    int gt0 = 0, eq0 = 0;
    for (int w = 0; w < warp; ++w) {
        gt0 += cnt_gt[w];
        eq0 += cnt_eq[w];
    }
    int32_t *out = a.kept + ((size_t)b * a.n_kv + h) * a.kept_stride;
    const uint32_t below = (1u << lane) - 1;
    for (int i = lo; i < hi; i += 32) {
        const bool in = i + lane < hi;
        const uint32_t key = in ? order_key(m[i + lane]) : 0u;
        const uint32_t bg = __ballot_sync(0xffffffffu, in && key > prefix), be = __ballot_sync(0xffffffffu, in && key == prefix);
        const int e = eq0 + __popc(be & below);                       // equal ones before this position
        const int at = gt0 + __popc(bg & below) + min(e, left);
        if (in && (key > prefix || (key == prefix && e < left))) out[at] = a.sink + i + lane;
        gt0 += __popc(bg);
        eq0 += __popc(be);
    }
}

__global__ void __launch_bounds__(256) evict_move_kernel(EvictArgs a) {
    const int h = blockIdx.y, b = blockIdx.z, hl = threadIdx.x & 7;
    int T, he, n, k;
    if (!read_request(a, b, T, he, n, k, false)) return;
    const size_t row0 = ((size_t)b * a.n_kv + h) * a.max_pages * a.page_size;
    const int32_t *kept = a.kept + ((size_t)b * a.n_kv + h) * a.kept_stride;
    const int G = kHeadDim / a.group;
    // 8 lanes a row: 4 with the key's 64 bytes, 4 with the value's
    for (int j = blockIdx.x * 32 + (threadIdx.x >> 3); j < k; j += gridDim.x * 32) {
        const int p = kept[j], to = a.sink + j;
        const int sp = a.spt[(size_t)b * a.max_pages + p / a.page_size], dp = a.dpt[(size_t)b * a.max_pages + to / a.page_size];
        if (hl == 0) a.mass_out[row0 + to] = a.mass[row0 + p];
        if (sp < 0 || sp >= a.src.n_pages || dp < 0 || dp >= a.dst.n_pages) {
            if (hl == 0) flag_status(a.status, OSCAR_DEV_BAD_INT4_PAGE);
            continue;
        }
        const size_t from = row4(sp, a.n_kv, h, a.page_size, p % a.page_size), at = row4(dp, a.n_kv, h, a.page_size, to % a.page_size);
        const uint8_t *sc = hl < 4 ? a.src.codes_k : a.src.codes_v;
        uint8_t *dc = hl < 4 ? a.dst.codes_k : a.dst.codes_v;
        reinterpret_cast<uint4 *>(dc + at * kRow4)[hl & 3] = reinterpret_cast<const uint4 *>(sc + from * kRow4)[hl & 3];
        if (hl < G)
            reinterpret_cast<uint2 *>(a.dst.scale_zero)[at * G + hl] = reinterpret_cast<const uint2 *>(a.src.scale_zero)[from * G + hl];
    }
    // the weights outside the kept rows: sink, recent rows, nothing behind them
    const int N = a.max_pages * a.page_size, shift = n - k, lo = min(a.sink, T);
    for (int i = blockIdx.x * 256 + threadIdx.x; i < N; i += gridDim.x * 256) {
        if (i < lo) a.mass_out[row0 + i] = a.mass[row0 + i];
        else if (i >= lo + k) a.mass_out[row0 + i] = i + shift < T ? a.mass[row0 + i + shift] : 0.f;
    }
}

}  // namespace

cudaError_t launch_evict(const oscar_layout_t &L, Int4PoolView src, const int32_t *spt, Int4PoolView dst,
                         const int32_t *dpt, int max_pages, int batch, const int32_t *seq_len, const int32_t *hist_end,
                         const int32_t *keep, const float *mass, float *mass_out, int32_t *kept, int kept_stride,
                         int32_t *status, cudaStream_t st) {
    const EvictArgs a{src, dst, spt, dpt, max_pages, L.page_size, L.n_kv_heads, L.group, L.sink, seq_len, hist_end, keep,
                      mass, mass_out, kept, kept_stride, status};
    evict_select_kernel<<<dim3(L.n_kv_heads, batch), kThreads, 0, st>>>(a);
    if (cudaError_t e = cudaGetLastError()) return e;
    const long long most = ((long long)max_pages * L.page_size + 255) / 256;
    const long long want = (8 * 152 + batch * L.n_kv_heads - 1) / (batch * L.n_kv_heads);
    evict_move_kernel<<<dim3((unsigned)(want < most ? want : most), L.n_kv_heads, batch), 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace oscar
