// Eviction from the INT4 history by accumulated weight: which positions stay, and the move of their rows.
//
// For each (request, kv head) the `keep` positions of largest weight in [sink, hist_end) are kept, ties
// going to the lowest position.  The weights are mapped to integers of the same order and the keep-th
// largest is found digit by digit from the top (histogram of the digit among the values that match the
// digits found so far, then the bin where the count from above reaches keep).  A position stays if its
// value is above that threshold, or equal to it and among the first `keep - above` equal ones.  The
// positions come out in order because each warp takes a run of them and knows the counts before its run.
// A second kernel copies the kept rows to their new pages, 8 lanes a row.

#include "int4.cuh"
#include "ptx.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;                 // digits of 11, 11 and 10 bits
constexpr int kCached = 16384;              // keys of a CTA's slice held in shared memory
constexpr int kCluster = 8;

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

__device__ __forceinline__ int ld_cluster(const int *p, int rank) {
    uint32_t ra;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(saddr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ra) : "memory");
    return v;
}

// One cluster of C CTAs (grid x = C·Hkv) per (request, kv head); CTA r takes the slice [r n / C, (r + 1) n / C)
// of the history and holds its keys in shared memory (kCached of them; the rest is read again each pass).
__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a, int C) {
    extern __shared__ uint32_t keys[];
    __shared__ int hist[kBins], tot[kBins];            // tot: the cluster's counts of this CTA's share of the bins
    __shared__ int bins[kBins];                        // the counts of the share that holds the digit
    __shared__ int cnt_gt[kWarps], cnt_eq[kWarps], red[kWarps];
    __shared__ int share, found[2], slice_gt, slice_eq;
    const int rank = blockIdx.x % C, h = blockIdx.x / C, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int T, he, n, k;
    if (!read_request(a, b, T, he, n, k, threadIdx.x == 0 && blockIdx.x == 0) || k == 0) return;     // the whole cluster alike
    const int lo = (int)((long long)rank * n / C), hi = (int)((long long)(rank + 1) * n / C);
    const float *m = a.mass + ((size_t)b * a.n_kv + h) * a.max_pages * a.page_size + a.sink + lo;
    const int len = hi - lo, cached = min(len, kCached);
    auto key_at = [&](int i) { return i < cached ? keys[i] : order_key(m[i]); };
    for (int i = threadIdx.x; i < cached; i += kThreads) keys[i] = order_key(m[i]);

    uint32_t prefix = 0;
    int left = k;                                      // still to find among the keys that match the prefix
    const int per = kBins / C;                         // bins of one CTA's share
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, nb = pass == 2 ? 1024 : 2048;
        const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u;
        for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < len; i += kThreads) {
            const uint32_t key = key_at(i);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (nb - 1)], 1);
        }
        if (C > 1) cluster_sync_all(); else __syncthreads();
        int sum = 0;
        for (int i = threadIdx.x; i < per; i += kThreads) {
            int v = 0;
            for (int r = 0; r < C; ++r) v += C > 1 ? ld_cluster(&hist[rank * per + i], r) : hist[i];
            tot[i] = v;
            sum += v;
        }
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) red[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            int s = 0;
            for (int w = 0; w < kWarps; ++w) s += red[w];
            share = s;
        }
        if (C > 1) cluster_sync_all(); else __syncthreads();
        // every CTA: the share, from the top, in which the count reaches `left`, then its bin
        int r = C - 1;
        for (; r > 0; --r) {
            const int s = C > 1 ? ld_cluster(&share, r) : share;
            if (left <= s) break;
            left -= s;
        }
        for (int i = threadIdx.x; i < per; i += kThreads) bins[i] = C > 1 ? ld_cluster(&tot[i], r) : tot[i];
        __syncthreads();
        if (warp == 0) {
            const int q = per / 32, top = per - lane * q;            // lane 0: the highest q bins
            int s = 0;
            for (int i = 1; i <= q; ++i) s += bins[top - i];
            int before = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += v;
            }
            before -= s;
            if (before < left && left <= before + s) {
                int i = 1;
                while (before + bins[top - i] < left) before += bins[top - i++];
                found[0] = r * per + top - i;
                found[1] = left - before;
            }
        }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        left = found[1];
    }

    // places: warp w takes [w len / W, (w + 1) len / W) of the slice; counts first, then positions in order
    const int w0 = (int)((long long)warp * len / kWarps), w1 = (int)((long long)(warp + 1) * len / kWarps);
    int gt = 0, eq = 0;
    for (int i = w0; i < w1; i += 32) {
        const bool in = i + lane < w1;
        const uint32_t key = in ? key_at(i + lane) : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, in && key > prefix));
        eq += __popc(__ballot_sync(0xffffffffu, in && key == prefix));
    }
    if (lane == 0) {
        cnt_gt[warp] = gt;
        cnt_eq[warp] = eq;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int x = 0, y = 0;
        for (int w = 0; w < kWarps; ++w) {
            x += cnt_gt[w];
            y += cnt_eq[w];
        }
        slice_gt = x;
        slice_eq = y;
    }
    if (C > 1) cluster_sync_all(); else __syncthreads();
    int gt0 = 0, eq0 = 0;
    for (int r = 0; r < rank; ++r) {
        gt0 += ld_cluster(&slice_gt, r);
        eq0 += ld_cluster(&slice_eq, r);
    }
    for (int w = 0; w < warp; ++w) {
        gt0 += cnt_gt[w];
        eq0 += cnt_eq[w];
    }
    int32_t *out = a.kept + ((size_t)b * a.n_kv + h) * a.kept_stride;
    const uint32_t below = (1u << lane) - 1;
    for (int i = w0; i < w1; i += 32) {
        const bool in = i + lane < w1;
        const uint32_t key = in ? key_at(i + lane) : 0u;
        const uint32_t bg = __ballot_sync(0xffffffffu, in && key > prefix), be = __ballot_sync(0xffffffffu, in && key == prefix);
        const int e = eq0 + __popc(be & below);                       // equal ones before this position
        const int at = gt0 + __popc(bg & below) + min(e, left);
        if (in && (key > prefix || (key == prefix && e < left))) out[at] = a.sink + lo + i + lane;
        gt0 += __popc(bg);
        eq0 += __popc(be);
    }
    if (C > 1) cluster_sync_all();                     // no CTA leaves while another reads its memory
}

// grid (X, Hkv, batch).  A row is 8 lanes: 4 with the key's 64 bytes, 4 with the value's; a thread has
// kMoveRows rows in flight (list entry, page table, data: three dependent loads each).
constexpr int kMoveRows = 4;

__global__ void __launch_bounds__(256) evict_move_kernel(EvictArgs a) {
    const int h = blockIdx.y, b = blockIdx.z, hl = threadIdx.x & 7;
    int T, he, n, k;
    if (!read_request(a, b, T, he, n, k, false)) return;
    const size_t row0 = ((size_t)b * a.n_kv + h) * a.max_pages * a.page_size;
    const int32_t *kept = a.kept + ((size_t)b * a.n_kv + h) * a.kept_stride;
    const int32_t *spt = a.spt + (size_t)b * a.max_pages, *dpt = a.dpt + (size_t)b * a.max_pages;
    const int G = kHeadDim / a.group, step = gridDim.x * 32;
    const uint8_t *sc = hl < 4 ? a.src.codes_k : a.src.codes_v;
    uint8_t *dc = hl < 4 ? a.dst.codes_k : a.dst.codes_v;
    for (long long j0 = blockIdx.x * 32 + (threadIdx.x >> 3); j0 < k; j0 += (long long)kMoveRows * step) {
        int p[kMoveRows], sp[kMoveRows], dp[kMoveRows];
        uint4 x[kMoveRows];
        uint2 z[kMoveRows];
        float w[kMoveRows];
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) p[u] = j0 + (long long)u * step < k ? kept[j0 + (long long)u * step] : -1;
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) {
            if (p[u] < 0) continue;
            const int to = a.sink + (int)(j0 + (long long)u * step);
            sp[u] = spt[p[u] / a.page_size];
            dp[u] = dpt[to / a.page_size];
            w[u] = hl == 0 ? a.mass[row0 + p[u]] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) {
            if (p[u] < 0) continue;
            if ((uint32_t)sp[u] >= (uint32_t)a.src.n_pages || (uint32_t)dp[u] >= (uint32_t)a.dst.n_pages) {
                if (hl == 0) flag_status(a.status, OSCAR_DEV_BAD_INT4_PAGE);
                dp[u] = -1;
                continue;
            }
            const size_t from = row4(sp[u], a.n_kv, h, a.page_size, p[u] % a.page_size);
            x[u] = reinterpret_cast<const uint4 *>(sc + from * kRow4)[hl & 3];
            if (hl < G) z[u] = reinterpret_cast<const uint2 *>(a.src.scale_zero)[from * G + hl];
        }
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) {
            if (p[u] < 0) continue;
            const int to = a.sink + (int)(j0 + (long long)u * step);
            if (hl == 0) a.mass_out[row0 + to] = w[u];
            if (dp[u] < 0) continue;
            const size_t at = row4(dp[u], a.n_kv, h, a.page_size, to % a.page_size);
            reinterpret_cast<uint4 *>(dc + at * kRow4)[hl & 3] = x[u];
            if (hl < G) reinterpret_cast<uint2 *>(a.dst.scale_zero)[at * G + hl] = z[u];
        }
    }
    // the weights outside the kept rows: sink, recent rows, nothing behind them
    const int N = a.max_pages * a.page_size, shift = n - k, lo = min(a.sink, T);
    for (long long i = blockIdx.x * 256 + threadIdx.x; i < N; i += gridDim.x * 256) {
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
    // Histories that can pass 8K tokens: eight CTAs a head (a slice each, counts joined across the
    // cluster); below, the passes are shorter than the cluster's barriers.
    const long long tokens = (long long)max_pages * L.page_size;
    const int C = tokens > 8192 ? kCluster : 1;
    const long long slice = (tokens + C - 1) / C;
    const int smem = 4 * (int)(slice < kCached ? slice : kCached);
    if (cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(evict_select_kernel), smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(C * L.n_kv_heads, batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    if (C > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = C;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    if (cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, C)) return e;
    const long long most = (tokens + 255) / 256;
    const long long want = (8 * 152 + batch * L.n_kv_heads - 1) / (batch * L.n_kv_heads);
    evict_move_kernel<<<dim3((unsigned)(want < most ? want : most), L.n_kv_heads, batch), 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace oscar
