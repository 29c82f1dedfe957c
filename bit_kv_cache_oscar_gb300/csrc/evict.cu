// Eviction from the INT4 history by accumulated weight: which positions stay, and the move of their rows.
//
// For each (request, kv head) the `keep` positions of largest weight in [sink, hist_end) are kept, ties
// going to the lowest position.  The weights are mapped to integers of the same order and the keep-th
// largest is found digit by digit from the top (histogram of the digit among the values that match the
// digits found so far, then the bin where the count from above reaches keep).  A position stays if its
// value is above that threshold, or equal to it and among the first `keep - above` equal ones.  The
// positions come out in order because each warp takes a run of them and knows the counts before its run.
// A second kernel copies the kept rows to their new pages, 8 lanes a row.
//
// Measured, two requests of 67K to 100K tokens, 8 kv heads, half kept: selection 31 us (latency: three passes
// of a histogram in shared memory, a cluster's barriers and remote reads; 7 MB are read), move 47 us = 4.0 TB/s
// (latency: list entry, page ids and data depend on each other).

#include <algorithm>

#include "int4.cuh"
#include "ptx.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;                 // digits of 11, 10 and 11 bits
constexpr int kCached = 16384;              // keys of a CTA's slice held in shared memory
constexpr int kCluster = 8;

struct EvictArgs {
    Int4PoolView src, dst;
    const int32_t *spt, *dpt;
    int max_pages, page_shift, n_kv, group, sink;
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
    const int t0 = a.seq_len[b], h0 = a.hist_end[b];           // all three on their way at once
    if (k == -1) return false;
    if (t0 < 0 || h0 < 0 || h0 > t0 || t0 > (a.max_pages << a.page_shift) || (h0 < a.sink && t0 >= a.sink)) {
        read_lengths(a.seq_len, a.hist_end, b, a.sink, a.max_pages << a.page_shift, a.status, T, he);
    } else {
        T = t0;
        he = max(h0, min(a.sink, t0));
    }
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

__device__ __forceinline__ void st_cluster(int *p, int rank, int v) {
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(saddr(p)), "r"(rank));
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(ra), "r"(v) : "memory");
}

// One cluster of C CTAs (grid x = C·Hkv) per (request, kv head); CTA r takes the slice [r n / C, (r + 1) n / C)
// of the history and holds its keys in shared memory (kCached of them; the rest is read again each pass).
// A pass: each CTA counts its slice's digits, sums its share of the bins over the cluster (all C remote
// reads in flight), sends the sums to every CTA, and each finds the digit among all the bins by itself.
template <int C>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a) {
    extern __shared__ uint32_t keys[];
    constexpr int kOwn = kBins / kThreads;             // bins of one thread in the search
    // four counters a bin (lane & 3): weights gather in few bins, and equal bins of a warp are added in turn
    __shared__ int4 hist[kBins];
    __shared__ int tot[C > 1 ? kBins : 1];             // the cluster's counts
    __shared__ int cnt_gt[kWarps], cnt_eq[kWarps], red[kWarps];
    __shared__ int found[2], slice_gt, slice_eq;
    const int rank = blockIdx.x % C, h = blockIdx.x / C, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto cluster_or_cta_sync = [] {
        if (C > 1) cluster_sync_all();
        else __syncthreads();
    };
    pdl_wait();
    pdl_trigger();                                     // the move may be set up meanwhile; it waits for this grid
    int T, he, n, k;
    if (!read_request(a, b, T, he, n, k, threadIdx.x == 0 && blockIdx.x == 0) || k == 0) return;     // the whole cluster alike
    const int lo = (int)((long long)rank * n / C), hi = (int)((long long)(rank + 1) * n / C);
    const float *m = a.mass + (((size_t)b * a.n_kv + h) * a.max_pages << a.page_shift) + a.sink + lo;
    const int len = hi - lo, cached = min(len, kCached);
    auto key_at = [&](int i) { return i < cached ? keys[i] : order_key(m[i]); };
#pragma unroll 8
    for (int i = threadIdx.x; i < cached; i += kThreads) keys[i] = order_key(m[i]);

    int *counters = reinterpret_cast<int *>(hist);
    uint32_t prefix = 0;
    int left = k;                                      // still to find among the keys that match the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 11 : 0, nb = pass == 1 ? 1024 : 2048;
        const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFF800u;
        for (int i = threadIdx.x; i < nb; i += kThreads) hist[i] = make_int4(0, 0, 0, 0);
        __syncthreads();
        auto count = [&](uint32_t key) {
            if ((key & mask) == prefix) atomicAdd(&counters[4 * ((key >> shift) & (nb - 1)) + (lane & 3)], 1);
        };
#pragma unroll 4
        for (int i = threadIdx.x; i < cached; i += kThreads) count(keys[i]);
        for (int i = cached + threadIdx.x; i < len; i += kThreads) count(order_key(m[i]));
        __syncthreads();
        const int per = nb / C;
        for (int i = threadIdx.x; i < nb; i += kThreads) {
            const int4 v = hist[i];
            hist[i].x = v.x + v.y + v.z + v.w;
        }
        cluster_or_cta_sync();
        if (C > 1) {
            for (int i = threadIdx.x; i < per; i += kThreads) {
                int v[C], t = 0;
#pragma unroll
                for (int r = 0; r < C; ++r) v[r] = ld_cluster(&hist[rank * per + i].x, r);
#pragma unroll
                for (int r = 0; r < C; ++r) t += v[r];
#pragma unroll
                for (int r = 0; r < C; ++r) st_cluster(&tot[rank * per + i], r, t);
            }
            cluster_sync_all();
        }
        // the digit: bins from the top, kOwn a thread
        int c[kOwn], sum = 0;
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int i = nb - 1 - (int)(threadIdx.x * kOwn + j);
            c[j] = i < 0 ? 0 : C > 1 ? tot[i] : hist[i].x;
            sum += c[j];
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) red[warp] = upto;
        __syncthreads();
        const int before0 = __reduce_add_sync(0xffffffffu, lane < warp ? red[lane & (kWarps - 1)] : 0);
        int before = upto - sum + before0;
        if (before < left && left <= before + sum) {
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                if (before < left && left <= before + c[j]) {
                    found[0] = nb - 1 - (int)(threadIdx.x * kOwn + j);
                    found[1] = left - before;
                    break;
                }
                before += c[j];
            }
        }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        left = found[1];
    }

    // places: warp w takes [w len / W, (w + 1) len / W) of the slice; counts first, then positions in order
    const int w0 = (int)((long long)warp * len / kWarps), w1 = (int)((long long)(warp + 1) * len / kWarps);
    int gt = 0, eq = 0;
#pragma unroll 4
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
    if (warp == 0) {
        const int x = __reduce_add_sync(0xffffffffu, lane < kWarps ? cnt_gt[lane & (kWarps - 1)] : 0);
        const int y = __reduce_add_sync(0xffffffffu, lane < kWarps ? cnt_eq[lane & (kWarps - 1)] : 0);
        if (lane == 0) {
            slice_gt = x;
            slice_eq = y;
        }
    }
    cluster_or_cta_sync();
    int gt0 = 0, eq0 = 0;
    if (C > 1) {
        int v[C], w[C];
#pragma unroll
        for (int r = 0; r < C; ++r) {
            v[r] = ld_cluster(&slice_gt, r);
            w[r] = ld_cluster(&slice_eq, r);
        }
#pragma unroll
        for (int r = 0; r < C; ++r) {
            gt0 += r < rank ? v[r] : 0;
            eq0 += r < rank ? w[r] : 0;
        }
    }
    gt0 += __reduce_add_sync(0xffffffffu, lane < warp ? cnt_gt[lane & (kWarps - 1)] : 0);
    eq0 += __reduce_add_sync(0xffffffffu, lane < warp ? cnt_eq[lane & (kWarps - 1)] : 0);
    int32_t *out = a.kept + ((size_t)b * a.n_kv + h) * a.kept_stride;
    const uint32_t below = (1u << lane) - 1;
#pragma unroll 4
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

// grid (X, Hkv, batch).  A row is 8 lanes: 4 with the key's 64 bytes, 4 with the value's.  List entry, page
// ids and data depend on each other, and what hides that is many warps with few registers each: one row a
// thread at a time and sixteen CTAs an SM, the next entry asked into L1 meanwhile (8 x 100K to half, read back:
// 588 us; without that 596; the next entry held in a register, 40 of them: 607.  2 x 100K: 149; four rows a thread,
// eight CTAs: 153; the next rows' entries and pages loaded ahead, four CTAs: 191).
__global__ void __launch_bounds__(256) evict_move_kernel(EvictArgs a) {
    const int h = blockIdx.y, b = blockIdx.z, hl = threadIdx.x & 7;
    int T, he, n, k;
    pdl_wait();                                        // the selection is complete
    if (!read_request(a, b, T, he, n, k, false)) return;
    const size_t row0 = ((size_t)b * a.n_kv + h) * a.max_pages << a.page_shift;
    const int32_t *kept = a.kept + ((size_t)b * a.n_kv + h) * a.kept_stride;
    const int32_t *spt = a.spt + (size_t)b * a.max_pages, *dpt = a.dpt + (size_t)b * a.max_pages;
    const int G = kHeadDim / a.group, step = gridDim.x * 32, in_page = (1 << a.page_shift) - 1;
    const uint8_t *sc = hl < 4 ? a.src.codes_k : a.src.codes_v;
    uint8_t *dc = hl < 4 ? a.dst.codes_k : a.dst.codes_v;
    for (long long j = blockIdx.x * 32 + (threadIdx.x >> 3); j < k; j += step) {
        const int p = kept[j], to = a.sink + (int)j;
        if (j + step < k) asm volatile("prefetch.global.L1 [%0];" ::"l"(kept + j + step));
        const int sp = spt[p >> a.page_shift], dp = dpt[to >> a.page_shift];
        if (hl == 0) a.mass_out[row0 + to] = a.mass[row0 + p];
        if ((uint32_t)sp >= (uint32_t)a.src.n_pages || (uint32_t)dp >= (uint32_t)a.dst.n_pages) {
            if (hl == 0) flag_status(a.status, OSCAR_DEV_BAD_INT4_PAGE);
            continue;
        }
        const size_t from = row4(sp, a.n_kv, h, a.page_shift, p & in_page), at = row4(dp, a.n_kv, h, a.page_shift, to & in_page);
        const uint4 x = reinterpret_cast<const uint4 *>(sc + from * kRow4)[hl & 3];
        uint2 z = make_uint2(0, 0);
        if (hl < G) z = reinterpret_cast<const uint2 *>(a.src.scale_zero)[from * G + hl];
        reinterpret_cast<uint4 *>(dc + at * kRow4)[hl & 3] = x;
        if (hl < G) reinterpret_cast<uint2 *>(a.dst.scale_zero)[at * G + hl] = z;
    }
    // the weights outside the kept rows: sink, recent rows, nothing behind them
    const int N = a.max_pages << a.page_shift, shift = n - k, lo = min(a.sink, T);
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
    const EvictArgs a{src, dst, spt, dpt, max_pages, page_shift(L), L.n_kv_heads, L.group, L.sink, seq_len, hist_end, keep,
                      mass, mass_out, kept, kept_stride, status};
    // Long histories of few heads: eight CTAs a head, a slice each, counts joined across the cluster.  Short ones
    // are done before a cluster's barriers are, and many heads fill the SMs by themselves: one CTA a head.  Whole
    // call, 8 heads, one and eight CTAs: 6K tokens 20.8 and 22.2 us, 9K 23.0 and 23.6, 16K 29.0 and 24.9; 64
    // heads, 16K 37 and 46, 40K 95 and 66; 128 heads, 40K 106 and 107; 256 heads, 40K 142 and 197.
    const long long tokens = (long long)max_pages * L.page_size, pairs = (long long)batch * L.n_kv_heads;
    const int C = tokens > 256 * std::max(32LL, pairs) ? kCluster : 1;
    const long long slice = (tokens + C - 1) / C;
    const int smem = 4 * (int)(slice < kCached ? slice : kCached);
    auto kern = C > 1 ? evict_select_kernel<kCluster> : evict_select_kernel<1>;
    if (cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(kern), smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(C * L.n_kv_heads, batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    if (cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a)) return e;
    // CTAs: about sixteen an SM, no more than there are runs of 32 rows
    const long long most = (tokens + 31) / 32, want = (16 * 152 + pairs - 1) / pairs;
    return launch_ahead(evict_move_kernel, dim3((unsigned)(want < most ? want : most), L.n_kv_heads, batch), 256, 0, st, a);
}

}  // namespace oscar
