// The accepted path of a tree of drafted tokens, and its rows moved together in every layer's BF16 pool.
//
// One CTA per (pool, request); each walks the request's tree on its own (a warp holds the tree's parents and tokens,
// eight nodes a lane, and finds a child by ballots), so no launch waits for another's path.
// A path's indices rise, so row i moves from position seq_len + path[i] to one at or before it.  A thread owns the same
// 16 bytes of every row: it reads a run of rows before it writes them, and what it writes lies before what it reads later.

#include "ptx.cuh"
#include "tree.cuh"

namespace oscar {
namespace {

constexpr int kPools = 64;                     // pools of one launch
constexpr int kThreads = 256;
constexpr int kRun = 8;                        // rows on their way a thread
constexpr int kNodes = OSCAR_TREE_MAX_NODES;

struct Pools {
    uint16_t *k[kPools], *v[kPools];
    int32_t n_pages[kPools];
};

struct AcceptArgs {
    AcceptInput in;
    TreeInput t;
    AcceptOutput out;
    const int32_t *pt;
    int max_pages, page_shift, n_kv;
    int first_pool;                            // of this launch: pool 0's CTAs write the outputs
    bool move;
    int32_t *status;
};

__global__ void __launch_bounds__(kThreads) accept_kernel(AcceptArgs a, const __grid_constant__ Pools pools) {
    __shared__ int path[kNodes], tok[kNodes], count;
    __shared__ int src_page[kNodes], dst_page[kNodes];
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    pdl_wait();
    int first;
    int n = read_nodes(a.t, b, a.status, first);
    const int T = a.in.seq_len[b];
    if (n > 0 && (T < 0 || T > 0x7fffffff - kNodes || (a.move && T + n > a.max_pages << a.page_shift))) {
        if (threadIdx.x == 0) flag_status(a.status, OSCAR_DEV_BAD_LENGTH);
        n = 0;
    }
    if (threadIdx.x < 32) {
        int par[kNodes / 32], dr[kNodes / 32];
#pragma unroll
        for (int i = 0; i < kNodes / 32; ++i) {
            const int j = 32 * i + lane;
            par[i] = j > 0 && j < n ? a.in.parents[first + j] : -1;
            dr[i] = j > 0 && j < n ? a.in.draft[first + j] : 0;
            if (par[i] >= j) par[i] = -1;
            if (j < n) tok[j] = a.in.target[first + j];
        }
        __syncwarp();
        int cur = 0, len = 0;
        while (cur >= 0 && len < n) {                      // indices rise along a path: n steps at most
            const int want = tok[cur];
            if (lane == 0) path[len] = cur;
            ++len;
            int next = -1;
#pragma unroll
            for (int i = 0; i < kNodes / 32; ++i) {
                if (next >= 0 || 32 * i >= n) break;
                const unsigned hit = __ballot_sync(0xffffffffu, par[i] == cur && dr[i] == want);
                if (hit) next = 32 * i + __ffs(hit) - 1;
            }
            cur = next;
        }
        if (lane == 0) count = len;
    }
    __syncthreads();
    const int len = count;
    if (blockIdx.x == 0 && a.first_pool == 0) {
        for (int i = threadIdx.x; i < a.out.stride; i += kThreads) {
            const size_t at = (size_t)b * a.out.stride + i;
            a.out.path[at] = i < len ? path[i] : -1;
            a.out.tokens[at] = i < len ? tok[path[i]] : -1;
        }
        if (threadIdx.x == 0) {
            a.out.accepted[b] = len;
            if (a.out.new_len) a.out.new_len[b] = T + len;
        }
    }
    if (!a.move) return;
    // physical pages of the path's rows; -1 where nothing is to move
    const int pool = blockIdx.x, n_pages = pools.n_pages[pool], in_page = (1 << a.page_shift) - 1;
    for (int i = threadIdx.x; i < len; i += kThreads) {
        int s = -1, d = -1;
        if (path[i] != i) {
            const int32_t *pt = a.pt + (size_t)b * a.max_pages;
            s = pt[(T + path[i]) >> a.page_shift];
            d = pt[(T + i) >> a.page_shift];
            if ((uint32_t)s >= (uint32_t)n_pages || (uint32_t)d >= (uint32_t)n_pages) {
                flag_status(a.status, OSCAR_DEV_BAD_BF16_PAGE);
                s = d = -1;
            }
        }
        src_page[i] = s;
        dst_page[i] = d;
    }
    __syncthreads();
    const int row16 = a.n_kv * (kHeadDim / 8);             // 16-byte pieces of a row
    for (int c = threadIdx.x; c < 2 * row16; c += kThreads) {
        uint4 *base = reinterpret_cast<uint4 *>(c < row16 ? pools.k[pool] : pools.v[pool]) + (c < row16 ? c : c - row16);
        for (int i0 = 1; i0 < len; i0 += kRun) {           // node 0 stays where it is
            uint4 x[kRun];
#pragma unroll
            for (int u = 0; u < kRun; ++u) {
                const int i = i0 + u;
                if (i < len && src_page[i] >= 0)
                    x[u] = base[(((size_t)src_page[i] << a.page_shift) + ((T + path[i]) & in_page)) * row16];
            }
#pragma unroll
            for (int u = 0; u < kRun; ++u) {
                const int i = i0 + u;
                if (i < len && src_page[i] >= 0) base[(((size_t)dst_page[i] << a.page_shift) + ((T + i) & in_page)) * row16] = x[u];
            }
        }
    }
}

}  // namespace

cudaError_t launch_tree_accept(const oscar_layout_t &L, const AcceptInput &in, const TreeInput &t, int batch, const AcceptOutput &out,
                               const oscar_bf16_pool_t *pools, int n_pools, const int32_t *pt, int max_pages, int32_t *status, cudaStream_t st) {
    AcceptArgs a{in, t, out, pt, max_pages, page_shift(L), L.n_kv_heads, 0, n_pools > 0, status};
    for (int i = 0; i == 0 || i < n_pools; i += kPools) {
        Pools p{};
        const int k = n_pools - i < kPools ? n_pools - i : kPools;
        for (int j = 0; j < k; ++j) {
            p.k[j] = pools[i + j].k;
            p.v[j] = pools[i + j].v;
            p.n_pages[j] = pools[i + j].n_pages;
        }
        a.first_pool = i;
        if (cudaError_t e = launch_ahead(accept_kernel, dim3(k > 0 ? k : 1, batch), kThreads, 0, st, a, p)) return e;
    }
    return cudaSuccess;
}

}  // namespace oscar
