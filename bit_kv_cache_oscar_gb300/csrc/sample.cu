// One token per row of logits by temperature, top-k, top-p, min-p and a given uniform number.
//
// Every filter keeps a prefix of the tokens in the order (falling logit, rising index), so what is kept is a pair
// (value v, index I): the logits above v, and those equal to v up to index I.  top-k and top-p are the same search, the
// shortest prefix whose weight reaches a target, with weight 1 or w; min-p is a value by itself.  Then the drawn token is
// one more search, in index order, for u of the kept weight.
//
// w = 2^-y, y = (m - x) log2(e) / T, is formed as a whole multiple of 2^-44: m - x exactly (a pair of floats), times a pair,
// split into whole and 256th parts (shift and table) and a rest |r| <= 2^-9 whose 2^-r - 1 takes three terms.  Sums of whole
// numbers have no order, so neither the number of CTAs nor atomics change a token, and are exact enough that u meets the same
// token as in 64-bit arithmetic (a sum in fp32, 2^-24 off, would miss for one row in a hundred over a large vocabulary).
//
// A cluster of 1 to 8 CTAs takes a row and holds it in shared memory, so a row is read once.  A search goes through bins: first
// 2,048 equal steps of y, whose order is the logits' order, then, within the bin that the target falls into, equal steps of the
// logits' bits until a bin is one value.  The entries of that first bin are gathered into a list, which the later levels read
// (unless they are too many: then the row again).  Weights in a bin are summed by 32-bit atomics on three parts of 15 bits.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "ptx.cuh"
#include "tree.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;                          // 4 a thread
constexpr float kDeep = 44.5f;                       // y from here on: weight zero
constexpr float kBinScale = kBins / kDeep;
constexpr int kList = 1024;                          // entries of a CTA's list
constexpr int kUnit = 44;                            // weights in units of 2^-44
constexpr int kLimb = 15;

struct SampleArgs {
    SampleInput in;
    int per;                                         // tokens of a CTA
    int32_t *tokens;
};

template <int TYPE> struct Type;
template <> struct Type<OSCAR_DTYPE_F32> {
    using raw = uint32_t;
    static __device__ __forceinline__ float get(uint4 v, int i) { return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w); }
    static __device__ __forceinline__ float one(uint32_t v) { return __uint_as_float(v); }
    static __device__ __forceinline__ uint32_t put(float f) { return __float_as_uint(f); }
};
template <> struct Type<OSCAR_DTYPE_BF16> {
    using raw = uint16_t;
    static __device__ __forceinline__ float get(uint4 v, int i) {
        const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
    static __device__ __forceinline__ float one(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t put(float f) { return (uint16_t)(__float_as_uint(f) >> 16); }     // exact here
};
template <> struct Type<OSCAR_DTYPE_F16> {
    using raw = uint16_t;
    static __device__ __forceinline__ float get(uint4 v, int i) {
        const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
        return __half2float(__ushort_as_half((uint16_t)(i & 1 ? w >> 16 : w)));
    }
    static __device__ __forceinline__ float one(uint16_t v) { return __half2float(__ushort_as_half(v)); }
    static __device__ __forceinline__ uint16_t put(float f) { return __half_as_ushort(__float2half_rn(f)); }
};

// Rising with falling x (-0 as +0).
__device__ __forceinline__ uint32_t falling_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? b : 0x7fffffffu - b;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k : 0x7fffffffu - k); }

struct Row {
    float top, ch, cl;                               // the largest logit; log2(e) / T as a pair
    float v;                                         // kept: x > v, or x == v and index <= I
    int I;
    const uint32_t *table;                           // 2^31 2^(-j / 256)
    __device__ __forceinline__ float depth(float x) const { return x == top ? 0.f : __fmul_rn(__fsub_rn(top, x), ch); }
    __device__ __forceinline__ bool kept(float x, int i) const { return x > v || (x == v && i <= I); }
    __device__ __forceinline__ uint64_t weight(float x) const {
        if (x == top) return 1ull << kUnit;
        const float d = __fsub_rn(top, x), bb = __fsub_rn(d, top);
        const float dl = __fsub_rn(__fsub_rn(top, __fsub_rn(d, bb)), __fadd_rn(x, bb));      // what d lacks, exactly
        const float y = __fmul_rn(d, ch);
        if (!(y < kDeep)) return 0;                  // NaN among them: infinite d, or no d and an infinite temperature's 0
        const float yl = __fmaf_rn(dl, ch, __fmaf_rn(d, cl, __fmaf_rn(d, ch, -y)));
        const float t = __fmaf_rn(y, 256.f, 12582912.f);
        const int k = __float_as_int(t) - 0x4B400000;
        const float r = __fadd_rn(__fmaf_rn(__fsub_rn(t, 12582912.f), -0x1p-8f, y), yl);
        // 2^-r - 1 = -a + a^2/2 - a^3/6 with a = r ln 2; the next term is below 2^-42
        const float p = __fmul_rn(r, __fmaf_rn(r, __fmaf_rn(r, -0.0555041087f, 0.240226507f), -0.693147181f));
        const uint32_t up = 0x80000000u + (uint32_t)(__float_as_int(__fmaf_rn(p, 0x1p31f, 12582912.f)) - 0x4B400000);
        return ((uint64_t)table[k & 255] * up) >> (62 - kUnit + (k >> 8));
    }
};

struct Shared {
    uint32_t hist[4][kBins];                         // counts, weights' three parts
    uint32_t table[256];
    uint32_t list_key[kList];
    uint64_t warp_sum[kWarps];                       // read by the cluster
    uint64_t scan[kWarps];
    float warp_top[kWarps];
    float top;                                       // of this CTA, read by the cluster
    uint32_t n_list, key_min, key_max;               // read by the cluster
    int pick_index;
    uint32_t bin;
    uint64_t before;
};

// A value of another CTA of the cluster.
template <typename T>
__device__ __forceinline__ T peer(const T *p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr(p)), "r"(rank));
    if constexpr (sizeof(T) == 8) {
        uint64_t x;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(r) : "memory");
        return (T)x;
    } else {
        uint32_t x;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(r) : "memory");
        T v;
        memcpy(&v, &x, 4);
        return v;
    }
}
__device__ __forceinline__ uint4 peer4(const uint32_t *p, int rank) {
    uint32_t r;
    uint4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(r) : "memory");
    return v;
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ uint64_t warp_scan64(uint64_t x, int lane) {          // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}
__device__ __forceinline__ void cluster_join() {
    __syncwarp();
    cluster_sync_all();
}

// The part of the row that this CTA holds: whole vectors, element e of vector j with index begin - skip + j VE + e; the
// places before and behind the part hold -inf.
template <int TYPE>
struct Part {
    using T = Type<TYPE>;
    static constexpr int VE = 16 / (int)sizeof(typename T::raw);
    const uint4 *vec;
    int nv, begin, skip;
    int C, rank;

    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        for (int j = threadIdx.x; j < nv; j += kThreads) {
            const uint4 x = vec[j];
            const int i0 = begin - skip + j * VE;
#pragma unroll
            for (int e = 0; e < VE; ++e) f(T::get(x, e), i0 + e);
        }
    }

    // The lowest index at which the running sum of f in index order reaches the target that goal(total) gives, kept within
    // 1 .. total; -1 where the total is 0.  All threads of all CTAs return it.
    template <typename F, typename G>
    __device__ __forceinline__ int pick(Shared &s, F f, G goal) const {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int lo = (int)((long long)nv * warp / kWarps), hi = (int)((long long)nv * (warp + 1) / kWarps);
        uint64_t sum = 0;
        for (int j = lo + lane; j < hi; j += 32) {
            const uint4 x = vec[j];
            const int i0 = begin - skip + j * VE;
#pragma unroll
            for (int e = 0; e < VE; ++e) sum += f(T::get(x, e), i0 + e);
        }
        sum = warp_sum64(sum);
        if (lane == 0) s.warp_sum[warp] = sum;
        if (threadIdx.x == 0) s.pick_index = -1;
        cluster_join();
        // every warp: sums before its own, and all
        uint64_t before = 0, total = 0;
        for (int k = lane; k < C * kWarps; k += 32) {
            const uint64_t x = peer(&s.warp_sum[k % kWarps], k / kWarps);
            total += x;
            if (k < rank * kWarps + warp) before += x;
        }
        before = warp_sum64(before);
        total = warp_sum64(total);
        uint64_t target = goal(total);
        target = target < 1 ? 1 : target > total ? total : target;
        if (total > 0 && before < target && target <= before + sum) {        // one warp of the cluster
            for (int j0 = lo; j0 < hi; j0 += 32) {
                const int j = j0 + lane;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (j < hi) x = vec[j];
                const int i0 = begin - skip + j * VE;
                uint64_t mine = 0;
#pragma unroll
                for (int e = 0; e < VE; ++e) mine += j < hi ? f(T::get(x, e), i0 + e) : 0;
                if (!__any_sync(0xffffffffu, mine > 0)) continue;
                const uint64_t upto = before + warp_scan64(mine, lane);
                const unsigned reached = __ballot_sync(0xffffffffu, upto >= target);
                if (reached) {
                    if (lane == __ffs(reached) - 1) {
                        uint64_t at = upto - mine;
                        int found = -1;
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            at += f(T::get(x, e), i0 + e);
                            if (found < 0 && at >= target) found = i0 + e;
                        }
                        s.pick_index = found;
                    }
                    break;
                }
                before = __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        cluster_join();
        int found = -1;
        for (int k = 0; k < C; ++k) found = max(found, peer(&s.pick_index, k));
        cluster_join();                              // read before they are written again
        return found;
    }

    // The bins of this search level, filled by every CTA: finds the first one up to which base and the weights reach the
    // target that goal(total) gives, and leaves it in s.bin with the weight before it in s.before.  False: no bin does.
    template <bool MASS, typename G>
    __device__ __forceinline__ bool find_bin(Shared &s, uint64_t base, G goal) const {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b0 = threadIdx.x * 4;
        cluster_join();
        uint64_t w[4] = {0, 0, 0, 0};
        for (int k = 0; k < C; ++k) {
            if (MASS) {
#pragma unroll
                for (int l = 0; l < 3; ++l) {
                    const uint4 h = peer4(&s.hist[1 + l][b0], k);
                    w[0] += (uint64_t)h.x << (kLimb * l);
                    w[1] += (uint64_t)h.y << (kLimb * l);
                    w[2] += (uint64_t)h.z << (kLimb * l);
                    w[3] += (uint64_t)h.w << (kLimb * l);
                }
            } else {
                const uint4 h = peer4(&s.hist[0][b0], k);
                w[0] += h.x;
                w[1] += h.y;
                w[2] += h.z;
                w[3] += h.w;
            }
        }
        const uint64_t mine = w[0] + w[1] + w[2] + w[3];
        const uint64_t upto = warp_scan64(mine, lane);
        if (lane == 31) s.scan[warp] = upto;
        if (threadIdx.x == 0) s.bin = kBins;
        __syncthreads();
        uint64_t before = base, total = 0;
        for (int k = 0; k < kWarps; ++k) {
            const uint64_t x = s.scan[k];
            if (k < warp) before += x;
            total += x;
        }
        const uint64_t target = goal(total);
        before += upto - mine;
        if (before < target && target <= before + mine) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (before < target && target <= before + w[i]) {
                    s.bin = b0 + i;
                    s.before = before;
                }
                before += w[i];
            }
        }
        cluster_join();                              // found, and the bins read by all
        return s.bin < kBins;
    }

    __device__ __forceinline__ void clear(Shared &s) const {
        uint4 *h = reinterpret_cast<uint4 *>(s.hist);
        for (int i = threadIdx.x; i < 4 * kBins / 4; i += kThreads) h[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    template <bool MASS>
    static __device__ __forceinline__ void add(Shared &s, int bin, uint64_t w) {
        if (MASS) {
            atomicAdd(&s.hist[1][bin], (uint32_t)w & ((1u << kLimb) - 1));
            atomicAdd(&s.hist[2][bin], (uint32_t)(w >> kLimb) & ((1u << kLimb) - 1));
            atomicAdd(&s.hist[3][bin], (uint32_t)(w >> (2 * kLimb)));
        } else {
            atomicAdd(&s.hist[0][bin], 1u);
        }
    }

    // Narrows what is kept to the shortest prefix whose weight (1 a token, or w) reaches the target.
    template <bool MASS, typename G>
    __device__ __forceinline__ void cut(Shared &s, Row &row, G goal) const {
        clear(s);
        each([&](float x, int i) {
            const float y = row.depth(x);
            if (y < kDeep && row.kept(x, i)) {
                const uint64_t w = MASS ? row.weight(x) : 1;
                if (w) add<MASS>(s, min((int)(y * kBinScale), kBins - 1), w);
            }
        });
        uint64_t target = 0;
        if (!find_bin<MASS>(s, 0, [&](uint64_t total) { return target = goal(total); })) return;
        const int bin = s.bin;
        uint64_t before = s.before;
        auto in_bin = [&](float x, int i) {
            const float y = row.depth(x);
            return y < kDeep && min((int)(y * kBinScale), kBins - 1) == bin && row.kept(x, i);
        };
        // the bin's entries and the range of their keys
        if (threadIdx.x == 0) {
            s.n_list = 0;
            s.key_min = 0xffffffffu;
            s.key_max = 0;
        }
        __syncthreads();
        uint32_t lo = 0xffffffffu, hi = 0;
        each([&](float x, int i) {
            if (!in_bin(x, i)) return;
            const uint32_t k = falling_key(x);
            lo = min(lo, k);
            hi = max(hi, k);
            const uint32_t at = atomicAdd(&s.n_list, 1u);
            if (at < kList) s.list_key[at] = k;
        });
        __syncwarp();
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if ((threadIdx.x & 31) == 0) {
            atomicMin(&s.key_min, lo);
            atomicMax(&s.key_max, hi);
        }
        cluster_join();
        lo = 0xffffffffu;
        hi = 0;
        for (int k = 0; k < C; ++k) {
            lo = min(lo, peer(&s.key_min, k));
            hi = max(hi, peer(&s.key_max, k));
        }
        const uint32_t n = s.n_list;
        for (;;) {
            const int shift = hi > lo ? max(0, 32 - __clz(hi - lo) - 11) : 0;          // (hi - lo) >> shift < 2048
            clear(s);
            auto count = [&](uint32_t k) {
                if (k >= lo && k <= hi) add<MASS>(s, (k - lo) >> shift, MASS ? row.weight(key_value(k)) : 1);
            };
            if (n <= kList)
                for (uint32_t i = threadIdx.x; i < n; i += kThreads) count(s.list_key[i]);
            else
                each([&](float x, int i) {
                    if (in_bin(x, i)) count(falling_key(x));
                });
            if (!find_bin<MASS>(s, before, [&](uint64_t) { return target; })) return;         // (the bin's sum reaches it: does not happen)
            before = s.before;
            lo += s.bin << shift;
            if (!shift) break;
            hi = min(hi, lo + ((1u << shift) - 1));
        }
        // one value left: the first ties of it
        const float v = key_value(lo);
        const uint64_t each_w = MASS ? row.weight(v) : 1, ties = (target - before + each_w - 1) / each_w;
        row.I = pick(s, [&](float x, int i) -> uint64_t { return x == v && row.kept(x, i); }, [&](uint64_t) { return ties; });
        row.v = v;
    }
};

template <int TYPE>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a) {
    using T = Type<TYPE>;
    using raw = typename T::raw;
    constexpr int VE = Part<TYPE>::VE;
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    uint4 *data = reinterpret_cast<uint4 *>(smem + ((sizeof(Shared) + 15) & ~size_t(15)));
    const int C = gridDim.x, rank = blockIdx.x, r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < 256) s.table[threadIdx.x] = threadIdx.x ? (uint32_t)__double2ull_rn(exp2(31.0 - threadIdx.x / 256.0)) : 0x80000000u;
    pdl_wait();
    const int begin = min(a.in.vocab, rank * a.per), n = min(a.in.vocab, begin + a.per) - begin;
    const raw *src = static_cast<const raw *>(a.in.logits) + (size_t)r * a.in.stride + begin;
    const int skip = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(raw));
    const Part<TYPE> part{data, (skip + n + VE - 1) / VE, begin, skip, C, rank};
    // the row's part to shared memory, NaN as -inf, and its largest
    float top = -INFINITY;
    {
        const raw *from = src - skip;                        // 16-byte aligned; only whole vectors inside the part are read
        auto whole = [&](int j) { return j * VE >= skip && (j + 1) * VE <= skip + n; };
        constexpr int U = 4;
        for (int j0 = threadIdx.x; j0 < part.nv; j0 += U * kThreads) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + u * kThreads;
                if (j < part.nv && whole(j)) x[u] = __ldg(reinterpret_cast<const uint4 *>(from) + j);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + u * kThreads;
                if (j >= part.nv) continue;
                raw y[VE];
                if (whole(j)) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float f = fmaxf(T::get(x[u], e), -INFINITY);
                        top = fmaxf(top, f);
                        y[e] = T::put(f);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const int i = j * VE + e;
                        const float f = i >= skip && i < skip + n ? fmaxf(T::one(from[i]), -INFINITY) : -INFINITY;
                        top = fmaxf(top, f);
                        y[e] = T::put(f);
                    }
                }
                memcpy(&data[j], y, 16);
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s.warp_top[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < kWarps; ++k) top = fmaxf(top, s.warp_top[k]);
        s.top = top;
    }
    cluster_join();
    top = -INFINITY;
    for (int k = 0; k < C; ++k) top = fmaxf(top, peer(&s.top, k));
    const float temp = a.in.temperature[r];
    int token = -1;
    if (top > -INFINITY) {
        auto first_of_top = [&] { return part.pick(s, [&](float x, int) -> uint64_t { return x == top; }, [](uint64_t) -> uint64_t { return 1; }); };
        if (!(temp > 0.f)) {
            token = first_of_top();
        } else {
            Row row;
            const double c = fmin(1.4426950408889634 / (double)temp, 0x1p120);
            row.top = top;
            row.ch = (float)c;
            row.cl = (float)(c - (double)row.ch);
            row.v = -INFINITY;
            row.I = 0x7fffffff;
            row.table = s.table;
            const int k = a.in.top_k ? a.in.top_k[r] : 0;
            if (k > 0 && k < a.in.vocab) part.template cut<false>(s, row, [&](uint64_t) -> uint64_t { return k; });
            const float p = a.in.top_p ? a.in.top_p[r] : 1.f;
            if (p < 1.f) {
                // the least whole number that is at least p of the total
                const uint64_t p64 = (uint64_t)((double)fmaxf(p, 0.f) * 0x1p64);
                part.template cut<true>(s, row, [&](uint64_t total) -> uint64_t {
                    const uint64_t t = __umul64hi(total, p64) + (total * p64 != 0);
                    return t < 1 ? 1 : t;
                });
            }
            const float mp = a.in.min_p ? a.in.min_p[r] : 0.f;
            if (mp > 1.f) {                              // no weight is that large: the first token of the order
                row.I = first_of_top();
                row.v = top;
            } else if (mp > 0.f) {
                const double least = mp == 1.f || top == INFINITY ? (double)top : (double)top + (double)temp * log((double)mp);
                const float v = __double2float_ru(least);
                if (v > row.v) {
                    row.v = v;
                    row.I = 0x7fffffff;
                }
            }
            const float u = fminf(fmaxf(a.in.u[r], 0.f), 0x1.fffffep-1f);
            const uint64_t u64 = (uint64_t)((double)u * 0x1p64);
            token = part.pick(s, [&](float x, int i) -> uint64_t { return row.kept(x, i) ? row.weight(x) : 0; },
                              [&](uint64_t total) -> uint64_t { return __umul64hi(total, u64) + 1; });
        }
    }
    if (rank == 0 && threadIdx.x == 0) a.tokens[r] = token;
    cluster_join();                                      // no CTA ends while another reads its memory
}

template <int TYPE>
cudaError_t launch_type(const SampleArgs &a, int C, int smem, cudaStream_t st) {
    auto kern = sample_kernel<TYPE>;
    if (cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(kern), smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(C, a.in.rows);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_sample(const SampleInput &in, int32_t *tokens, cudaStream_t st) {
    // CTAs a row: as many as leave room for two on an SM, and more (8 at most) while the rows leave SMs idle and a CTA
    // has 2,048 tokens or more
    const int size = in.dtype == OSCAR_DTYPE_F32 ? 4 : 2;
    const int room = 112 * 1024 - (int)sizeof(Shared) - 64;
    int C = 1;
    while (C < 8 && (in.vocab + C - 1) / C * size > room) C *= 2;
    while (C < 8 && (long long)in.rows * C * 2 <= 304 && in.vocab / (2 * C) >= 2048) C *= 2;
    SampleArgs a{in, (in.vocab + C - 1) / C, tokens};
    const int smem = (int)((sizeof(Shared) + 15) & ~size_t(15)) + ((a.per + 2 * (16 / size)) * size + 15) / 16 * 16;
    switch (in.dtype) {
        case OSCAR_DTYPE_F32: return launch_type<OSCAR_DTYPE_F32>(a, C, smem, st);
        case OSCAR_DTYPE_BF16: return launch_type<OSCAR_DTYPE_BF16>(a, C, smem, st);
        default: return launch_type<OSCAR_DTYPE_F16>(a, C, smem, st);
    }
}

}  // namespace oscar
