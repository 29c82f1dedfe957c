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
// A cluster of 1 to 8 CTAs takes a row and holds it in shared memory, so a row is read once.  The filters' search goes through
// bins: 4,096 equal steps of y, whose order is the logits' order, counted by atomics.  For top-k the counts give the bin that the
// target falls into; for top-p, with the sum of all weights, the few bins that it can fall into (a bin's weights differ by 0.8 %).
// Where no more than 2,048 entries lie up to there, they go to the first CTA, which sorts them, cuts the order by every filter, sorts
// what is left by index and draws.  Where that many lie in those bins alone, it sorts these and says where the cut is, and the draw
// goes through the row.  Where more do (flat rows), further levels of bins follow, within a bin equal steps of the logits' bits, until
// a bin is one value; weights in a bin are then summed by 32-bit atomics on three parts of 15 bits.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "pairs.cuh"
#include "ptx.cuh"
#include "tree.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr float kDeep = 44.5f;                       // y from here on: weight zero
// Bins of counts, and of weights.
template <bool MASS> constexpr int kBins = MASS ? 2048 : 4096;
template <bool MASS> constexpr float kBinScale = kBins<MASS> / kDeep;
template <bool MASS>
__device__ __forceinline__ uint32_t bin_of(float y) { return (uint32_t)min((int)(y * kBinScale<MASS>), kBins<MASS> - 1); }
constexpr int kList = 2048;                          // entries that one CTA sorts
constexpr int kKeys = 1024;                          // entries of a CTA's list for the further levels
constexpr int kUnit = 44;                            // weights in units of 2^-44
constexpr int kLimb = 15;

// 2^31 2^(-j / 256), each within 2^-17 of a unit before its rounding (256 products in 64 bits).
struct Table {
    uint32_t t[256];
    constexpr Table() : t() {
        double x = 2147483648.0;
        for (int j = 0; j < 256; ++j, x *= 0.99729605608547012625765991384792) t[j] = (uint32_t)(x + 0.5);
    }
};
__device__ constexpr Table kTable{};

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
    // Weights of two logits.
    __device__ __forceinline__ void weights(float xa, float xb, uint64_t &wa, uint64_t &wb) const {
        const f2 minus = pair(-1.f, -1.f), x = pair(xa, xb), t = pair(top, top), magic = pair(12582912.f, 12582912.f);
        const f2 d = fma2(x, minus, t), bb = add2(d, pair(-top, -top));
        // what d lacks, exactly: (top - (d - bb)) - (x + bb)
        const f2 dl = fma2(add2(x, bb), minus, fma2(fma2(bb, minus, d), minus, t));
        const f2 c = pair(ch, ch), ny = mul2(d, pair(-ch, -ch));                              // -y, and what it lacks
        const f2 yl = fma2(dl, c, fma2(d, pair(cl, cl), fma2(d, c, ny)));
        const f2 kt = fma2(ny, pair(-256.f, -256.f), magic);
        // -r; 2^-r - 1 = -a + a^2/2 - a^3/6 with a = r ln 2; the next term is below 2^-42
        const f2 nr = fma2(yl, minus, fma2(add2(kt, pair(-12582912.f, -12582912.f)), pair(0x1p-8f, 0x1p-8f), ny));
        const f2 p = mul2(nr, fma2(nr, fma2(nr, pair(0.0555041087f, 0.0555041087f), pair(0.240226507f, 0.240226507f)), pair(0.693147181f, 0.693147181f)));
        const f2 q = fma2(p, pair(0x1p31f, 0x1p31f), magic);
        float na, nb, ka, kb, qa, qb;
        unpair(ny, na, nb);
        unpair(kt, ka, kb);
        unpair(q, qa, qb);
        auto whole = [&](float xx, float n, float k, float m) -> uint64_t {
            // NaN among the depths: infinities less themselves or by 0
            if (!(n > -kDeep)) return xx == top ? 1ull << kUnit : 0;
            const uint32_t kb = __float_as_uint(k);                        // 0x4B400000 + k
            return ((uint64_t)table[kb & 255] * (__float_as_uint(m) + (0x80000000u - 0x4B400000u))) >> (62 - kUnit + ((kb >> 8) & 63));
        };
        wa = whole(xa, na, ka, qa);
        wb = whole(xb, nb, kb, qb);
    }
    __device__ __forceinline__ uint64_t weight(float x) const {
        uint64_t a, b;
        weights(x, x, a, b);
        return a;
    }
};

struct Shared {
    union alignas(16) {                              // (cleared 16 bytes at a time)
        uint32_t count[kBins<false>];
        uint32_t mass[3][kBins<true>];               // weights' three parts
        struct {
            uint64_t list[kList], weight[kList];     // entries to sort; their weights
        };
        uint64_t steps[kWarps][32];                  // sums of each warp's steps through its vectors
    };
    uint32_t table[256];
    uint32_t list_key[kKeys];
    uint64_t warp_sum[kWarps];                       // read by the cluster
    uint64_t scan[kWarps];
    float warp_top[kWarps];
    float top;                                       // of this CTA, read by the cluster
    uint32_t n_list, key_min, key_max;               // read by the cluster
    uint32_t n_some, n_all, cursor;
    int pick_index;
    uint32_t bin, bin_from, bin_behind;
    uint64_t before, total, slice;
    float cut_v;                                     // of the first CTA, read by the cluster
    int cut_i;
    // the row's arguments
    float temp, ch, cl;
    int top_k, min_mode;                             // min_p: 0 off, 1 top + min_off, 2 the largest logit, 3 one token
    uint64_t p64, u64;
    bool top_p;
    double min_off;
};
constexpr int kSharedBytes = (sizeof(Shared) + 15) / 16 * 16;

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

// The n entries of s.list (falling key | index) sorted upwards, the places behind them up to the next power of two filled up.
__device__ __forceinline__ void sort_list(Shared &s, int n) {
    int size = 2;
    while (size < n) size *= 2;
    for (int i = n + threadIdx.x; i < size; i += kThreads) s.list[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= size; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
            for (int i = threadIdx.x; i < size / 2; i += kThreads) {
                const int x = 2 * i - (i & (j - 1)), y = x + j;
                const uint64_t u = s.list[x], v = s.list[y];
                if ((u > v) == ((x & k) == 0)) {
                    s.list[x] = v;
                    s.list[y] = u;
                }
            }
            if (j > 32 || size > 2 * kThreads) __syncthreads();
            else if (j > 1) __syncwarp();            // the next step's pairs of a warp are its own
            else __syncthreads();
        }
}

// Inclusive sums of four values a thread over the CTA, in thread order.
__device__ __forceinline__ void block_scan(Shared &s, uint64_t (&x)[4]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    x[1] += x[0];
    x[2] += x[1];
    x[3] += x[2];
    uint64_t before = warp_scan64(x[3], lane);
    if (lane == 31) s.scan[warp] = before;
    before -= x[3];
    __syncthreads();
    for (int k = 0; k < warp; ++k) before += s.scan[k];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] += before;
    __syncthreads();
}

// Where the prefix of a row's order that reaches the target ends, among the n entries unsorted in s.list, before which there is
// weight `base` (of 1 an entry, or w): the entry's value and index.
template <bool MASS>
__device__ __forceinline__ void cut_list(Shared &s, const Row &row, int n, uint64_t base, uint64_t target) {
    const int first = 4 * threadIdx.x;
    sort_list(s, n);
    uint64_t sum[4], w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = w[e] = first + e >= n ? 0 : MASS ? row.weight(key_value((uint32_t)(s.list[first + e] >> 32))) : 1;
    block_scan(s, sum);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (base + sum[e] - w[e] < target && (base + sum[e] >= target || first + e == n - 1)) {       // (the last one reaches it)
            s.cut_v = key_value((uint32_t)(s.list[first + e] >> 32));
            s.cut_i = (int)(uint32_t)s.list[first + e];
        }
    __syncthreads();
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

    // The weight of those of a vector's entries that on(x, i) holds for.
    template <bool ALL, typename F>
    __device__ __forceinline__ uint64_t weigh(const Row &row, const uint4 &x, int i0, F on) const {
        uint32_t use = 0;
        if (!ALL) {
#pragma unroll
            for (int e = 0; e < VE; ++e) use |= (uint32_t)on(T::get(x, e), i0 + e) << e;
            if (!use) return 0;
        }
        uint64_t sum = 0;
#pragma unroll
        for (int e = 0; e < VE; e += 2) {
            uint64_t wa, wb;
            row.weights(T::get(x, e), T::get(x, e + 1), wa, wb);
            if (ALL || ((use >> e) & 1)) sum += wa;
            if (ALL || ((use >> e) & 2)) sum += wb;
        }
        return sum;
    }

    // The lowest index at which the running sum of f in index order reaches the target that goal(total) gives, kept within
    // 1 .. total; -1 where the total is 0.  All threads of all CTAs return it.
    // LAST: the thread that finds it writes it to *token instead, and nobody else learns it (a total of 0 writes nothing).
    // fv: the sum of f over a vector.
    template <bool LAST, typename F, typename G>
    __device__ __forceinline__ int pick(Shared &s, F f, G goal, int32_t *token = nullptr) const {
        return pick_by<LAST>(s, f, [&](const uint4 &x, int i0) {
            uint64_t sum = 0;
#pragma unroll
            for (int e = 0; e < VE; ++e) sum += f(T::get(x, e), i0 + e);
            return sum;
        }, goal, token);
    }
    template <bool LAST, typename F, typename V, typename G>
    __device__ __forceinline__ int pick_by(Shared &s, F f, V fv, G goal, int32_t *token) const {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int lo = (int)((long long)nv * warp / kWarps), hi = (int)((long long)nv * (warp + 1) / kWarps);
        uint64_t sum = 0;
        int step = 0;
        for (int j0 = lo; j0 < hi; j0 += 32, ++step) {
            const int j = j0 + lane;
            uint64_t mine = 0;
            if (j < hi) {
                mine = fv(vec[j], begin - skip + j * VE);
            }
            if (__any_sync(0xffffffffu, mine != 0)) mine = warp_sum64(mine);
            if (lane == 0) s.steps[warp][step] = mine;
            sum += mine;
        }
        __syncwarp();
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
            const uint64_t mine = lane < step ? s.steps[warp][lane] : 0, upto = before + warp_scan64(mine, lane);
            const int at = __ffs(__ballot_sync(0xffffffffu, upto >= target)) - 1;
            before = __shfl_sync(0xffffffffu, upto - mine, at);
            const int j = lo + 32 * at + lane, i0 = begin - skip + j * VE;
            uint4 x = make_uint4(0, 0, 0, 0);
            uint64_t w = 0;
            if (j < hi) {
                x = vec[j];
                w = fv(x, i0);
            }
            uint64_t to = before + warp_scan64(w, lane);
            if (lane == __ffs(__ballot_sync(0xffffffffu, to >= target)) - 1) {
                to -= w;
                int found = -1;
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    to += f(T::get(x, e), i0 + e);
                    if (found < 0 && to >= target) found = i0 + e;
                }
                if (LAST) *token = found;
                else s.pick_index = found;
            }
        }
        if (LAST) return total > 0;
        cluster_join();
        int found = -1;
        for (int k = 0; k < C; ++k) found = max(found, peer(&s.pick_index, k));
        cluster_join();                              // read before they are written again
        return found;
    }

    // The bins of this search level, filled by every CTA: finds the first one up to which base and the weights reach the
    // target that goal(total) gives, and the weight before it.  False: no bin does.
    // LEAST: the bins of y hold counts, taken for the least weight that so many entries there can have; bin is one by which the
    // true weights have reached the target, from the first by which they can have.  A true sum lies between that and 1 / 0.99 of it
    // (2^(1 / kBinScale) is 1.0076) and a unit an entry.  Both ends are sought twice, from the sum up to a bin and from the sum behind
    // it, of which z (the true sum of all) less the target may remain: the latter is the sharper the closer top-p is to 1.
    struct Found {
        uint32_t bin, from;
        uint64_t before;
    };
    template <bool MASS, bool LEAST = false, typename G>
    __device__ __forceinline__ bool find_bin(Shared &s, uint64_t base, G goal, Found &found, const uint64_t &z = 0) const {
        // each CTA sums a slice of the bins over the cluster, up to N of them a thread
        constexpr int N = kBins<MASS> / kThreads;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slice = kBins<MASS> / C, per = (slice + kThreads - 1) / kThreads;
        const int b0 = rank * slice + threadIdx.x * per;
        const bool on = (int)threadIdx.x * per < slice;
        cluster_join();
        uint64_t w[N], mine = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            w[i] = 0;
            if (!on || i >= per) continue;
            for (int k = 0; k < C; ++k)
#pragma unroll
                for (int l = 0; l < (MASS ? 3 : 1); ++l) w[i] += (uint64_t)peer(MASS ? &s.mass[l][b0 + i] : &s.count[b0 + i], k) << (kLimb * l);
            if (LEAST) w[i] *= (uint64_t)(ex2_approx(kUnit - (b0 + i + 1) * (1.f / kBinScale<MASS>)) * 0.999f);
            mine += w[i];
        }
        const uint64_t upto = warp_scan64(mine, lane);
        if (lane == 31) s.scan[warp] = upto;
        if (threadIdx.x == 0) s.bin = s.bin_from = s.bin_behind = kBins<MASS>;
        __syncthreads();
        uint64_t before = base + upto - mine;
        for (int k = 0; k < warp; ++k) before += s.scan[k];
        if (threadIdx.x == kThreads - 1) s.slice = before + mine - base;
        cluster_join();
        uint64_t total = 0;
        for (int k = 0; k < C; ++k) {
            const uint64_t x = peer(&s.slice, k);
            if (k < rank) before += x;
            total += x;
        }
        const uint64_t target = goal(total);
        if (LEAST) {
            constexpr uint64_t kEntries = OSCAR_SAMPLE_MAX_VOCAB;
            auto share = [&](uint64_t x) { return x > kEntries ? __umul64hi(x - kEntries, (uint64_t)(0.99 * 0x1p63) << 1) : 0; };
            const uint64_t low = max((unsigned long long)share(target), 1ull), rest = z - target, rest_low = share(rest);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint64_t upto_i = before + w[i], behind = total - before, behind_i = total - upto_i;
                if (before < target && target <= upto_i) atomicMin(&s.bin, (uint32_t)(b0 + i));
                if (before < low && low <= upto_i) s.bin_from = b0 + i;
                if (behind > rest_low && behind_i <= rest_low) atomicMin(&s.bin, (uint32_t)(b0 + i));
                if (behind > rest && behind_i <= rest) s.bin_behind = b0 + i;
                before = upto_i;
            }
        } else if (before < target && target <= before + mine) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (before < target && target <= before + w[i]) {
                    s.bin = b0 + i;
                    s.before = before;
                }
                before += w[i];
            }
        }
        cluster_join();
        uint32_t bin = kBins<MASS>, from = kBins<MASS>, behind = kBins<MASS>;
        uint64_t at = 0;
        for (int k = 0; k < C; ++k) {
            const uint32_t x = peer(&s.bin, k);
            if (x < bin) {
                bin = x;
                at = peer(&s.before, k);
            }
            if (LEAST) {
                from = min(from, peer(&s.bin_from, k));
                behind = min(behind, peer(&s.bin_behind, k));
            }
        }
        if (LEAST) from = max(from < kBins<MASS> ? from : 0u, behind < kBins<MASS> ? behind : 0u);
        found = Found{bin, from, at};
        return bin < kBins<MASS>;
    }

    template <bool MASS>
    __device__ __forceinline__ void clear(Shared &s) const {
        uint4 *h = reinterpret_cast<uint4 *>(s.count);
        for (int i = threadIdx.x; i < (MASS ? 3 : 1) * kBins<MASS> / 4; i += kThreads) h[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    template <bool MASS>
    static __device__ __forceinline__ void add(Shared &s, int bin, uint64_t w) {
        if (MASS) {
            atomicAdd(&s.mass[0][bin], (uint32_t)w & ((1u << kLimb) - 1));
            atomicAdd(&s.mass[1][bin], (uint32_t)(w >> kLimb) & ((1u << kLimb) - 1));
            atomicAdd(&s.mass[2][bin], (uint32_t)(w >> (2 * kLimb)));
        } else {
            atomicAdd(&s.count[bin], 1u);
        }
    }
    // The bins of y.
    template <bool MASS>
    __device__ __forceinline__ void depths(Shared &s, const Row &row) const {
        clear<MASS>(s);
        each([&](float x, int i) {
            const float y = row.depth(x);
            if (y < kDeep && row.kept(x, i)) {
                const uint64_t w = MASS ? row.weight(x) : 1;
                if (w) add<MASS>(s, bin_of<MASS>(y), w);
            }
        });
    }

    // Entries counted in the bins from .. to and 0 .. to of this CTA, for the cluster to read behind the next barrier.
    __device__ __forceinline__ void count_entries(Shared &s, uint32_t from, uint32_t to) const {
        uint32_t some = 0, all = 0;
        for (uint32_t i = threadIdx.x; i <= to; i += kThreads) {
            const uint32_t n = s.count[i];
            all += n;
            if (i >= from) some += n;
        }
        some = __reduce_add_sync(0xffffffffu, some);
        all = __reduce_add_sync(0xffffffffu, all);
        if (threadIdx.x == 0) s.n_some = s.n_all = 0;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            atomicAdd(&s.n_some, some);
            atomicAdd(&s.n_all, all);
        }
    }

    // The entries of the bins from .. to that row keeps, of all CTAs, to the first CTA's list; at: where this one's begin.  Every CTA
    // is done with its bins: their memory becomes the list.
    __device__ __forceinline__ void gather(Shared &s, const Row &row, uint32_t from, uint32_t to, uint32_t at) const {
        if (threadIdx.x == 0) s.cursor = at;
        __syncthreads();
        uint32_t list;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(list) : "r"(saddr(s.list)), "r"(0));
        each([&](float x, int i) {
            const float y = row.depth(x);
            const uint32_t bin = bin_of<false>(y);
            if (!(y < kDeep) || bin < from || bin > to || !row.kept(x, i)) return;
            const uint32_t here = __activemask(), lane = threadIdx.x & 31, first = __ffs(here) - 1;
            uint32_t place = 0;
            if (lane == first) place = atomicAdd(&s.cursor, (uint32_t)__popc(here));
            place = __shfl_sync(here, place, first) + __popc(here & ((1u << lane) - 1));
            if (place < kList)
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(list + 8 * place), "l"((uint64_t)falling_key(x) << 32 | (uint32_t)i) : "memory");
        });
        cluster_join();                              // the list is complete
    }

    // A value a thread, summed by warps, for the cluster to read behind the next barrier; and the sum over the cluster.
    static __device__ __forceinline__ void publish(Shared &s, uint64_t x) {
        __syncwarp();
        x = warp_sum64(x);
        if ((threadIdx.x & 31) == 0) s.warp_sum[threadIdx.x >> 5] = x;
    }
    __device__ __forceinline__ uint64_t published(Shared &s) const {
        uint64_t x = 0;
        for (int k = threadIdx.x & 31; k < C * kWarps; k += 32) x += peer(&s.warp_sum[k % kWarps], k / kWarps);
        return warp_sum64(x);
    }

    // Narrows what is kept by top-k (MASS false, k tokens) or top-p (s.p64 of the kept weight).  With whole: returns how many
    // entries the first CTA's list holds, if all that can be kept are there (nothing is narrowed then); else 0.  weighed: the kept
    // weight (top-p).  (What a CTA publishes is not written again before all have passed another barrier.)
    template <bool MASS>
    __device__ __forceinline__ uint32_t narrow(Shared &s, Row &row, uint64_t k, bool whole, uint64_t &weighed) const {
        clear<false>(s);
        uint64_t sum = 0;
        const bool all = row.v == -INFINITY;
        for (int j = threadIdx.x; j < nv; j += kThreads) {
            const uint4 x = vec[j];
            const int i0 = begin - skip + j * VE;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float xe = T::get(x, e), y = row.depth(xe);
                if (y < kDeep && (all || row.kept(xe, i0 + e))) add<false>(s, bin_of<false>(y), 1);
            }
            if (MASS) sum += all ? weigh<true>(row, x, i0, [](float, int) { return true; }) : weigh<false>(row, x, i0, [&](float xe, int i) { return row.kept(xe, i); });
        }
        if (MASS) publish(s, sum);
        uint64_t target = k;
        Found f;
        const bool found = find_bin<false, MASS>(s, 0, [&](uint64_t) {
            if (MASS) {
                weighed = published(s);
                target = __umul64hi(weighed, s.p64) + (weighed * s.p64 != 0);
                if (target < 1) target = 1;
            }
            return target;
        }, f, weighed);
        if (!MASS && !found) return 0;               // fewer than k have weight: all stay
        const uint32_t to = found ? f.bin : kBins<false> - 1, from = !MASS ? to : min(f.from, to);
        count_entries(s, from, to);
        cluster_join();
        uint32_t some = 0, some_at = 0, every = 0, every_at = 0;
        for (int r = 0; r < C; ++r) {
            const uint32_t x = peer(&s.n_some, r), y = peer(&s.n_all, r);
            if (r < rank) {
                some_at += x;
                every_at += y;
            }
            some += x;
            every += y;
        }
        if (whole && every <= kList) {
            gather(s, row, 0, to, every_at);
            return every;
        }
        if (some > kList) {
            cut<MASS>(s, row, [&](uint64_t) { return target; });
            return 0;
        }
        if (MASS) {
            // the weight above those bins
            sum = 0;
            for (int j = threadIdx.x; j < nv; j += kThreads)
                sum += weigh<false>(row, vec[j], begin - skip + j * VE, [&](float x, int i) {
                    const float y = row.depth(x);
                    return y < kDeep && bin_of<false>(y) < from && (all || row.kept(x, i));
                });
            publish(s, sum);
        }
        gather(s, row, from, to, some_at);
        if (rank == 0) cut_list<MASS>(s, row, some, MASS ? published(s) : f.before, target);
        cluster_join();
        row.v = peer(&s.cut_v, 0);
        row.I = peer(&s.cut_i, 0);
        return 0;
    }

    // Narrows what is kept to the shortest prefix whose weight (1 a token, or w) reaches the target.
    template <bool MASS, typename G>
    __device__ __forceinline__ void cut(Shared &s, Row &row, G goal) const {
        depths<MASS>(s, row);
        uint64_t target = 0;
        Found f;
        if (!find_bin<MASS>(s, 0, [&](uint64_t total) { return target = goal(total); }, f)) return;
        const uint32_t bin = f.bin;
        uint64_t before = f.before;
        auto in_bin = [&](float x, int i) {
            const float y = row.depth(x);
            return y < kDeep && bin_of<MASS>(y) == bin && row.kept(x, i);
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
            if (at < kKeys) s.list_key[at] = k;
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
            clear<MASS>(s);
            auto count = [&](uint32_t k) {
                if (k >= lo && k <= hi) add<MASS>(s, (k - lo) >> shift, MASS ? row.weight(key_value(k)) : 1);
            };
            if (n <= kKeys)
                for (uint32_t i = threadIdx.x; i < n; i += kThreads) count(s.list_key[i]);
            else
                each([&](float x, int i) {
                    if (in_bin(x, i)) count(falling_key(x));
                });
            if (!find_bin<MASS>(s, before, [&](uint64_t) { return target; }, f)) return;      // (the bin's sum reaches it: does not happen)
            before = f.before;
            lo += f.bin << shift;
            if (!shift) break;
            hi = min(hi, lo + ((1u << shift) - 1));
        }
        // one value left: the first ties of it
        const float v = key_value(lo);
        const uint64_t each_w = MASS ? row.weight(v) : 1, ties = (target - before + each_w - 1) / each_w;
        row.I = pick<false>(s, [&](float x, int i) -> uint64_t { return x == v && row.kept(x, i); }, [&](uint64_t) { return ties; });
        row.v = v;
    }
};

// The draw from a row's first n entries, unsorted in s.list, by one CTA: total is what top-p is of, where the list does not hold it
// all (0: the first k entries' weight).
__device__ __forceinline__ int draw_list(Shared &s, const Row &row, int n, int k, uint64_t total) {
    static_assert(kList == 4 * kThreads, "four entries a thread");
    const int first = 4 * threadIdx.x;
    sort_list(s, n);
    int keep = min(n, k);
    uint64_t sum[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sum[e] = first + e < keep ? row.weight(key_value((uint32_t)(s.list[first + e] >> 32))) : 0;
        s.weight[first + e] = sum[e];
    }
    block_scan(s, sum);
    if (threadIdx.x == kThreads - 1 && total == 0) s.total = sum[3];
    if (threadIdx.x == 0) s.n_list = keep;
    __syncthreads();
    if (s.top_p) {
        const uint64_t z = total ? total : s.total;
        uint64_t target = __umul64hi(z, s.p64) + (z * s.p64 != 0);
        if (target < 1) target = 1;
        uint64_t before = sum[0] - s.weight[first];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (before < target && sum[e] >= target) atomicMin(&s.n_list, (uint32_t)(first + e + 1));
            before = sum[e];
        }
    }
    // min-p: behind the entry before the first that is too small (row.v: the least logit)
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (first + e > 0 && first + e < keep && (s.min_mode == 3 || key_value((uint32_t)(s.list[first + e] >> 32)) < row.v))
            atomicMin(&s.n_list, (uint32_t)(first + e));
    __syncthreads();
    keep = s.n_list;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (first + e == keep - 1) s.before = __umul64hi(sum[e], s.u64) + 1;
    // by index, with the place that holds the weight
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (first + e < keep) s.list[first + e] = (s.list[first + e] << 32) | (uint32_t)(first + e);
    __syncthreads();
    sort_list(s, keep);
    const uint64_t target = s.before;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = first + e < keep ? s.weight[(uint32_t)s.list[first + e]] : 0;
    const uint64_t own = sum[0];
    block_scan(s, sum);
    uint64_t before = sum[0] - own;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (before < target && sum[e] >= target) s.pick_index = (int)(s.list[first + e] >> 32);
        before = sum[e];
    }
    __syncthreads();
    return s.pick_index;
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(SampleArgs a) {
    using T = Type<TYPE>;
    using raw = typename T::raw;
    constexpr int VE = Part<TYPE>::VE;
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    uint4 *data = reinterpret_cast<uint4 *>(smem + kSharedBytes);
    const int C = gridDim.x, rank = blockIdx.x, r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < 256) s.table[threadIdx.x] = kTable.t[threadIdx.x];
    pdl_wait();
    if (threadIdx.x == kThreads - 1) {               // the row's arguments: 64-bit operations are few on this GPU
        const float temp = a.in.temperature[r], p = a.in.top_p ? a.in.top_p[r] : 1.f, mp = a.in.min_p ? a.in.min_p[r] : 0.f;
        const double c = fmin(1.4426950408889634 / (double)temp, 0x1p120);
        s.temp = temp;
        s.ch = (float)c;
        s.cl = (float)(c - (double)s.ch);
        s.top_k = a.in.top_k ? a.in.top_k[r] : 0;
        s.top_p = p < 1.f;
        s.p64 = (uint64_t)((double)fmaxf(p, 0.f) * 0x1p64);
        s.u64 = (uint64_t)((double)fminf(fmaxf(a.in.u[r], 0.f), 0x1.fffffep-1f) * 0x1p64);
        // (an infinite temperature: every finite logit weighs 1, which a min_p up to 1 keeps)
        s.min_mode = mp > 1.f ? 3 : mp == 1.f && temp < INFINITY ? 2 : mp > 0.f ? 1 : 0;
        s.min_off = s.min_mode != 1 ? 0.0 : temp < INFINITY ? (double)temp * log((double)mp) : -INFINITY;
    }
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
    const float temp = s.temp;
    int32_t *token = a.tokens + r;
    if (!(top > -INFINITY)) {
        if (rank == 0 && threadIdx.x == 0) *token = -1;
    } else if (!(temp > 0.f)) {
        part.template pick<true>(s, [&](float x, int) -> uint64_t { return x == top; }, [](uint64_t) -> uint64_t { return 1; }, token);
    } else {
        Row row{top, s.ch, s.cl, -INFINITY, 0x7fffffff, s.table};
        float least = -INFINITY;                     // min-p's, for the sorted list
        if (s.min_mode) least = s.min_mode >= 2 || top == INFINITY ? top : __double2float_ru((double)top + s.min_off);
        const bool by_count = s.top_k > 0 && s.top_k < a.in.vocab;
        uint64_t weighed = 0;
        uint32_t n = 0;
        if (by_count) n = part.template narrow<false>(s, row, s.top_k, true, weighed);
        if (!n && s.top_p) n = part.template narrow<true>(s, row, 0, !by_count, weighed);
        if (n) {
            if (rank == 0) {
                row.v = least;
                const int t = draw_list(s, row, n, by_count ? s.top_k : n, weighed);
                if (threadIdx.x == 0) *token = t;
            }
            return;                                  // nothing of another CTA is read from here on
        }
        if (s.min_mode == 3) {                       // no weight is that large: the first token of the order
            row.I = part.template pick<false>(s, [&](float x, int) -> uint64_t { return x == top; }, [](uint64_t) -> uint64_t { return 1; });
            row.v = top;
        } else if (least > row.v) {
            row.v = least;
            row.I = 0x7fffffff;
        }
        const bool all = row.v == -INFINITY;
        part.template pick_by<true>(
            s, [&](float x, int i) -> uint64_t { return row.kept(x, i) ? row.weight(x) : 0; },
            [&](const uint4 &x, int i0) {
                auto kept = [&](float xe, int i) { return row.kept(xe, i); };
                return all ? part.template weigh<true>(row, x, i0, kept) : part.template weigh<false>(row, x, i0, kept);
            },
            [&](uint64_t total) -> uint64_t { return __umul64hi(total, s.u64) + 1; }, token);
    }
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
    // CTAs a row: as many as leave room for two on an SM (115,712 bytes each), and more (8 at most) while the rows leave SMs idle
    // and a CTA has 2,048 tokens or more
    const int size = in.dtype == OSCAR_DTYPE_F32 ? 4 : 2, room = 115712 - kSharedBytes - 48;
    int C = 1;
    while (C < 8 && (in.vocab + C - 1) / C * size > room) C *= 2;
    while (C < 8 && (long long)in.rows * C * 2 <= 2 * kSms && in.vocab / (2 * C) >= 2048) C *= 2;
    SampleArgs a{in, (in.vocab + C - 1) / C, tokens};
    const int smem = kSharedBytes + ((a.per + 2 * (16 / size)) * size + 15) / 16 * 16;
    switch (in.dtype) {
        case OSCAR_DTYPE_F32: return launch_type<OSCAR_DTYPE_F32>(a, C, smem, st);
        case OSCAR_DTYPE_BF16: return launch_type<OSCAR_DTYPE_BF16>(a, C, smem, st);
        default: return launch_type<OSCAR_DTYPE_F16>(a, C, smem, st);
    }
}

}  // namespace oscar
