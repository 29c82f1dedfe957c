// Attention of many query rows (a tree's nodes times the query heads of a kv head) over an INT4 history on the 5th-generation
// tensor cores: the history's slots of the partials for 128 query rows of a kv head at a time, group 128.
//
// Per 128 positions, with f16 operands and fp32 sums in tensor memory (tcgen05, M128 N128 K16, eight steps each):
//   D[row][t] = sum_c Q'[row][c] n_t,c           the query rows (tensor memory) by the codes as subnormals n 2^-24 (odd nibbles: 16 n)
//   e = f s_t D + z_t zq_row - M_row,  p = 2^e   f undoes the scalings, zq = sm sum_c q_c, M the row's reference
//   O[row][c] += sum_t (p s'_t) (n'_t,c - 8),  l += p,  zs += p (z'_t + 8 s'_t)
// A product p s' is one f16 number, 2^-11 relative; M is raised whenever one passes 2^15 (then brought to 2^8) or p passes 2^110,
// so that the largest p s' so far, not the largest p, sits near the top of f16's range.  Codes are centred for the reason given
// in attn_tree.cu.  Both operands of codes lie in shared memory as they come, a position's channels together: K-major for the
// logits, MN-major for the values, so both are unpacked the same way.
//
// Up to 32 (64) rows are held four times (twice) in the 128 lanes, and each copy takes the logits of its own quarter (half) of
// the positions; its p s' elsewhere are zeros.  So all softmax warps work however few rows there are, and the copies' results are
// joined like splits.
//
// One CTA an SM: warps 0-7 softmax (two per lane quarter, half of the positions each, under one reference), 8-11 unpack keys,
// 12-15 values, 16 copies, 17 issues the products; logits of a tile are formed while the softmax of the tile before runs.  Two
// buffers of unpacked codes and of logits; p s' takes the place of its logits.

#include <cuda_fp16.h>

#include <algorithm>

#include "tree_window.cuh"

namespace oscar {
namespace {

constexpr int kT = 128;                          // positions of a tile
constexpr int kR = 128;                          // query rows of a CTA
constexpr int kStages = 3;
constexpr int kSoftWarps = 8, kUnpackWarps = 4;  // (unpack: of keys, and of values)
constexpr int kThreads = 32 * (kSoftWarps + 2 * kUnpackWarps + 2);
constexpr int kSzBuffers = 4;
constexpr int kOperand = kT * kHeadDim * 2;      // 32 KB
constexpr int kHalf = kOperand / 2;              // its channels 0..63
constexpr int kStageCodes = kT * kRow4;          // 8 KB
constexpr int kStageBytes = 2 * kStageCodes + kT * 8;
constexpr int kOffK = 0, kOffV = 2 * kOperand, kOffStage = 4 * kOperand;
constexpr int kOffSz = kOffStage + kStages * kStageBytes;          // [buffers][2][64] float4
constexpr int kSzBytes = 2 * kT / 2 * 16;
constexpr int kOffMeta = kOffSz + kSzBuffers * kSzBytes;           // barriers, piece masks, TMEM address
constexpr int kOffPair = kOffMeta + 512;         // [4 quarters][2][32] float2
constexpr int kSmem = kOffPair + 4 * 2 * 32 * 8 + 1024;
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384;
constexpr float kNoRef = -1e30f;
constexpr float kMostW = 0x1p15f, kMostP = 0x1p110f;
constexpr float kNewW = 8.f, kNewP = 100.f;      // a new reference brings p s' to 2^8 at most, p to 2^100
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(kT >> 3) << 17) | ((uint32_t)(kR >> 4) << 24);      // f16, f16, fp32
constexpr uint32_t kIdescMN = kIdesc | (1u << 16);                                                      // B MN-major

// As mbar_wait, but given up after about a second: roles wait for one another in a chain.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity) {
    for (int i = 0; i < 1 << 19; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return false;
}

struct Meta {
    uint64_t full[kStages], empty[kStages], kready[2], vready[2], kfree[2], vfree[2], szready[kSzBuffers], szfree[kSzBuffers], sfull[2], pready[2], pvdone;
    uint32_t ok[kStages];                        // pieces of 16 positions that were copied
    alignas(8) uint32_t valid[kSzBuffers][4], masked[kSzBuffers];    // of the tile whose scales are there: bits of usable positions; some are not
    float max_q;
    uint32_t tmem, stuck;                        // stuck: a copy or product may still be under way
};

static_assert(sizeof(Meta) <= 512, "up to kOffPair");

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle: 64 elements of 8 k in an atom of 1,024 bytes, the next
// 8 k `1024` bytes further (stride offset), the next 64 elements kHalf bytes further (leading offset).
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(kHalf >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
// D[tmem] (+)= A[tmem] . B[smem], f16.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// The two softmax warps of a lane quarter.
__device__ __forceinline__ void pair_sync(int quarter) { asm volatile("bar.sync %0, 64;" ::"r"(quarter + 1) : "memory"); }
__device__ __forceinline__ bool pair_any(int quarter, bool x) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)x), "r"(quarter + 1)
                 : "memory");
    return r != 0;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
          "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// A code word's operand: channels 0 4 | 1 5 | 2 6 | 3 7 of its eight.
__device__ __forceinline__ uint4 subnormal(uint32_t w) {
    const uint32_t v = w >> 8;
    return make_uint4(w & kM0, w & kM1, v & kM0, v & kM1);
}
__device__ __forceinline__ uint4 centred(uint32_t w) {
    const uint32_t v = w >> 8;
    return make_uint4(centred_low(w), centred_high(w), centred_low(v), centred_high(v));
}

// The tiles of this CTA's split: tile i holds the positions p0(i) .. + 127.
struct Tiles {
    int first, n, lo, hi;                        // valid positions [lo, hi)
    __device__ __forceinline__ Tiles(int sink, int he, int S, int s) {
        const int t0 = sink / kT, nt = he > sink ? (he + kT - 1) / kT - t0 : 0;
        first = t0 + (int)((long long)s * nt / S);
        n = t0 + (int)((long long)(s + 1) * nt / S) - first;
        lo = sink;
        hi = he;
    }
    __device__ __forceinline__ int p0(int i) const { return (first + i) * kT; }
};

// One softmax thread's row.
struct RowState {
    float zq, M, l, zs;
};

// The logits (less the reference), base 2, of two positions: D in d0, d1, the constants of pair j at sk.
__device__ __forceinline__ f2 shifted_logits(const float4 *sk, int j, uint32_t d0, uint32_t d1, f2 zq2, f2 m2) {
    const float4 c = sk[j];
    return fma2(pair(c.x, c.y), pair(__uint_as_float(d0), __uint_as_float(d1)), fma2(pair(c.z, c.w), zq2, m2));
}

// A warp's part of a tile, NU x 16 positions: tS the first one's logits, sk: f s | z of the keys, sv: s' | z' + 8 s' of the values
// (two positions each), valid: the bits of usable positions.
template <int NU>
struct Unit {
    uint32_t tS;
    const float4 *sk, *sv;
    uint64_t valid;
};

// p s' packed in w, the sums in l and zs; true where a reference is due.
template <int NU, bool FULL>
__device__ __forceinline__ bool tile_softmax(const RowState &st, const Unit<NU> &x, uint32_t (&w)[NU * 8], float &l, float &zs) {
    const f2 zq2 = pair(st.zq, st.zq), m2 = pair(-st.M, -st.M);
    f2 l2[2] = {0ull, 0ull}, z2[2] = {0ull, 0ull};
    __half2 most = __half2half2(__ushort_as_half(0));
    uint32_t r[2][16];
    tmem_ld16(x.tS, r[0]);
    tmem_ld_wait();
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        if (u + 1 < NU) tmem_ld16(x.tS + 16 * (u + 1), r[(u + 1) & 1]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float e0, e1, w0, w1;
            unpair(shifted_logits(x.sk, 8 * u + j, r[u & 1][2 * j], r[u & 1][2 * j + 1], zq2, m2), e0, e1);
            if (!FULL) {
                if (!((x.valid >> (16 * u + 2 * j)) & 1)) e0 = -INFINITY;
                if (!((x.valid >> (16 * u + 2 * j + 1)) & 1)) e1 = -INFINITY;
            }
            const f2 p = pair(ex2_approx(e0), ex2_approx(e1));
            const float4 cv = x.sv[8 * u + j];
            l2[j & 1] = add2(l2[j & 1], p);
            z2[j & 1] = fma2(p, pair(cv.z, cv.w), z2[j & 1]);
            unpair(mul2(p, pair(cv.x, cv.y)), w0, w1);
            const __half2 h = __floats2half2_rn(w0, w1);
            most = __hmax2(most, h);
            w[8 * u + j] = *reinterpret_cast<const uint32_t *>(&h);
        }
        if (u + 1 < NU) tmem_ld_wait();
    }
    float a, b;
    unpair(add2(l2[0], l2[1]), a, b);
    l = a + b;
    unpair(add2(z2[0], z2[1]), a, b);
    zs = a + b;
    return fmaxf(__low2float(most), __high2float(most)) >= kMostW || l >= kMostP;
}

// New references for the rows of the pair of warps that need one, and what was summed under the old ones brought to them: each
// warp takes half of O's columns.
template <int NU>
__device__ __forceinline__ void new_reference(RowState &st, const Unit<NU> &x, uint32_t tO, bool has_o, int quarter, int half, int lane,
                                              float2 *pairs) {
    float top = -INFINITY, topw = -INFINITY;     // largest logit, largest logit + log2 s'
    const f2 zq2 = pair(st.zq, st.zq);
#pragma unroll 1
    for (int u = 0; u < 2 * NU; ++u) {
        uint32_t r[8];
        tmem_ld8(x.tS + 8 * u, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float e[2];
            unpair(shifted_logits(x.sk, 4 * u + j, r[2 * j], r[2 * j + 1], zq2, 0ull), e[0], e[1]);
            const float4 cv = x.sv[4 * u + j];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (!((x.valid >> (8 * u + 2 * j + k)) & 1)) continue;
                top = fmaxf(top, e[k]);
                topw = fmaxf(topw, e[k] + __log2f(k ? cv.y : cv.x));
            }
        }
    }
    pairs[(quarter * 2 + half) * 32 + lane] = make_float2(top, topw);
    pair_sync(quarter);
    const float2 other = pairs[(quarter * 2 + (half ^ 1)) * 32 + lane];
    top = fmaxf(top, other.x);
    topw = fmaxf(topw, other.y);
    float M = st.M;
    // kept where it will do: 2^(topw - M) and 2^(top - M) within the limits the tile is checked for, with a margin for rounding
    if (topw - M >= 14.9f || top - M >= 102.f) M = fmaxf(M, fmaxf(topw - kNewW, top - kNewP));
    const float f = ex2_approx(st.M - M);
    st.M = M;
    st.l *= f;
    st.zs *= f;
    if (!has_o) return;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        uint32_t r[8];
        tmem_ld8(tO + 64 * half + 8 * c, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * f);
        tmem_st8(tO + 64 * half + 8 * c, r);
    }
    tmem_st_wait();
}

template <int REP>
__device__ __forceinline__ void softmax_loop(const TreeArgs &a, const Tiles &ti, Meta &mt, uint8_t *sm, uint32_t tmem, int warp, int lane,
                                             RowState &st) {
    constexpr int NU = 4 / REP;                  // units of 16 positions
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int copy = REP == 1 ? 0 : REP == 2 ? quarter >> 1 : quarter;
    const int first = (2 * copy + half) * NU;    // this warp's first unit
    float2 *pairs = reinterpret_cast<float2 *>(sm + kOffPair);
    bool gone = false;
    for (int i = 0; i < ti.n; ++i) {
        const int b = i & 1, z = i % kSzBuffers;
        const uint32_t ph = (i >> 1) & 1;
        // a warp whose wait ran out waits no more, but goes on: its partner's barriers count it
        if (!gone && !(wait_for(saddr(&mt.sfull[b]), ph) && wait_for(saddr(&mt.szready[z]), (i / kSzBuffers) & 1))) {
            if (lane == 0) flag_status(a.status, OSCAR_DEV_WAIT_TIMEOUT);
            gone = true;
        }
        tc_fence_after();
        Unit<NU> x;
        const uint32_t tS = tmem + kColS + b * 128 + lanes;
        x.tS = tS + 16 * first;
        x.sk = reinterpret_cast<const float4 *>(sm + kOffSz + z * kSzBytes) + 8 * first;
        x.sv = x.sk + kT / 2;
        const bool full = !mt.masked[z];
        x.valid = ~0ull;
        if (!full) x.valid = *reinterpret_cast<const uint64_t *>(&mt.valid[z][2 * (first >> 2)]) >> (16 * (first & 3));
        uint32_t w[NU * 8];
        float l, zs;
        auto form = [&] { return full ? tile_softmax<NU, true>(st, x, w, l, zs) : tile_softmax<NU, false>(st, x, w, l, zs); };
        if (pair_any(quarter, form())) {
            if (!gone && i > 0 && !wait_for(saddr(&mt.pvdone), (i - 1) & 1)) {
                if (lane == 0) flag_status(a.status, OSCAR_DEV_WAIT_TIMEOUT);
                gone = true;
            }
            tc_fence_after();
            new_reference<NU>(st, x, tmem + kColO + lanes, i > 0, quarter, half, lane, pairs);
            form();
            pair_sync(quarter);                  // both are done with the logits
        }
        st.l += l;
        st.zs += zs;
        // p s' in the logits' place, zeros where other copies of the row have theirs
#pragma unroll
        for (int u = 0; u < NU; ++u) tmem_st8(tS + 8 * (first + u), &w[8 * u]);
        if (REP > 1) {
            uint32_t none[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) none[j] = 0u;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (u / (2 * NU) != copy && (u & 1) == half) tmem_st8(tS + 8 * u, none);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(saddr(&mt.pready[b]));
            mbar_arrive(saddr(&mt.szfree[z]));
        }
    }
}

// 128 threads unpack the keys' (VALUES: the values') codes of each tile.  A thread's 16 bytes (32 channels) of a position are four
// chunks of the operand; the order in which lanes write theirs keeps each group of eight lanes on different banks.
template <bool VALUES>
__device__ __forceinline__ void unpack_loop(const TreeArgs &a, const Tiles &ti, Meta &mt, uint8_t *sm, int tid, int lane, float fac) {
    for (int i = 0; i < ti.n; ++i) {
        const int b = i & 1, st = i % kStages, z = i % kSzBuffers;
        bool ok = wait_for(saddr(&mt.full[st]), (i / kStages) & 1);
        if (ok && i >= 2) ok = wait_for(saddr(VALUES ? &mt.vfree[b] : &mt.kfree[b]), ((i >> 1) & 1) ^ 1);
        if (ok && !VALUES && i >= kSzBuffers) ok = wait_for(saddr(&mt.szfree[z]), ((i / kSzBuffers) & 1) ^ 1);
        if (!ok) {
            if (lane == 0) flag_status(a.status, OSCAR_DEV_WAIT_TIMEOUT);
            return;
        }
        const uint8_t *stage = sm + kOffStage + st * kStageBytes;
        const uint8_t *codes = stage + (VALUES ? kStageCodes : 0);
        uint8_t *op = sm + (VALUES ? kOffV : kOffK) + b * kOperand;
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = *reinterpret_cast<const uint4 *>(codes + 16 * (tid + 128 * k));
        const int q = tid & 3, swap = q >> 1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = (tid >> 2) + 32 * k;
            uint8_t *row = op + swap * kHalf + (t >> 3) * 1024 + (t & 7) * 128;
            const uint32_t word[4] = {swap ? x[k].z : x[k].x, swap ? x[k].w : x[k].y, swap ? x[k].x : x[k].z, swap ? x[k].y : x[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int chunk = 4 * (q & 1) + (j ^ (2 * swap));
                *reinterpret_cast<uint4 *>(row + ((chunk ^ (t & 7)) << 4)) = VALUES ? centred(word[j]) : subnormal(word[j]);
            }
        }
        if (!VALUES && tid < kT / 2) {
            // scales and zeros of positions 2 tid, 2 tid + 1; zeros where nothing was copied or the position is outside
            const uint32_t pieces = mt.ok[st];
            const uint4 rec = *reinterpret_cast<const uint4 *>(stage + 2 * kStageCodes + 16 * tid);
            const int p = ti.p0(i) + 2 * tid;
            const bool have = (pieces >> (tid >> 3)) & 1, in0 = have && p >= ti.lo && p < ti.hi, in1 = have && p + 1 >= ti.lo && p + 1 < ti.hi;
            const uint32_t k0 = in0 ? rec.x : 0u, v0 = in0 ? rec.y : 0u, k1 = in1 ? rec.z : 0u, v1 = in1 ? rec.w : 0u;
            float4 *sz = reinterpret_cast<float4 *>(sm + kOffSz + z * kSzBytes);
            sz[tid] = make_float4(lo16(k0) * fac, lo16(k1) * fac, hi16(k0), hi16(k1));
            sz[kT / 2 + tid] = make_float4(lo16(v0), lo16(v1), fmaf(8.f, lo16(v0), hi16(v0)), fmaf(8.f, lo16(v1), hi16(v1)));
            if (tid < 4) {
                const int p32 = ti.p0(i) + 32 * tid, lo = min(max(ti.lo - p32, 0), 32), hi = min(max(ti.hi - p32, 0), 32);
                const uint32_t below = hi >= 32 ? ~0u : (1u << hi) - 1, from = lo >= 32 ? 0u : ~0u << lo, two = pieces >> (2 * tid);
                mt.valid[z][tid] = below & from & ((two & 1 ? 0xffffu : 0u) | (two & 2 ? 0xffff0000u : 0u));
                if (tid == 0) mt.masked[z] = pieces != 0xffu || ti.p0(i) < ti.lo || ti.p0(i) + kT > ti.hi;
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(saddr(VALUES ? &mt.vready[b] : &mt.kready[b]));
            if (!VALUES) mbar_arrive(saddr(&mt.szready[z]));
            mbar_arrive(saddr(&mt.empty[st]));
        }
    }
}

__device__ __forceinline__ void copy_loop(const TreeArgs &a, const Tiles &ti, Meta &mt, uint8_t *sm, int b, int h, int lane) {
    const int sh = a.page_shift, ps = 1 << sh, npc = kT >> sh;               // pages of a tile
    const int32_t *pt = a.ipt + (size_t)b * a.max_pages;
    const uint64_t pol = l2_evict_first_policy();
    int next = -1;                                                           // this lane's page of the next tile
    auto page_of = [&](int i) {
        const int p = ti.p0(i) + lane * ps;
        return i < ti.n && lane < npc && p + ps > ti.lo && p < ti.hi ? pt[p >> sh] : -2;
    };
    next = page_of(0);
    int issued = ti.n;
    for (int i = 0; i < ti.n; ++i) {
        const int st = i % kStages, page = next;
        next = page_of(i + 1);
        if (page != -2 && (uint32_t)page >= (uint32_t)a.i4_pages) flag_status(a.status, OSCAR_DEV_BAD_INT4_PAGE);
        const bool have = page != -2 && (uint32_t)page < (uint32_t)a.i4_pages;
        if (i >= kStages && !wait_for(saddr(&mt.empty[st]), ((i / kStages) & 1) ^ 1)) {
            if (lane == 0) flag_status(a.status, OSCAR_DEV_WAIT_TIMEOUT);
            issued = i;
            break;
        }
        const uint32_t got = __ballot_sync(0xffffffffu, have);
        const uint32_t bar = saddr(&mt.full[st]);
        if (lane == 0) {
            uint32_t ok = 0;                                                 // by 16 positions
            for (int k = 0; k < npc; ++k)
                if ((got >> k) & 1) ok |= ((1u << (ps >> 4)) - 1) << (k * (ps >> 4));
            mt.ok[st] = ok;
            mbar_arrive_expect_tx(bar, (uint32_t)__popc(got) * ps * (2 * kRow4 + 8));
        }
        __syncwarp();
        if (have) {
            const size_t row = ((size_t)page * a.n_kv + h) << sh;
            const uint32_t dst = saddr(sm + kOffStage + st * kStageBytes);
            tma_load_1d(dst + lane * ps * kRow4, a.codes_k + row * kRow4, ps * kRow4, bar, pol);
            tma_load_1d(dst + kStageCodes + lane * ps * kRow4, a.codes_v + row * kRow4, ps * kRow4, bar, pol);
            tma_load_1d(dst + 2 * kStageCodes + lane * ps * 8, a.sz + row * 4, ps * 8, bar, pol);
        }
    }
    // every copy has landed before the CTA goes on, also where a wait ran out
    for (int i = max(0, issued - kStages); i < issued; ++i)
        if (!wait_for(saddr(&mt.full[i % kStages]), (i / kStages) & 1)) {
            if (lane == 0) {
                flag_status(a.status, OSCAR_DEV_WAIT_TIMEOUT);
                mt.stuck = 1;
            }
            break;
        }
}

// The whole warp waits, one elected lane issues.
__device__ __forceinline__ void product_loop(const TreeArgs &a, const Tiles &ti, Meta &mt, uint32_t sb, uint32_t tmem) {
    uint32_t elected;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(elected));
    const uint64_t dk = sw128_kmajor_desc(sb + kOffK), dv = mn_desc(sb + kOffV);
    uint32_t last = 0, last_phase = 0;           // the newest commit's barrier: all products so far
    auto values = [&](int j) {                   // O += p s' . codes of tile j
        const int b = j & 1;
        const uint32_t ph = (j >> 1) & 1;
        if (!wait_for(saddr(&mt.pready[b]), ph) || !wait_for(saddr(&mt.vready[b]), ph)) return false;
        tc_fence_after();
        if (elected) {
            const uint64_t d = dv + (uint64_t)(b * (kOperand >> 4));
            const uint32_t p = tmem + kColS + b * 128, o = tmem + kColO;
            mma_ts(o, p, d, kIdescMN, j != 0);
#pragma unroll
            for (int kk = 1; kk < kT / 16; ++kk) mma_ts(o, p + 8 * kk, d + (2048 >> 4) * kk, kIdescMN, 1);
            tc_commit(saddr(&mt.vfree[b]));
            tc_commit(saddr(&mt.pvdone));
        }
        last = saddr(&mt.pvdone);
        last_phase = j & 1;
        __syncwarp();
        return true;
    };
    bool ok = true;
    for (int i = 0; ok && i < ti.n; ++i) {
        const int b = i & 1;
        if (!(ok = wait_for(saddr(&mt.kready[b]), (i >> 1) & 1))) break;
        tc_fence_after();
        if (elected) {
            const uint64_t d = dk + (uint64_t)(b * (kOperand >> 4));
            const uint32_t s = tmem + kColS + b * 128, q = tmem + kColQ;
#pragma unroll
            for (int kk = 0; kk < kHeadDim / 16; ++kk) mma_ts(s, q + 8 * kk, d + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4), kIdesc, kk != 0);
            tc_commit(saddr(&mt.kfree[b]));
            tc_commit(saddr(&mt.sfull[b]));
        }
        last = saddr(&mt.sfull[b]);
        last_phase = (i >> 1) & 1;
        __syncwarp();
        if (i > 0) ok = values(i - 1);
    }
    if (ok && ti.n > 0) ok = values(ti.n - 1);
    // every product is done before its operands and tensor memory are given up, also where a wait ran out
    const bool done = !last || wait_for(last, last_phase);
    if (elected && !(ok && done)) flag_status(a.status, OSCAR_DEV_WAIT_TIMEOUT);
    if (elected && !done) mt.stuck = 1;
}

// Slot S of two tiles of 16 query rows, the BF16 rows: half of the warps a tile.  (A call: inlined it takes registers from the
// history's loops.)
__device__ __noinline__ void window_cta(const TreeArgs a, uint8_t *sm, int item, int pairs) {
    constexpr int W = kThreads / 64, bytes = std::max(join_bytes<W>(), W * 8192) + 4096;
    static_assert(2 * bytes <= kSmem - 1024, "the fragments, and the values and the join, of both lie in shared memory beside each other");
    const int half = threadIdx.x / (32 * W), warp = threadIdx.x / 32 - W * half, lane = threadIdx.x & 31;
    const int row0 = (2 * (item % pairs) + half) * kTile, h = item / pairs % a.n_kv, b = item / pairs / a.n_kv;
    const TreeRequest rq(a, b);
    const int rows = min(kTile, rq.n * a.G - row0);
    if (rows <= 0) return;                       // (the halves have barriers of their own)
    uint8_t *own = sm + half * bytes;
    Rows x;
    clear(x);
    window_warp<W, true>(a, rq, b, h, row0, rows, reinterpret_cast<uint4 *>(own + bytes - 4096), reinterpret_cast<uint4 *>(own + warp * 8192),
                         1 + half, warp, lane, x);
    tile_sync<W, true>(1 + half);                // values are read: results take their place
    join_warps<W, true>(a, rq, h, row0, rows, a.part.S, false, own, 1 + half, 32 * warp + lane, warp, lane, x);
}

// grid (S x row blocks, Hkv, batch and more): the history's CTAs, the row blocks of a split next to each other; behind them in the order
// of z those of the BF16 rows, one a request, kv head and pair of 16-row tiles, on the SMs that the former leave and, after them, on
// all.  (One launch: a second one that starts beside the first would read what earlier kernels wrote without a wait of its own for
// them.  Behind the first it cost 12 us: 8 nodes, 100K, 75 us for 61.)
__global__ void __launch_bounds__(kThreads, 1) tree_tc_kernel(const TreeArgs a, int blocks, int batch, int pairs) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
    if ((int)blockIdx.z >= batch) {
        const int item = ((blockIdx.z - batch) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
        pdl_wait();
        if (item < pairs * a.n_kv * batch) window_cta(a, sm, item, pairs);
        return;
    }
    Meta &mt = *reinterpret_cast<Meta *>(sm + kOffMeta);
    const uint32_t sb = saddr(sm);
    const int slot = blockIdx.x / blocks, row0 = blockIdx.x % blocks * kR, h = blockIdx.y, b = blockIdx.z, S = a.part.S;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kThreads / 32 - 1) {
        tmem_alloc(saddr(&mt.tmem), 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(saddr(&mt.full[i]), 1);
            mbar_init(saddr(&mt.empty[i]), 2 * kUnpackWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(saddr(&mt.kready[i]), kUnpackWarps);
            mbar_init(saddr(&mt.vready[i]), kUnpackWarps);
            mbar_init(saddr(&mt.kfree[i]), 1);
            mbar_init(saddr(&mt.vfree[i]), 1);
            mbar_init(saddr(&mt.sfull[i]), 1);
            mbar_init(saddr(&mt.pready[i]), kSoftWarps);
        }
        for (int i = 0; i < kSzBuffers; ++i) {
            mbar_init(saddr(&mt.szready[i]), kUnpackWarps);
            mbar_init(saddr(&mt.szfree[i]), kSoftWarps);
        }
        mbar_init(saddr(&mt.pvdone), 1);
        mt.max_q = 0.f;
        mt.stuck = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    const TreeRequest rq(a, b);
    const int rows = min(kR, rq.n * a.G - row0);
    const Tiles ti(a.sink, rq.he, S, slot);
    const int rep = rows <= 32 ? 4 : rows <= 64 ? 2 : 1, pad = kR / rep;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&mt.tmem);
    RowState st{0.f, kNoRef, 0.f, 0.f};
    float fac = 0.f;
    if (rows > 0 && ti.n > 0) {
        // the lane's query row, and the largest finite element of all rows: they share a scaling
        const int row = (32 * (warp & 3) + lane) % pad;
        const bool on = row < rows;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (on ? tree_row(a, rq, h, row0 + row) * kHeadDim : 0));
        float mx = 0.f, sum = 0.f;
        if (warp < kSoftWarps) {
#pragma unroll
            for (int i = 0; i < kHeadDim / 8; ++i) {
                const uint4 x = on ? src[i] : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x0 = fabsf(lo16(w[e])), x1 = fabsf(hi16(w[e]));
                    mx = fmaxf(mx, fmaxf(x0 < INFINITY ? x0 : 0.f, x1 < INFINITY ? x1 : 0.f));
                    sum += lo16(w[e]) + hi16(w[e]);
                }
            }
            st.zq = a.scale2 * sum;
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (lane == 0) atomicMax(reinterpret_cast<int *>(&mt.max_q), __float_as_int(mx));       // (not negative)
        }
        __syncthreads();
        mx = mt.max_q;
        const int ex = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 117);                  // |q| < 2^(ex + 1)
        const float m0 = __uint_as_float((uint32_t)(14 - ex + 127) << 23), m1 = m0 * 0.0625f;
        fac = a.scale2 * __uint_as_float((uint32_t)(10 + ex + 127) << 23);                           // 2^24 / m0
        // as f16, in the order of the unpacked codes, odd nibbles' channels by 1/16
        if (warp < kSoftWarps) {
#pragma unroll
        for (int ii = 0; ii < 2; ++ii) {         // each warp of a quarter one half
            const int i = 2 * (warp >> 2) + ii;
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint4 x = on ? src[4 * i + k] : make_uint4(0, 0, 0, 0);
                w[4 * k + 0] = pack_h2(lo16(x.x) * m0, lo16(x.z) * m0);
                w[4 * k + 1] = pack_h2(hi16(x.x) * m1, hi16(x.z) * m1);
                w[4 * k + 2] = pack_h2(lo16(x.y) * m0, lo16(x.w) * m0);
                w[4 * k + 3] = pack_h2(hi16(x.y) * m1, hi16(x.w) * m1);
            }
            tmem_st16(tmem + kColQ + ((uint32_t)(32 * (warp & 3)) << 16) + 16 * i, w);
        }
        tmem_st_wait();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (rows > 0 && ti.n > 0) {
        if (warp < kSoftWarps) {
            if (rep == 4) softmax_loop<4>(a, ti, mt, sm, tmem, warp, lane, st);
            else if (rep == 2) softmax_loop<2>(a, ti, mt, sm, tmem, warp, lane, st);
            else softmax_loop<1>(a, ti, mt, sm, tmem, warp, lane, st);
            if (!wait_for(saddr(&mt.pvdone), (ti.n - 1) & 1) && lane == 0) flag_status(a.status, OSCAR_DEV_WAIT_TIMEOUT);
            tc_fence_after();
        } else if (warp < kSoftWarps + kUnpackWarps) {
            unpack_loop<false>(a, ti, mt, sm, threadIdx.x - 32 * kSoftWarps, lane, fac);
        } else if (warp < kSoftWarps + 2 * kUnpackWarps) {
            unpack_loop<true>(a, ti, mt, sm, threadIdx.x - 32 * (kSoftWarps + kUnpackWarps), lane, fac);
        } else if (warp == kSoftWarps + 2 * kUnpackWarps) {
            copy_loop(a, ti, mt, sm, b, h, lane);
        } else {
            product_loop(a, ti, mt, sb, tmem);
        }
    }
    __syncwarp();
    __syncthreads();                             // every copy and product is done: results take the operands' place
    const bool write = rows > 0 && !mt.stuck;    // (or one was waited for in vain, and flagged: there are no results)
    float *res = reinterpret_cast<float *>(sm), *rm = res + kR * kResRow, *rl = rm + kR, *rz = rl + 2 * kR;
    const int half = warp >> 2, at = 32 * (warp & 3) + lane;
    if (warp < kSoftWarps && write) {
        rl[half * kR + at] = st.l;
        rz[half * kR + at] = st.zs;
    }
    __syncthreads();
    if (warp < kSoftWarps && write) {
        const float l = rl[at] + rl[kR + at], zs = rz[at] + rz[kR + at];
        if (half == 0) rm[at] = l > 0.f ? st.M : l != l ? l : -INFINITY;         // (NaN where a logit was: it has to reach the row)
        if (ti.n > 0)
#pragma unroll 1
            for (int c = 2 * half; c < 2 * half + 2; ++c) {
                uint32_t r[32];
                tmem_ld32(tmem + kColO + ((uint32_t)(32 * (warp & 3)) << 16) + 32 * c, r);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k) {    // a code word's columns are its channels 0 4 1 5 2 6 3 7
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[(j >> 1) + 4 * (j & 1)] = __uint_as_float(r[8 * k + j]) + zs;
                    float *to = res + at * kResRow + 32 * c + 8 * k;
                    *reinterpret_cast<float4 *>(to) = make_float4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<float4 *>(to + 4) = make_float4(x[4], x[5], x[6], x[7]);
                }
            }
    }
    tc_fence_before();
    __syncthreads();
    // a row's copies joined, a warp a row
    for (int row = write ? warp : rows; row < rows; row += kThreads / 32) {
        float M = -INFINITY;
        for (int k = 0; k < rep; ++k) M = fmaxf(M, rm[row + k * pad]);
        float L = 0.f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < rep; ++k) {
            const int from = row + k * pad;
            const float f = rm[from] != -INFINITY ? exp2f(rm[from] - M) : 0.f;
            if (f == 0.f) continue;
            const float4 x = *reinterpret_cast<const float4 *>(res + from * kResRow + 4 * lane);
            L = fmaf(rl[from] + rl[kR + from], f, L);
            A = make_float4(fmaf(x.x, f, A.x), fmaf(x.y, f, A.y), fmaf(x.z, f, A.z), fmaf(x.w, f, A.w));
        }
        const size_t to = tree_row(a, rq, h, row0 + row) * (S + 1) + slot;
        *reinterpret_cast<float4 *>(a.part.acc + to * kHeadDim + 4 * lane) = A;
        if (lane == 0) {
            a.part.m[to] = L != L ? L : M;
            a.part.l[to] = L;
        }
    }
    if (warp == kThreads / 32 - 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

// Layers of z behind the history's that hold the BF16 rows' CTAs.
static long long window_layers(const TreeArgs &a, int max_rows, int batch) {
    const long long layer = (long long)a.part.S * ((max_rows + kR - 1) / kR), items = (long long)((max_rows + 2 * kTile - 1) / (2 * kTile)) * batch;
    return (items + layer - 1) / layer;
}

bool tree_tc_fits(const TreeArgs &a, int max_rows, int batch) { return batch + window_layers(a, max_rows, batch) <= 65535; }

cudaError_t launch_tree_tc(const TreeArgs &a, int max_rows, int batch, cudaStream_t st) {
    if (cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(tree_tc_kernel), kSmem)) return e;
    const int blocks = (max_rows + kR - 1) / kR, pairs = (max_rows + 2 * kTile - 1) / (2 * kTile);
    return launch_ahead(tree_tc_kernel, dim3(a.part.S * blocks, a.n_kv, (unsigned)(batch + window_layers(a, max_rows, batch))), kThreads, kSmem, st, a, blocks,
                        batch, pairs);
}

}  // namespace oscar
