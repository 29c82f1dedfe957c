/*
 * oscar_int4.h — the 4-bit history of liboscar.so: a cache laid out as [BF16 sink | INT4 history | BF16
 * recent], written, attended to, weighed and evicted from.
 *
 * The OSCAR pages measure their 2-bit history against a 4-bit one (OSCAR news article, Fig. 3 paragraph:
 * the 4-bit reference at 4.25 bits per element).  This header adds that tier next to the 2-bit one: the
 * same layout, BF16 pool, page tables, partials and merge as oscar.h, another pool.  Memory, streams and
 * errors follow oscar.h: device pointers owned by the caller, asynchronous calls on the caller's stream,
 * host checks before anything is enqueued, device checks that skip and flag.  Every call keeps the order
 * of its stream: it is set up while the kernel before it ends, and reads memory once that has completed.
 * What the 4-bit calls cost a step:
 *   oscar_append_kv              the step's q, k, v: normalised, rotated, k and v into the BF16 pool
 *   oscar_decode_attention_int4  attention over history and BF16 rows, with the merge
 *   oscar_attention_mass_int4    optional: the weights an eviction ranks by
 *   oscar_demote_int4            the token that leaves the recent window (or a prompt's whole history)
 * and between steps, oscar_evict_int4 and oscar_promote_int4.
 */
#ifndef OSCAR_INT4_H
#define OSCAR_INT4_H

#include "oscar.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status bit, next to those of oscar.h. */
#define OSCAR_DEV_BAD_INT4_PAGE 0x10  /* INT4 page id outside [0, n_pages) */

/*
 * Paged INT4 pool of one layer (device memory, caller-owned): the history of a cache kept at 4 bits
 * (the 4-bit reference of the OSCAR pages, 4.25 bits per element at group 128), stored as it is given,
 * without a rotation.  A page holds one kv head's tokens together:
 *   codes_k, codes_v : uint8 [n_pages][n_kv_heads][page_size][head_dim/2], channel c of a row in bits
 *                      4·(c mod 2) .. 4·(c mod 2) + 3 of byte c/2
 *   scale_zero       : bf16 bits [n_pages][n_kv_heads][page_size][head_dim/group][4]: key scale, key
 *                      zero, value scale, value zero of each group of `group` consecutive channels
 * A row's quantizer, per group: lo = c·min, hi = c·max (fp32; a signed zero read as +0), zero =
 * bf16(lo), scale = bf16((hi - lo)/15), code = the integer nearest to (x - zero)/scale (ties to even,
 * decided on the exact quotient), clamped to 0..15, code 0 if scale == 0.  Value: zero + code·scale.
 * Rows are expected finite, their range below the largest float.  All three base addresses must be
 * 16-byte aligned, and n_pages·n_kv_heads·page_size must be below 2^31.
 */
typedef struct {
    uint8_t *codes_k;
    uint8_t *codes_v;
    uint16_t *scale_zero;
    int32_t n_pages;
} oscar_int4_pool_t;

/*
 * New tokens into the BF16 cache: for each token i < n, with b = req_idx[i] and p = positions[i],
 *   q_out[i][h] = rope(rms(q[i][h]) * q_weight),  every query head h < Hq
 *   pool.k at (page_table[b·max_pages_per_req + p/ps], p % ps, h) = rope(rms(k[i][h]) * k_weight)
 *   pool.v there = v[i][h],  every kv head h < n_kv_heads
 * with rms(x) = x / sqrt(mean(x^2) + eps) over the head's 128 channels and rope the rotation of the
 * first rot_dim channels by the token's row of `rope`; all in fp32, rounded once to bf16.
 *   q, k, v        bf16, token i's heads at q + i·q_stride (elements): [Hq][head_dim], k and v
 *                  [n_kv_heads][head_dim]; 16-byte aligned, strides multiples of 8 and at least a
 *                  token's row (slices of one projection's output need no copy).  q and q_out may
 *                  both be NULL: keys and values only.
 *   q_weight, k_weight  bf16 [head_dim], or NULL: that tensor is not normalised.
 *   rope           fp32 [rope_rows][128], row r: cos of its 64 angles, then their sin; channel pair
 *                  j < rot_dim/2 turns by angle j: (a, b) -> (a cos - b sin, b cos + a sin).
 *                  interleaved = 0: pair j is channels j and j + rot_dim/2; 1: channels 2j, 2j + 1.
 *                  rot_dim a multiple of 16 up to 128.  NULL: no rotation.
 *   positions      int32 [n] cache positions; -1 marks a padding token, for which nothing is written.
 *   rope_positions int32 [n] or NULL (= positions): the rows of `rope`, where a token's position in
 *                  the text is not its place in the cache (after oscar_evict_int4).
 *   q_out          bf16 [n][Hq][head_dim], 16-byte aligned; may be q itself if q_stride = Hq·head_dim.
 * A token whose req_idx, position or rope row is out of range is skipped and flagged
 * (OSCAR_DEV_BAD_LENGTH); one whose page is bad still gets its q_out (OSCAR_DEV_BAD_BF16_PAGE).
 * Two tokens of one call with the same slot race.  n = 0 is a no-op.
 */
OSCAR_API oscar_status_t oscar_append_kv(const oscar_layout_t *layout, const uint16_t *q, int64_t q_stride,
                                         const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                                         int32_t n, const uint16_t *q_weight, const uint16_t *k_weight, float eps,
                                         const float *rope, int32_t rope_rows, int32_t rot_dim, int32_t interleaved,
                                         const oscar_bf16_pool_t *pool, const int32_t *page_table,
                                         int32_t max_pages_per_req, int32_t batch, const int32_t *req_idx,
                                         const int32_t *positions, const int32_t *rope_positions, uint16_t *q_out,
                                         void *stream);

/*
 * BF16 rows to the INT4 pool, as stored (no rotation): every position p in [pos_begin[b], pos_end[b])
 * of every request, every kv head, K with clip ratio c_K and V with c_V.  One token per step and a
 * whole prompt's history are the same call.  Ranges as for oscar_demote_range: pos_begin, pos_end int32
 * [batch]; a bad one is skipped and flagged (OSCAR_DEV_BAD_LENGTH), an empty one demotes nothing; rows
 * on a bad page are skipped and flagged.  Positions that two requests map to the same INT4 slot race.
 */
OSCAR_API oscar_status_t oscar_demote_int4(const oscar_layout_t *layout, const oscar_bf16_pool_t *src,
                                           const int32_t *bf16_page_table, const oscar_int4_pool_t *dst,
                                           const int32_t *int4_page_table, int32_t max_pages_per_req, int32_t batch,
                                           const int32_t *pos_begin, const int32_t *pos_end, float c_K, float c_V,
                                           void *stream);

/*
 * The way back: every position in [pos_begin[b], pos_end[b]) of the INT4 pool restored (zero +
 * code·scale, rounded once to bf16) into the BF16 pool's page of that position, for a consumer that
 * reads BF16 (a prompt's next chunk).  Ranges, pages and errors as for oscar_demote_int4.
 */
OSCAR_API oscar_status_t oscar_promote_int4(const oscar_layout_t *layout, const oscar_int4_pool_t *src,
                                            const int32_t *int4_page_table, const oscar_bf16_pool_t *dst,
                                            const int32_t *bf16_page_table, int32_t max_pages_per_req, int32_t batch,
                                            const int32_t *pos_begin, const int32_t *pos_end, void *stream);

/* A history split count for oscar_decode_attention_int4 that fills the GPU (1..1024). */
OSCAR_API int32_t oscar_suggest_splits_int4(const oscar_layout_t *layout, int32_t batch, int32_t max_hist_tokens,
                                            int32_t sm_count);

/*
 * Decode attention over [BF16 sink | INT4 history | BF16 recent]: arguments as for
 * oscar_decode_attention, with the unrotated bf16 q (16-byte aligned) against both pools and an INT4
 * pool as the history.  Any n_kv_heads; the layout's codebook levels are not used.
 * Writes every slot of `partials`: the history is cut into S splits of whole 32-token blocks (at absolute
 * positions 32 i), the BF16 rows are dealt out to the same splits, slot S is written empty.  With out or
 * out_f32 non-NULL also their merge, as oscar_merge(R_V = NULL) defines it, lse optional.  Query products and softmax sums are fp32 or finer;
 * a probability times its value scale enters the value product in two fp16 parts (2^-21 relative, or 2^-30 of the
 * largest one so far); of 16 tokens' products with their codes, what lies 2^-17 below a unit of the largest is cut off.
 * Query elements below 2^-25 of their head's largest lose low bits.
 *   merge_counters  NULL: the merge is a second launch.  Else int32 [batch·n_kv_heads], all zero, left
 *                   zero: the last CTA of a request's kv head to finish merges it, in the same launch
 *                   and in slot order whichever CTA that is.  Calls that may run concurrently must
 *                   share neither merge_counters nor partials.
 * A request with seq_len 0 gets out = 0, lse = -inf.
 */
OSCAR_API oscar_status_t oscar_decode_attention_int4(const oscar_layout_t *layout, const uint16_t *q,
                                                     const oscar_bf16_pool_t *bf16_pool,
                                                     const int32_t *bf16_page_table,
                                                     const oscar_int4_pool_t *int4_pool,
                                                     const int32_t *int4_page_table, int32_t max_pages_per_req,
                                                     const int32_t *seq_len, const int32_t *hist_end, int32_t batch,
                                                     float sm_scale, const oscar_partials_t *partials, uint16_t *out,
                                                     float *out_f32, float *lse, int32_t *merge_counters,
                                                     void *stream);

/*
 * The attention weight of one decode step, added to a running sum per position (what an eviction by
 * accumulated attention weight ranks by): for every request b, kv head h and position p < seq_len[b],
 *   mass[b][h][p] += sum over h's query heads of exp(sm_scale·q·k_p - lse)
 * over the same rows as oscar_decode_attention_int4, whose lse it takes.
 *   lse   fp32 [batch][Hq] natural log-sum-exp; a head with lse = -inf adds nothing.
 *   mass  fp32 [batch][n_kv_heads][max_pages_per_req·page_size]; positions from seq_len on and those on
 *         a bad page are left as they were.
 * Every position is added to once, by one thread: the sums do not depend on the order of execution.
 */
OSCAR_API oscar_status_t oscar_attention_mass_int4(const oscar_layout_t *layout, const uint16_t *q,
                                                   const oscar_bf16_pool_t *bf16_pool,
                                                   const int32_t *bf16_page_table,
                                                   const oscar_int4_pool_t *int4_pool,
                                                   const int32_t *int4_page_table, int32_t max_pages_per_req,
                                                   const int32_t *seq_len, const int32_t *hist_end, int32_t batch,
                                                   float sm_scale, const float *lse, float *mass, void *stream);

/*
 * Eviction from the INT4 history by accumulated weight: of request b's history [sink, hist_end[b]),
 * each kv head keeps the keep[b] positions of largest mass (ties: the lowest position first; NaN ranks
 * above every number) and their rows move, in ascending position order, to positions sink, sink + 1, ...
 * of the pages in dst_page_table.  Heads keep different tokens; the new history end is sink + keep[b].
 *   src, src_page_table / dst, dst_page_table   both tables [batch][max_pages_per_req].  src and dst may
 *             be the same pool, but no destination page may be a source page of any request (a kept row
 *             moves while others are still read); the same table for both is refused.  The source pages
 *             are only read, so requests may share them (a common prefix).
 *   keep      int32 [batch]; -1: request b is left alone, nothing of it is written.  Outside
 *             [0, hist_end - sink] or above kept_stride: skipped and flagged (OSCAR_DEV_BAD_LENGTH).
 *   mass      fp32 [batch][n_kv_heads][max_pages_per_req·page_size], as oscar_attention_mass_int4 leaves it.
 *   mass_out  same shape, not overlapping mass: the weights at the new positions: [0, sink) as they were,
 *             the kept ones, then those of [hist_end, seq_len), then 0.
 *   kept      int32 [batch][n_kv_heads][kept_stride]: the old position of each kept row, ascending;
 *             entries from keep[b] on are left as they were.
 * Positions in the cache shrink by hist_end - sink - keep: pass the tokens' positions in the text to
 * oscar_append_kv as rope_positions from then on.  When that is a multiple of page_size the request's
 * recent BF16 pages need no copy, only their places in its page table.
 */
OSCAR_API oscar_status_t oscar_evict_int4(const oscar_layout_t *layout, const oscar_int4_pool_t *src,
                                          const int32_t *src_page_table, const oscar_int4_pool_t *dst,
                                          const int32_t *dst_page_table, int32_t max_pages_per_req, int32_t batch,
                                          const int32_t *seq_len, const int32_t *hist_end, const int32_t *keep,
                                          const float *mass, float *mass_out, int32_t *kept, int32_t kept_stride,
                                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* OSCAR_INT4_H */
