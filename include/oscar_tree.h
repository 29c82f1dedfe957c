/*
 * oscar_tree.h — a step of speculative decoding over the mixed cache of liboscar.so: attention of a tree of
 * drafted tokens per request, the token sampled at each of them, and the accepted path moved into the cache.
 *
 * A request's tree has n nodes: node 0 is its newest token (known, not yet in the cache), the others are
 * drafted.  Node j's key and value are the BF16 rows at position seq_len + j (oscar_append_kv writes them,
 * with the node's depth in the tree as its place in the text), whatever the node's depth.  A step is then
 *   oscar_append_kv               the nodes' q, k, v
 *   oscar_tree_attention_int4     per layer: every node over the cache and the nodes it may see
 *   oscar_sample                  a token per node from the model's logits
 *   oscar_tree_accept             the path that the sampled tokens confirm; its rows moved together
 * after which the cache ends at the new length and oscar_demote_int4 goes on as after any step.
 * Memory, streams and errors follow oscar.h: device pointers owned by the caller, asynchronous calls on the
 * caller's stream, host checks before anything is enqueued, device checks that skip and flag.  Every call
 * keeps the order of its stream.  Calls that may run concurrently must not share partials or outputs;
 * nothing is kept between calls, and no output may overlap an input.
 */
#ifndef OSCAR_TREE_H
#define OSCAR_TREE_H

#include "oscar_int4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define OSCAR_TREE_MAX_NODES 256

/* A history split count for oscar_tree_attention_int4 and _bounded that fills the GPU (1..1024); max_nodes: nodes
 * of the largest tree; max_hist_tokens: of the longest history, for which the kernel of the history is chosen too
 * (oscar_tree_attention_int4_bounded takes the same number). */
OSCAR_API int32_t oscar_suggest_splits_tree_int4(const oscar_layout_t *layout, int32_t batch, int32_t max_nodes,
                                                 int32_t max_hist_tokens, int32_t sm_count);

/*
 * Attention of every node of every request's tree over [BF16 sink | INT4 history | BF16 recent] and the
 * nodes it may see: with b its request, T = seq_len[b] and he = hist_end[b], node i meets the positions
 * [0, T) as oscar_decode_attention_int4 does and the position T + j of every node j it sees.
 *   q           bf16 [n][Hq][head_dim], 16-byte aligned: the nodes of request 0, then of request 1, ...
 *   node_begin  int32 [batch + 1]: request b's nodes are the rows [node_begin[b], node_begin[b + 1]).
 *               Rows from node_begin[batch] on, and the outputs there, are left alone.
 *   mask        int32 [n][mask_words], 32 nodes a word: node i of a request sees its node j if bit j % 32
 *               of word j / 32 of row i is set (bits from the request's node count on are not read).
 *               mask_words at least max_nodes / 32, rounded up.  A node's own bit has no other meaning than
 *               the others'.  NULL: node i sees the nodes 0 .. i (a chain, as of a prompt's chunk).
 *   max_nodes   1..OSCAR_TREE_MAX_NODES, at least the nodes of every request.
 *   page tables hold the nodes' positions too: T + nodes <= max_pages_per_req·page_size.
 *   partials    scratch for n rows (oscar_partials_ml_floats(layout, n, S) and so on).
 *   out         bf16 [n][Hq][head_dim], 8-byte aligned; lse (optional) fp32 [n][Hq], natural logarithm.
 * A node that sees nothing (an empty mask row where T = 0) gets out = 0 and lse = -inf.  What a node does not
 * see does not reach its output, infinities and NaN included; a NaN among the logits of what it sees makes its output
 * and lse NaN.  A request with a bad node range, or whose nodes pass the page table, is skipped and flagged
 * (OSCAR_DEV_BAD_LENGTH); rows on a bad page are not seen, and flagged.  Where node_begin falls, ranges of other
 * requests may share node rows, whose outputs are then nobody's.
 * Query products and softmax sums are fp32 or finer.  Of the history, a probability times its value scale
 * enters the value product as one fp16 number (2^-11 relative) under a scaling that follows the largest one
 * so far, and meets codes less 8; of the BF16 rows a probability enters in two bf16 parts (2^-16).  (The decode
 * call keeps two fp16 parts.  Before they are rounded to bf16, which takes 1.6·10^-3 of their norm, outputs here are
 * off by 2 to 3·10^-4 of it.)  The tensor cores
 * cut a split's running sums off at 2^-23 every 16 positions: splits as suggested are 16K positions long at most, or
 * 4K a warp, and a count below the suggestion's makes them longer.  Query elements below 2^-25 of the largest finite
 * one that shares a scaling with them lose low bits: their head's, or, on the kernel for many rows, the largest of 128
 * rows (nodes times query heads of a kv head); from 2^118 on they count as infinite.  Logits (times log2 e) are expected
 * within 2^26: beyond, where fp32's last bit is 8 and more, outputs may be infinite or NaN.
 */
OSCAR_API oscar_status_t oscar_tree_attention_int4(const oscar_layout_t *layout, const uint16_t *q, int32_t n,
                                                   const int32_t *node_begin, const int32_t *mask,
                                                   int32_t mask_words, int32_t max_nodes,
                                                   const oscar_bf16_pool_t *bf16_pool,
                                                   const int32_t *bf16_page_table,
                                                   const oscar_int4_pool_t *int4_pool,
                                                   const int32_t *int4_page_table, int32_t max_pages_per_req,
                                                   const int32_t *seq_len, const int32_t *hist_end, int32_t batch,
                                                   float sm_scale, const oscar_partials_t *partials, uint16_t *out,
                                                   float *lse, void *stream);

/*
 * The same call for histories of at most max_hist_tokens (1 and more), of which there may be fewer than the page tables
 * have room for.  Which of two kernels takes the history goes by this bound, in oscar_suggest_splits_tree_int4 as here;
 * oscar_tree_attention_int4 goes by the page tables' room, max_pages_per_req·page_size.  A table as wide as the longest
 * request a server admits wants the bound: the kernel for long histories is slower on short ones.  The bound decides
 * on time and last bits alone: longer histories are met in full.
 */
OSCAR_API oscar_status_t oscar_tree_attention_int4_bounded(const oscar_layout_t *layout, const uint16_t *q, int32_t n,
                                                           const int32_t *node_begin, const int32_t *mask,
                                                           int32_t mask_words, int32_t max_nodes,
                                                           const oscar_bf16_pool_t *bf16_pool,
                                                           const int32_t *bf16_page_table,
                                                           const oscar_int4_pool_t *int4_pool,
                                                           const int32_t *int4_page_table, int32_t max_pages_per_req,
                                                           int32_t max_hist_tokens, const int32_t *seq_len,
                                                           const int32_t *hist_end, int32_t batch, float sm_scale,
                                                           const oscar_partials_t *partials, uint16_t *out, float *lse,
                                                           void *stream);

/* Types of logits. */
#define OSCAR_DTYPE_F32 0
#define OSCAR_DTYPE_BF16 1
#define OSCAR_DTYPE_F16 2

#define OSCAR_SAMPLE_MAX_VOCAB 262144

/*
 * One token per row of logits, by the row's temperature, filters and uniform number.  With x a row, m its
 * largest logit, w_i = exp((x_i - m) / temperature), and the row's tokens ordered by falling logit (ties: the
 * lowest index first), the kept tokens are the first ones of that order, as many as every filter allows:
 *   top_k  the first top_k tokens                                   (off: NULL, or a value <= 0)
 *   top_p  of those, the fewest first ones whose w sum to at least top_p of their total
 *                                                                  (off: NULL, or a value >= 1 or NaN;
 *                                                                   a value <= 0 keeps one token)
 *   min_p  the tokens with w_i >= min_p                             (off: NULL, or a value <= 0 or NaN)
 * and one at least.  The token is the kept one of lowest index i for which the w of the kept tokens up to and
 * including i sum to more than u times their total.
 *   logits       [rows][vocab] of the given type, row r at logits + r·stride (elements; stride >= vocab, or 0: one
 *                row for all); any alignment of the type.  -inf: never drawn.  NaN counts as -inf.  Where the largest logit is
 *                +inf, the tokens that have it share the weight alone.
 *   temperature  fp32 [rows]; 0 (or less, or NaN): the largest logit's lowest index, the filters and u are not
 *                read; +inf: every finite logit weighs the same.
 *   u            fp32 [rows] in [0, 1) (values outside are clamped to it).
 *   tokens       int32 [rows]; -1 for a row with no logit above -inf.
 * Weights below 2^-44 of the largest one count as zero; the others enter as whole multiples of it, within 2^-30 of
 * their size or one unit, so a sum does not depend on its order, and the token on nothing but the arguments.
 */
OSCAR_API oscar_status_t oscar_sample(const void *logits, int32_t dtype, int64_t stride, int32_t rows, int32_t vocab,
                                      const float *temperature, const int32_t *top_k, const float *top_p,
                                      const float *min_p, const float *u, int32_t *tokens, void *stream);

/*
 * The accepted path of every request's tree, and its rows moved together.  From node 0 on: a node is accepted;
 * its next one is the child (lowest index first) whose drafted token is the one that was sampled at the node;
 * without such a child the path ends.
 *   target      int32 [n]: the token sampled at each node (oscar_sample).
 *   draft       int32 [n]: the token each node stands for (node 0's is not read).
 *   parents     int32 [n]: the parent's index in its request's tree, below the node's own (node 0's is not read).
 *               A node whose parent is not in [0, its own index) is nobody's child.
 *   node_begin  as for oscar_tree_attention_int4; seq_len int32 [batch] the length without the nodes.
 *   accepted    int32 [batch]: nodes on the path, node 0 among them.
 *   path        int32 [batch][path_stride]: their indices, then -1.
 *   tokens      int32 [batch][path_stride]: the tokens sampled at them (the step's output; the last one is the
 *               next step's node 0), then -1.  path_stride >= max_nodes.
 *   new_len     int32 [batch] or NULL: seq_len + accepted; not the array seq_len itself.
 *   pools       host array of n_pools BF16 pools (each layer's; 0 and NULL: nothing is moved), of the same
 *               layout and page table [batch][max_pages_per_req].  The rows of path node i, every kv head, move
 *               to position seq_len + i.  No two requests may share the pages of those positions.  The arrays of all
 *               pools, keys and values, lie apart (refused otherwise).
 * A request with no nodes gets accepted = 0.  One with a bad node range, a bad seq_len, or nodes that pass the
 * page table (where pools are given) is skipped and flagged (OSCAR_DEV_BAD_LENGTH): accepted = 0, an empty path,
 * new_len = seq_len.  A row from or to a bad page is not moved, and flagged (OSCAR_DEV_BAD_BF16_PAGE).
 */
OSCAR_API oscar_status_t oscar_tree_accept(const oscar_layout_t *layout, const int32_t *target, const int32_t *draft,
                                           const int32_t *parents, int32_t n, const int32_t *node_begin,
                                           int32_t max_nodes, const int32_t *seq_len, int32_t batch,
                                           int32_t *accepted, int32_t *path, int32_t *tokens, int32_t path_stride,
                                           int32_t *new_len, const oscar_bf16_pool_t *pools, int32_t n_pools,
                                           const int32_t *page_table, int32_t max_pages_per_req, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* OSCAR_TREE_H */
