/*
 * bq_decode.h - C ABI of the decoding operators of libbq.so: what chooses
 * the next tokens from logits, and what verifies a tree of drafted tokens
 * over the 4-bit cache of bq_layer.h in one pass.
 *
 *   - a tree's visibility masks and positions (bq_tree_mask);
 *   - attention of its nodes over the prefix and their ancestors
 *     (bq_attn_kv4_tree);
 *   - sampling with temperature, top-k, top-p and min-p from given random
 *     numbers (bq_sample);
 *   - the walk down the tree along the sampled tokens (bq_tree_accept);
 *   - the move of the accepted tokens' keys and values to the places behind
 *     the prefix (bq_kv4_compact).
 *
 * The conventions of bq.h and bq_layer.h hold (device pointers owned by the
 * caller, streams, errors, no device memory allocated, reentrancy; index
 * arrays are device memory that the host does not read, and an index outside
 * its range is never followed).  What a call does not compute stays as it was.
 *
 * A tree is a list of nodes, the parent of node i a node before it, node 0
 * the root: the last token that is certain.  The nodes of sequence b are the
 * last ones of its cache: node i of q_len is key seq_len - q_len + i, whatever
 * its depth; the keys before node 0 are the prefix.  q_start [batch + 1] int32
 * gives the first node of each sequence in the arrays over all nodes, then the
 * end; each is taken within [0, total_q], and a sequence whose end is not past
 * its start has none; q_start NULL: max_q_len nodes each (total_q = batch *
 * max_q_len, BQ_ERR_SHAPE otherwise).  max_q_len, at most BQ_TREE_MAX, is the
 * most nodes of one sequence that are computed, its first ones; q_len counts
 * all of them.
 */
#ifndef BQ_DECODE_H
#define BQ_DECODE_H

#include "bq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BQ_TREE_MAX 1024
#define BQ_F32 2 /* logits' type, beside enum bq_dtype */

/*
 * bq_tree_mask - what each node sees, and its position:
 *   bit j % 32 of mask[i][j / 32] is set for node i itself and its ancestors,
 *   position[i] = seq_len - q_len + depth of i (the root's is 0).
 *
 *   parents    [total_q] int32, the parent's number within its tree; one that
 *              is not in [0, i) makes node i a root of its own
 *   seq_lens   [batch] int32, keys in the cache with the nodes; NULL: 0, and
 *              q_len is not subtracted (position = depth)
 *   mask       [total_q, mask_words] 32-bit words, bits past q_len are 0; node
 *              32 * mask_words and what is past it has no bit
 *   positions  [total_q] int32, or NULL
 * 1 <= mask_words <= BQ_TREE_MAX / 32 (BQ_ERR_SHAPE).
 */
int bq_tree_mask(const int32_t *parents, const int32_t *q_start, const int32_t *seq_lens, int64_t batch, int64_t total_q,
                 int64_t max_q_len, int64_t mask_words, uint32_t *mask, int32_t *positions, void *stream);

/*
 * bq_attn_kv4_tree - bq_attn_kv4 for the nodes of trees: a row attends to the
 * whole prefix and to the nodes of its mask, and with window > 0 to the last
 * `window` of these keys only (in the order of the cache).
 *
 *   mask       [total_q, mask_words] 32-bit words, any bits (bq_tree_mask
 *              gives a node and its ancestors): bit j % 32 of word j / 32 of a
 *              row is node j; bits at or past q_len count as 0, and so does a
 *              node before the start of the cache (q_len > seq_len)
 * The other arguments, and what is said of them, are those of bq_attn_kv4;
 * a row that sees no key gives zeros (lse -infinity).  Which kernel a call takes
 * and how it is split go by max_blocks * page_size, not by seq_lens, which the host
 * does not read: a table no wider than its sequences is the faster one.
 * 1 <= mask_words <= BQ_TREE_MAX / 32 (BQ_ERR_SHAPE).
 */
int bq_attn_kv4_tree(const void *q, int64_t q_stride, int dtype, const int32_t *q_start, const int32_t *seq_lens,
                     const int32_t *block_table, int64_t batch, int64_t total_q, int64_t max_q_len, int q_heads,
                     int kv_heads, int head_dim, const void *cache, int64_t num_pages, int page_size, int64_t max_blocks,
                     const uint32_t *mask, int64_t mask_words, float softmax_scale, int64_t window, void *out, float *lse,
                     void *workspace, int64_t workspace_bytes, void *stream);

/* Device workspace bytes with which bq_attn_kv4_tree splits sequences of up
 * to max_len keys (max_blocks * page_size); 0: it does not split; negative:
 * -BQ_ERR_SHAPE.  Host-only. */
int64_t bq_attn_kv4_tree_workspace_bytes(int64_t batch, int64_t max_q_len, int q_heads, int kv_heads, int head_dim,
                                         int64_t max_len);

/*
 * bq_sample - one token per row of logits, by the row's own settings.  The
 * weight of token i is w_i = exp((x_i - max x) / temperature).  In descending
 * order of x, equal ones by index, it is kept if
 *   top-k   it is one of the first top_k                    (top_k > 0), and
 *   top-p   the weights before it that top-k keeps sum to less than top_p
 *           times those of all tokens that top-k keeps      (top_p < 1), and
 *   min-p   w_i >= min_p, min_p taken at most 1             (min_p > 0);
 * the first one always is.  The token is the first one in the order of indices
 * at which the kept weights up to and with it sum to more than u times all kept
 * weights, the last kept one if none is.
 *
 *   logits       rows x vocab of dtype (BQ_F16, BQ_BF16 or BQ_F32), row_stride
 *                elements between rows (at least vocab).  -infinity and NaN
 *                have weight 0 and are not drawn; beside +infinity all finite
 *                ones have
 *   u            [rows] fp32 in [0, 1); below 0 counts as 0, others draw the
 *                last kept token
 *   temperature  [rows] fp32, or NULL (1); not above 0, or NaN: the first
 *                token of the greatest logit, whatever the other settings are
 *   top_k        [rows] int32, or NULL: off; off where it is not above 0
 *   top_p, min_p [rows] fp32, or NULL: off
 *   tokens       [rows] int32; -1 for a row whose logits are all -infinity or
 *                NaN
 *   logprobs     [rows] fp32, or NULL: the log of the probability with which
 *                the token is drawn, log(w / all kept weights); -infinity
 *                beside token -1
 *   workspace    device memory, 16-byte aligned, no particular contents; NULL
 *                with 0 bytes, or fewer than bq_sample_workspace_bytes, for
 *                none (one workgroup a row then does all of its work).  Calls
 *                that share one must not overlap.
 * A row with top_k is fastest up to some 48 to 256, by the sizes; a greater top_k
 * costs several times as much.
 * Weights are held as multiples of 2^-F of the greatest one, F = min(46, 61 -
 * ceil(log2 vocab)), from a 64-bit exponential, and one that rounds to 0 is not
 * drawn; their sums are exact, so that the result does not depend on the order in
 * which they are taken, nor on the workspace.  In a log probability only the sum
 * is of such multiples; w is the logit's own, however small.
 * 0 <= rows <= BQ_MAX_DIM, 1 <= vocab <= 2^24 (BQ_ERR_SHAPE); logits aligned to
 * their type.
 */
int bq_sample(const void *logits, int64_t row_stride, int dtype, int64_t rows, int64_t vocab, const float *u,
              const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
              float *logprobs, void *workspace, int64_t workspace_bytes, void *stream);

/* Device workspace bytes with which bq_sample shares rows between workgroups
 * (0: it does not); negative: -BQ_ERR_SHAPE.  Host-only. */
int64_t bq_sample_workspace_bytes(int64_t rows, int64_t vocab, int dtype);

/*
 * bq_tree_accept - the path from the root on which each node's token is the
 * one that was sampled at its parent; of several such children the first.
 *
 *   tokens, parents  [total_q] int32: the drafted tree
 *   sampled          [total_q] int32: the model's token at each node
 *   path             [batch, max_path] int32: the nodes of the path, path[0] =
 *                    0, in ascending order, then -1
 *   count            [batch] int32: nodes of the path, from 1 to max_path (the
 *                    walk stops there); 0 for a sequence without nodes
 *   next_token       [batch] int32: the token sampled at the last of them; -1
 *                    for a sequence without nodes
 * Nodes whose parent is not a node before them are not reached.  1 <= max_path
 * <= BQ_TREE_MAX (BQ_ERR_SHAPE).
 */
int bq_tree_accept(const int32_t *tokens, const int32_t *parents, const int32_t *sampled, const int32_t *q_start,
                   int64_t batch, int64_t total_q, int64_t max_q_len, int64_t max_path, int32_t *path, int32_t *count,
                   int32_t *next_token, void *stream);

/*
 * bq_kv4_compact - moves keys and values within the cache, for every kv head
 * and layer: key (prefix + path[j]) to (prefix + j) for the first count[b]
 * entries of a path, prefix = seq_len - q_len, as if all were read before any
 * is written.
 *
 *   cache         num_layers caches of num_pages pages, layer_stride bytes
 *                 between them (a multiple of 16, at least a cache's bytes),
 *                 all with the same block table
 *   q_start, max_q_len  the nodes, as above; here only their numbers count
 *                 (max_q_len bounds nothing but where q_start is NULL)
 *   path          [batch, max_path] int32, count [batch] int32 (taken within
 *                 [0, max_path]): an entry that is not in [j, q_len) is left
 *                 out, and so is one whose key or place lies outside the
 *                 block table or the cache
 *   seq_lens      [batch] int32, keys with the nodes
 * No two sequences share a page that is written.  1 <= max_path <= BQ_TREE_MAX,
 * 0 <= num_layers <= 65536 (BQ_ERR_SHAPE); head_dim, page_size, kv_heads and
 * max_blocks as for bq_attn_kv4.
 */
int bq_kv4_compact(void *cache, int64_t num_layers, int64_t layer_stride, int64_t num_pages, int page_size, int kv_heads,
                   int head_dim, const int32_t *block_table, int64_t max_blocks, const int32_t *q_start,
                   const int32_t *seq_lens, int64_t batch, int64_t total_q, int64_t max_q_len, const int32_t *path,
                   const int32_t *count, int64_t max_path, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BQ_DECODE_H */
