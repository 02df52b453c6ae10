/*
 * bq_layer.h - C ABI of the decoder-layer operators of libbq.so: what a
 * low-bit attention layer needs around the products of bq.h.
 *
 *   - 4-bit weights with a scale (and zero point) per group of K, times
 *     16-bit activations (bq_gemm_w4g_a16);
 *   - the norms of queries and keys per head with the position rotation in
 *     the same pass (bq_qk_norm_rope), and the same with keys and values
 *     quantized into a 4-bit paged cache (bq_qk_norm_rope_kv4);
 *   - that cache read back (bq_kv4_read) and attended to (bq_attn_kv4).
 *
 * The conventions of bq.h hold (device pointers owned by the caller, streams,
 * errors, no device memory allocated, reentrancy), with these additions:
 *  - 16-bit tensors are fp16 or bf16, chosen by `dtype` (enum bq_dtype).
 *  - Tensors with a `_stride` argument are dense within a token and may have
 *    any distance between tokens (the rows of a fused projection).
 *  - int32 / int64 index arrays are device memory that the host does not
 *    read: an index outside its range (a page, a slot, a position, a length)
 *    is never followed; each call says what becomes of its token.
 *
 * The cache is num_pages pages of bq_kv4_page_bytes bytes.  A page holds
 * page_size tokens of every kv head; per kv head (page_size * (D + 8) bytes):
 *   K codes  [page_size][D/2]           channel d even in the low nibble of
 *                                       byte d/2, codes 0..15
 *   V codes  [page_size/4][units][4][U] U = 2 bytes (D = 64) or 4; unit u of
 *                                       a token holds channels 2Uu ..
 *                                       2Uu + 2U - 1, packed as for K
 *   K params [page_size][2] fp16        scale, min
 *   V params [page_size][2] fp16
 * and the value of a code is code * scale + min (bq_qk_norm_rope_kv4 stores
 * scales of at least 0; a cache laid out by other means may hold negative
 * ones).  Token t of a sequence lies
 * in page block_table[t / page_size] at t % page_size; a slot is
 * page * page_size + offset.
 */
#ifndef BQ_LAYER_H
#define BQ_LAYER_H

#include "bq.h"

#ifdef __cplusplus
extern "C" {
#endif

enum bq_dtype {
    BQ_F16 = 0,
    BQ_BF16 = 1
};

/*
 * bq_gemm_w4g_a16 - C = T(sum_k A[m,k] * (c[n,k] - zero[n,g]) * scale[n,g]),
 * g = k / group: 4-bit weights with group scales, fp32 accumulation.
 *
 *   A          [M, K] 16-bit (dtype), finite; bf16 values of magnitude below
 *              2^100 (the kernels sum a * (c + 136) in fp32)
 *   B          [N, K/2] uint8, the layout of bq_pack_int4: codes c in -8..7
 *              (bq_quantize_pack over the rows of the weight viewed as
 *              [N * K/group, group] gives B and scale)
 *   scale_f16  [N, K/group] fp16
 *   zero_f16   [N, K/group] fp16, in units of codes, or NULL (0)
 *   group      32, 64 or 128 (BQ_ERR_ARG otherwise)
 *   C          [M, N] of dtype
 *   workspace  device memory for sums over parts of K, 16-byte aligned, no
 *              particular contents; NULL with 0 bytes, or fewer than
 *              bq_gemm_w4g_workspace_bytes, for none (K is not split, the sums
 *              are taken in another order).  Calls that share one must not
 *              overlap.
 * M > 16 rounds each weight once to dtype (in fp16, one past 65504 becomes
 * infinite); smaller M uses the exact weights.  A row's low bits therefore
 * depend on M, and on whether K is split.
 * 0 <= M, N <= BQ_MAX_DIM, M * N <= BQ_MAX_OUT, 0 <= K <= BQ_MAX_K, K a
 * multiple of 64 and of group (BQ_ERR_SHAPE); pointers 16-byte aligned.
 * K == 0 writes zeros.
 */
int bq_gemm_w4g_a16(const void *A, int dtype, const uint8_t *B, const void *scale_f16, const void *zero_f16, int group,
                    void *C, int64_t M, int64_t N, int64_t K, void *workspace, int64_t workspace_bytes, void *stream);

/* Device workspace bytes with which bq_gemm_w4g_a16 splits K for this shape
 * (0: it does not); negative: -BQ_ERR_SHAPE.  Host-only. */
int64_t bq_gemm_w4g_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * bq_qk_norm_rope - per head of queries and keys:
 *   y = x * w / sqrt(mean(x^2) + eps)     (w NULL: y = x)
 * then the rotation of the first rot_dim channels by the token's position,
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * for the pairs (i, i + rot_dim/2), or (2i, 2i + 1) if interleaved; fp32,
 * rounded once to dtype.
 *
 *   q, k          tokens x q_heads x head_dim and tokens x kv_heads x
 *                 head_dim, q_stride / k_stride elements between tokens
 *                 (at least a token's size, multiples of 8); finite values.
 *                 With weights, bf16 values lie below 2^60 in magnitude, and
 *                 mean(x^2) + eps above 2^-100: squares and the product with
 *                 the weight are fp32
 *   q_weight, k_weight  [head_dim] of dtype; both or neither (BQ_ERR_NULL)
 *   cos, sin      [max_pos, rot_dim/2] fp32
 *   positions     [tokens] int32; a token whose position is outside
 *                 [0, max_pos) is left out: its outputs stay as they were
 *   rot_dim       a multiple of 16 from 0 to head_dim; 0 (no rotation) needs
 *                 neither cos, sin nor positions
 *   q_out, k_out  [tokens, heads, head_dim] dense, not overlapping q or k
 * head_dim 64, 128 or 256; q_heads or kv_heads may be 0 (the tensors of that
 * kind are then not used).
 */
int bq_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, int dtype, int64_t tokens, int q_heads,
                    int kv_heads, int head_dim, const void *q_weight, const void *k_weight, double eps, const float *cos,
                    const float *sin, int64_t max_pos, int rot_dim, int interleaved, const int32_t *positions, void *q_out,
                    void *k_out, void *stream);

/* Bytes of a page of the 4-bit cache: kv_heads * page_size * (head_dim + 8);
 * negative: -BQ_ERR_SHAPE (head_dim 64, 128 or 256; page_size 16, 32, 64,
 * 128 or 256; 1 <= kv_heads <= 65536).  Host-only. */
int64_t bq_kv4_page_bytes(int kv_heads, int head_dim, int page_size);

/*
 * bq_qk_norm_rope_kv4 - bq_qk_norm_rope with the keys, rounded to dtype, and
 * the values written to the cache in 4 bits instead of to k_out.  Per token
 * and head, in fp32 with correctly rounded quotients:
 *   min = fp16(min x), scale = fp16((max x - min) / 15)
 *   code = nearest((x - min) / scale), ties to even, in 0..15; 0 if scale = 0
 * min is held within [-65504, 65504] and scale within [0, 65504], so that
 * finite bf16 values outside fp16's range give finite ones: a row below the
 * range reads back as -65504, values more than 15 * 65504 above min as that.
 *
 *   v       tokens x kv_heads x head_dim, v_stride between tokens
 *   cache   num_pages pages, 16-byte aligned
 *   slots   [tokens] int64, different from each other; a token whose slot is
 *           outside [0, num_pages * page_size) is not written (its query is)
 * q_heads may be 0: keys and values only.  With no weights and rot_dim 0 this
 * is a plain write to the cache.  A token left out for its position writes
 * nothing.  NaN and infinities give unspecified codes for their token and
 * head, and nothing else.
 */
int bq_qk_norm_rope_kv4(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                        int dtype, int64_t tokens, int q_heads, int kv_heads, int head_dim, const void *q_weight,
                        const void *k_weight, double eps, const float *cos, const float *sin, int64_t max_pos, int rot_dim,
                        int interleaved, const int32_t *positions, void *q_out, void *cache, int64_t num_pages,
                        int page_size, const int64_t *slots, void *stream);

/*
 * bq_kv4_read - the keys and values of the given slots, dense:
 * k_out, v_out [tokens, kv_heads, head_dim] of dtype, dtype(code * scale +
 * min).  A slot outside the cache leaves its rows as they were; a slot may
 * occur more than once.
 */
int bq_kv4_read(const void *cache, int64_t num_pages, int page_size, int kv_heads, int head_dim, const int64_t *slots,
                int64_t tokens, int dtype, void *k_out, void *v_out, void *stream);

/*
 * bq_attn_kv4 - attention of queries over the cache, one softmax per query
 * row and head:
 *   out = sum_t softmax_t(softmax_scale * q . K[t]) V[t]
 * over the keys t <= p (and t > p - window if window > 0), where a sequence's
 * queries stand at the end of its cache: query i of q_len has position
 * p = seq_len - q_len + i.  q_heads / kv_heads query heads share a kv head.
 * A row with no keys gives zeros (lse -infinity).
 *
 *   q            total_q x q_heads x head_dim, q_stride between tokens; bf16
 *                values of magnitude below 2^100
 *   q_start      [batch + 1] int32, the first query of each sequence, then
 *                the end; each is taken within [0, total_q], and a sequence
 *                whose end is not past its start has none; NULL: max_q_len
 *                queries each (total_q = batch * max_q_len)
 *   max_q_len    the most queries of one sequence that are computed, its first
 *                ones; further ones of a sequence are left out: their outputs
 *                stay as they were, like rows behind the last sequence, and
 *                the positions of the others do not depend on it (q_len counts
 *                all of a sequence's queries)
 *   seq_lens     [batch] int32, keys in the cache with the new ones; taken
 *                within [0, max_blocks * page_size]
 *   block_table  [batch, max_blocks] int32; tokens of a page outside
 *                [0, num_pages) are not attended to
 *   out          [total_q, q_heads, head_dim] of dtype
 *   lse          NULL or [total_q, q_heads] fp32: log sum exp of the scaled
 *                scores
 *   workspace    device memory for parts of long sequences, 16-byte aligned,
 *                no particular contents; NULL with 0 bytes, or fewer than
 *                bq_attn_kv4_workspace_bytes, for none (sequences are not
 *                split).  Calls that share one must not overlap.
 * The cache's values are used exactly, the products and sums are fp32; p times
 * a key's V scale is held in 22 bits for fp16 outputs and 11 for bf16, and to
 * 2^-29 of the row's largest p times the largest V scale that the row sees.
 * Keys that a row does not see change no bit of its result, whatever their
 * codes and parameters are.  Where sequences are split, the length of the
 * parts follows from the call's sizes and its longest sequence, and with it the
 * order of the sums: a sequence's low bits can differ between batches.
 * q_heads a multiple of kv_heads, max_blocks * page_size <= 2^30, total_q <=
 * 2^30 (BQ_ERR_SHAPE); softmax_scale finite, of any sign (BQ_ERR_ARG).
 */
int bq_attn_kv4(const void *q, int64_t q_stride, int dtype, const int32_t *q_start, const int32_t *seq_lens,
                const int32_t *block_table, int64_t batch, int64_t total_q, int64_t max_q_len, int q_heads, int kv_heads,
                int head_dim, const void *cache, int64_t num_pages, int page_size, int64_t max_blocks, float softmax_scale,
                int64_t window, void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream);

/* Device workspace bytes with which bq_attn_kv4 splits sequences of up to
 * max_len keys (max_blocks * page_size); 0: it does not split; negative:
 * -BQ_ERR_SHAPE.  Host-only. */
int64_t bq_attn_kv4_workspace_bytes(int64_t batch, int64_t max_q_len, int q_heads, int kv_heads, int head_dim,
                                    int64_t max_len);

#ifdef __cplusplus
}
#endif

#endif /* BQ_LAYER_H */
