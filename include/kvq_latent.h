/*
 * kvq_latent.h -- C ABI of libkvq, third part: latent attention.  All heads
 * share one latent vector per token, which is key and value at once, and
 * beside it one key part that carries the position rotation.  A paged 8-bit
 * cache of both, the append that rotates and quantises, the attention that
 * reads the cache in its absorbed form (queries and results in the latent
 * space; one token per sequence or a chunk of them), the dense read-back, and
 * the attention over keys and values multiplied out per head (the expanded
 * form, cheaper for long prompts).
 *
 * The conventions of kvq.h hold here too: caller-owned device memory, nothing
 * allocated at call time, everything asynchronous on `stream`, host checks
 * before anything is enqueued, data-dependent problems reported in the
 * caller's device flag word.  Calls work on the current device, which has to
 * be the one that holds the buffers and the stream.
 *
 * Cache layout.  G = min(page_size, 64) tokens form a group, row = latent_dim +
 * 2 rope_dim bytes; the pool `data` is uint8 [num_pages][page_size/G][G * row + G]:
 *   codes      [G/8][row/16][8][16] at 0: 8 tokens x 16 channels make one
 *              128-byte tile of the tensor core's operand layout, for the
 *              scores and for the sums over tokens alike.
 *   exponents  uint8 [G] at G * row: e of each token, its scale s = 2^(e - 127).
 * A token's row holds E4M3(c / s) of the latent c, then hi = E4M3(k / s) and
 * lo = E4M3(k / s - hi) of the rotated key part k:
 *     latent = E4M3(code) * s,   key part = (E4M3(hi) + E4M3(lo)) * s,
 * the key part exact down to 2^-9 of the token's largest magnitude and off by
 * at most 2^-17 of that below (a bf16 value has 8 significant bits, an E4M3
 * value 4, its steps end at 2^-9).  The append sets s to the smallest power of two with
 * max(|c|, |k|) <= 448 s, at least 2^-126.  e = 255 marks a token that held an
 * Inf or NaN (its codes are 0): it reads back as NaN.  Codes are never NaN.
 * (A latent over 248 2^120, bf16's last 3%, rounds to 2^128, which is Inf in fp32.)
 */
#ifndef KVQ_LATENT_H
#define KVQ_LATENT_H

#include "kvq_fp8_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Description of one latent cache (one layer).  Device memory owned by the
 * caller; a page of a sequence is found as in kvq_cache. */
typedef struct kvq_latent_cache {
  int32_t latent_dim;        /* 128, 256 or 512 */
  int32_t rope_dim;          /* 32 or 64 */
  int32_t page_size;         /* tokens per page, one of 16, 32, 64, 128, 256 */
  int32_t max_pages_per_seq; /* row length of page_table (or pages per sequence when contiguous) */
  int64_t num_pages;         /* pages in the pool */
  const int32_t *page_table; /* device int32 [batch][max_pages_per_seq] or NULL (contiguous) */
  void *data;                /* the page pool, 16-byte aligned */
} kvq_latent_cache;

/* Bytes of a latent page pool (0 for invalid sizes). */
size_t kvq_latent_pool_bytes(int64_t num_pages, int32_t page_size, int32_t latent_dim, int32_t rope_dim);

/*
 * kvq_latent_append -- rotate the new tokens' key parts and query parts by
 * their positions and write latents and key parts to the cache, in one launch.
 * Token t of sequence b sits at position d_start_pos[b] + t.  The rotation is
 * kvq_rope_append's over all rope_dim channels: every product and sum rounded
 * to fp32, the result to bf16; the key part is quantised from its bf16 values.
 *   batch, n_new  sequences and new tokens per sequence, >= 0.
 *   d_start_pos   device int32 [batch].
 *   d_new_lens    device int32 [batch] or NULL: sequence b has n_b =
 *                 d_new_lens[b] <= n_new new tokens; NULL: all n_new.  The
 *                 padding is not read; its rows of q_out and k_out, and the
 *                 cache behind the last new token, stay as they were.
 *   q             device bf16: rope_dim contiguous values per head and token,
 *                 q_head_stride elements from one head to the next and
 *                 q_token_stride from one token to the next ([batch][n_new]);
 *                 NULL with num_q_heads == 0.
 *   c, k          device bf16: latent_dim (rope_dim) contiguous values per
 *                 token, c_stride (k_stride) elements from token to token.
 *                 All strides are multiples of 8 and leave no overlap, so the
 *                 parts of packed projections go in as they are.
 *   table, table_rows  device float [table_rows][rope_dim], 16-byte aligned
 *                 (kvq_rope_table's layout); NULL and 0: no rotation.
 *   interleaved   0: pairs (i, i + rope_dim/2); 1: pairs (2i, 2i + 1).
 *   q_out         device bf16, laid out by q_out_token_stride and
 *                 q_out_head_stride (for instance the tail of each head's
 *                 absorbed query); may be q itself with the same strides,
 *                 otherwise disjoint from the inputs.
 *   k_out         device bf16 [batch][n_new][rope_dim], contiguous, or NULL:
 *                 the rotated key parts; disjoint from the inputs.
 * No page may be written through two entries of the page table in one call.
 * Device flags: NONFINITE, PAGE_OOB (the page's tokens are skipped), BAD_LENGTH
 * (a negative start, n_b outside 0..n_new: the sequence is skipped), POSITION (a
 * position past the table: the sequence's tokens from there on are left out).
 * Host errors: INVALID_ARGUMENT, UNSUPPORTED (more than 2^30 threads' work in
 * one call: split the batch).
 */
kvq_status kvq_latent_append(const kvq_latent_cache *cache, int32_t batch, int32_t n_new, const int32_t *d_start_pos,
                             const int32_t *d_new_lens, int32_t num_q_heads, const void *q, int64_t q_token_stride,
                             int64_t q_head_stride, const void *c, int64_t c_stride, const void *k, int64_t k_stride,
                             const float *table, int64_t table_rows, int32_t interleaved, void *q_out,
                             int64_t q_out_token_stride, int64_t q_out_head_stride, void *k_out, int32_t *d_err_flag,
                             kvq_stream stream);

/*
 * kvq_latent_dequant -- dense rows of a latent cache: c_out
 * [batch][max_len][latent_dim] and k_out [batch][max_len][rope_dim] in
 * out_dtype (KVQ_DTYPE_*, rounded once), positions >= d_seq_lens[b] written
 * as 0.  16-byte aligned.  Device flags: PAGE_OOB (the page's positions are
 * written as 0), BAD_LENGTH (a negative length: as 0).
 */
kvq_status kvq_latent_dequant(const kvq_latent_cache *cache, int32_t batch, const int32_t *d_seq_lens, int32_t max_len,
                              int32_t out_dtype, void *c_out, void *k_out, int32_t *d_err_flag, kvq_stream stream);

/*
 * kvq_latent_attn -- attention over a latent cache, absorbed form: query token
 * i (0 <= i < n_b) of sequence b sits at position T_b - n_b + i and attends
 * positions 0 .. T_b - n_b + i,
 *   out[b][i][h][:] = sum_t softmax_t(softmax_scale * q[b][i][h] . [c_t, k_t]) c_t.
 * With chunk == 1 and d_chunk_lens == NULL it is a decode step: T_b == 0 gives
 * a zero row.
 *   num_q_heads  >= 1; all heads read the same cache.
 *   d_seq_lens   device int32 [batch]: T_b, the chunk's tokens included.
 *   d_chunk_lens device int32 [batch] or NULL: n_b <= chunk (a padded batch);
 *                NULL: chunk.  Rows i >= n_b of out stay as they were.
 *   q            device bf16 [batch][chunk][num_q_heads][latent_dim + rope_dim].
 *   out          device [batch][chunk][num_q_heads][latent_dim] of out_dtype.
 *                Both 16-byte aligned.
 *   workspace    kvq_latent_attn_workspace_bytes(...) bytes, 16-byte aligned,
 *                not shared by calls that may overlap.
 * q enters the products exactly down to 2^-9 of its row's largest element, and
 * off by at most 2^-17 of that below (2^-136 in rows whose largest is under
 * 2^-119).  A weight enters the second product times its token's scale, off by at
 * most 2^-8 + 2^-11 of that, or 2^-17 of the largest such product that the row attends.
 * Sums, softmax statistics and their joins are fp32.  So are scores, times
 * softmax_scale log2 e: they have to lie in its range (softmax_scale times the row's
 * and a token's largest magnitude under 2^115 is enough).
 * A row that attends a token marked as non-finite, or whose query holds an Inf
 * or NaN, is NaN; no other row is touched by either.
 * Device flags: BAD_LENGTH (n_b outside 0..chunk: the sequence is skipped;
 * T_b < n_b, or T_b < 0: its n_b rows are written as 0), PAGE_OOB (the page's
 * tokens are left out), TIMEOUT (kvq_test_set_wait_limit_ns reaches this call's
 * waits and kvq_expanded_attn's, too).
 * Host errors: INVALID_ARGUMENT, WORKSPACE, UNSUPPORTED (2^30 rows and more).
 */
size_t kvq_latent_attn_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t latent_dim, int32_t chunk);
kvq_status kvq_latent_attn(const kvq_latent_cache *cache, int32_t batch, int32_t num_q_heads, int32_t chunk,
                           const int32_t *d_seq_lens, const int32_t *d_chunk_lens, const void *q, float softmax_scale,
                           void *out, int32_t out_dtype, void *workspace, size_t workspace_bytes, int32_t *d_err_flag,
                           kvq_stream stream);

/*
 * kvq_expanded_attn -- causal attention of a chunk of query tokens over dense
 * keys and values, the keys' position part shared by all heads:
 *   out[b][i][h] = sum_t softmax_t(softmax_scale * (q[b][i][h][:d] . k[b][t][h]
 *                  + q[b][i][h][d:] . k_rope[b][t])) v[b][t][h],
 * t = 0 .. T_b - n_b + i, with T_b and n_b as in kvq_latent_attn.
 *   head_dim (d)  64 or 128; rope_dim 64.
 *   q            device bf16 [batch][chunk][num_heads][d + rope_dim], contiguous.
 *   k, v         device bf16: d contiguous values per head and token, strides
 *                in elements from head to head (at least d) and from token to
 *                token (at least a token's heads: head-major keys are refused),
 *                tokens in the order [batch][max_len].
 *   k_rope       device bf16: rope_dim contiguous values per token,
 *                k_rope_stride elements from token to token.
 *                Strides are multiples of 8, all pointers 16-byte aligned.
 *   max_len      tokens per sequence in k, k_rope and v; positions from T_b on
 *                are not used.
 *   out          device [batch][chunk][num_heads][d] of out_dtype, 16-byte aligned.
 * q, k and v enter the products as they are; a weight is rounded to bf16, sums and
 * softmax statistics are fp32; scores have to lie in its range, with softmax_scale log2 e
 * and without.  Finite values up to bf16's largest do not overflow a sum where the
 * scores, times softmax_scale log2 e, are under 2^27 (over larger ones, 2^119 / T_b and
 * less does not).  Products of a weight and a value that are under fp32's normal range
 * are lost, which is less than T_b^2 2^-117 in a result (T_b^2 2^-109 over scores past
 * 2^14).  A row that attends a value that is Inf or NaN is not finite in its channel; no
 * Inf or NaN among the keys and values behind a row's position reaches the row.  A row
 * whose scores are all -Inf is NaN.
 * Host errors: INVALID_ARGUMENT, UNSUPPORTED (2^30 rows and more, max_len above
 * 2^30).
 * Device flags: BAD_LENGTH (n_b outside 0..chunk, T_b > max_len: the sequence is
 * skipped; T_b < n_b, or T_b < 0: its n_b rows are written as 0), TIMEOUT.
 */
kvq_status kvq_expanded_attn(int32_t batch, int32_t num_heads, int32_t head_dim, int32_t rope_dim, int32_t chunk,
                             int32_t max_len, const int32_t *d_seq_lens, const int32_t *d_chunk_lens, const void *q,
                             const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *k_rope,
                             int64_t k_rope_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                             float softmax_scale, void *out, int32_t out_dtype, int32_t *d_err_flag,
                             kvq_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_LATENT_H */
