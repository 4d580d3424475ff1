/*
 * kvq_fp8_block.h -- C ABI of libkvq, second part: a paged key/value cache of
 * FP8 E4M3 codes with one fp32 scale per 16 tokens of one kv head, the
 * attention that reads it (one token per sequence, or a chunk of them), and
 * the append with the rotary position embedding applied on the way, into this
 * cache or the FP4 / NVFP4 caches of kvq.h.
 *
 * The conventions of kvq.h hold here too: caller-owned device memory, nothing
 * allocated at call time, everything asynchronous on `stream`, host checks
 * before anything is enqueued, data-dependent problems reported in the
 * caller's device flag word, query head h reading kv head h / (Hq / Hkv).
 * Calls work on the current device, which has to be the one that holds the
 * buffers and the stream.
 *
 * 8-bit paged cache (format KVQ_FORMAT_FP8_E4M3_BLOCK, in kvq_cache: page_size
 * one of 16, 32, 64, 128, 256; head_dim 64 or 128; v_data, k_scale and v_scale
 * NULL; page_table and max_pages_per_seq as for the FP4 caches).
 *   A block is 16 consecutive positions (16 i .. 16 i + 15) of one kv head.
 *   Its keys share one fp32 scale and its values another:
 *     value = fp32(E4M3(code) * scale).
 *   The append sets scales to powers of two; the readers take any finite
 *   scale >= 0.
 *   The pool `data` is uint8 [num_pages][num_kv_heads][page_size/G][bytes],
 *   G = min(page_size, 64) tokens per group, and one group is contiguous:
 *     K codes [G/8][head_dim/16][8][16] at 0: 8 tokens x 16 channels make one
 *              128-byte tile of the tensor core's K-major operand layout.
 *     V codes [G/16][head_dim][16] at G*head_dim: the 16 tokens of a block
 *              side by side per channel, in the order 0 1 8 9 2 3 10 11 4 5 12
 *              13 6 7 14 15, which is the order a thread of an m16n8k16
 *              product holds them in.
 *     scales   float [G/16][2] (K, V) at 2*G*head_dim, padded to 16 bytes.
 *   bytes = 2*G*head_dim + max(16, G/2).
 */
#ifndef KVQ_FP8_BLOCK_H
#define KVQ_FP8_BLOCK_H

#include "kvq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of an output. */
enum {
  KVQ_DTYPE_F32 = 0,
  KVQ_DTYPE_BF16 = 1
};

/* Bytes of an 8-bit page pool (0 for invalid sizes). */
size_t kvq_fp8_block_pool_bytes(int64_t num_pages, int32_t num_kv_heads, int32_t page_size, int32_t head_dim);

/*
 * kvq_rope_table -- the cosines and sines of a rotary position embedding,
 * angle(p, i) = p * base^(-2 i / rotary_dim), taken in fp64 and rounded to
 * fp32.  Any other table of this shape (scaled positions, other frequencies)
 * serves kvq_rope_append as well.
 *   table  device float [num_positions][rotary_dim]: of each position first
 *          the rotary_dim/2 cosines, then the sines.
 * rotary_dim even, 2..512; base > 0.  Host errors: INVALID_ARGUMENT.
 */
kvq_status kvq_rope_table(int64_t num_positions, int32_t rotary_dim, double base, float *table, kvq_stream stream);

/*
 * kvq_rope_append -- rotate the new tokens' queries and keys by their
 * positions and append keys and values to a paged cache, in one launch.
 * Token t of sequence b sits at position p = d_start_pos[b] + t.  For each
 * pair (x0, x1) of the first rotary_dim channels of a head,
 *     y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin   (table row p),
 * every product and sum rounded to fp32 and the result to bf16; the other
 * channels pass unchanged.  The rotated keys are quantised from their bf16
 * values, so the cache holds what kvq_append (kvq_fp8_block_append for an
 * 8-bit cache) writes for bf16 keys rotated beforehand, bit for bit.
 *   cache        FP4, NVFP4 or 8-bit block cache (an FP8 window ring is
 *                refused with UNSUPPORTED: append k_out to it).
 *   batch, n_new sequences and new tokens per sequence, >= 0.
 *   d_start_pos  device int32 [batch].
 *   d_new_lens   device int32 [batch] or NULL: sequence b has n_b =
 *                d_new_lens[b] <= n_new new tokens (a padded batch); NULL: all
 *                n_new.  The padding is not read; its rows of q_out and k_out
 *                and the cache behind the last new token stay as they were.
 *   q            device bf16, num_q_heads * head_dim contiguous values per
 *                token, or NULL with num_q_heads == 0 (nothing to rotate).
 *   k, v         device bf16, num_kv_heads * head_dim contiguous values per
 *                token.
 *   q_stride, k_stride, v_stride  elements from one token to the next, tokens
 *                in the order [batch][n_new]: multiples of 8, at least a
 *                token's values; this takes the parts of one packed projection
 *                as they are.
 *   table, table_rows, rotary_dim  device float [table_rows][rotary_dim]
 *                (16-byte aligned), rotary_dim a multiple of 16 up to head_dim;
 *                rotary_dim 0: no rotation, the table is ignored.
 *   interleaved  0: pairs (i, i + rotary_dim/2); 1: pairs (2i, 2i + 1).
 *   q_out        device bf16 [batch][n_new][num_q_heads][head_dim],
 *                contiguous; may be q itself when q_stride is
 *                num_q_heads * head_dim; otherwise disjoint from the inputs.
 *   k_out        device bf16 [batch][n_new][num_kv_heads][head_dim] or NULL:
 *                the rotated keys; as q_out.
 * No page may be written through two entries of the page table in one call.
 * Device flags:
 * NONFINITE, PAGE_OOB (the page's tokens are skipped), BAD_LENGTH (a negative
 * start, n_b outside 0..n_new: the sequence is skipped), POSITION (a position
 * past the table: the sequence's tokens from there on are left out).  Host
 * errors: INVALID_ARGUMENT, UNSUPPORTED (the ring; batch * n_new *
 * num_kv_heads * head_dim / 32, or the same of the query heads / 8, near 2^30 in
 * one call: split the batch).
 */
kvq_status kvq_rope_append(const kvq_cache *cache, int32_t batch, int32_t n_new, const int32_t *d_start_pos,
                           const int32_t *d_new_lens, int32_t num_q_heads, const void *q, int64_t q_stride,
                           const void *k, int64_t k_stride, const void *v, int64_t v_stride, const float *table,
                           int64_t table_rows, int32_t rotary_dim, int32_t interleaved, void *q_out, void *k_out,
                           int32_t *d_err_flag, kvq_stream stream);

/*
 * kvq_fp8_block_append -- quantise the new tokens into an 8-bit block cache.
 * For each block and side (K, V), with amax over its new tokens' values:
 *   s_new = the smallest power of two with amax <= 448 s_new, at least 2^-126;
 *   s     = max(s_old, s_new) when positions of the block before the first
 *           new token are kept, s_new when the block starts with this call
 *           (so a page that is used again carries nothing over);
 *   code  = RNE_e4m3(x / s) for new tokens; kept codes become
 *           RNE_e4m3(E4M3(code) * (s_old / s)) when s > s_old -- exact but for
 *           results under 2^-6, as s_old / s is a power of two.
 * Codes of the block behind the last new token stay as they were (they are
 * read only once a later append has written them).
 *   Arguments and flags as kvq_rope_append's (contiguous k, v: strides
 *   num_kv_heads * head_dim).  A block with Inf or NaN input sets NONFINITE;
 *   its scale is then 2^120 and its codes are what the conversion gives.
 */
kvq_status kvq_fp8_block_append(const kvq_cache *cache, int32_t batch, int32_t n_new, const int32_t *d_start_pos,
                                const int32_t *d_new_lens, const void *k, const void *v, int32_t *d_err_flag,
                                kvq_stream stream);

/*
 * kvq_fp8_block_dequant -- dense values of an 8-bit block cache: k_out, v_out
 * [batch][max_len][num_kv_heads][head_dim] in out_dtype (KVQ_DTYPE_*, rounded
 * once), positions >= d_seq_lens[b] written as 0.  Device flags: PAGE_OOB (the
 * page's positions are written as 0), BAD_LENGTH.
 */
kvq_status kvq_fp8_block_dequant(const kvq_cache *cache, int32_t batch, const int32_t *d_seq_lens, int32_t max_len,
                                 int32_t out_dtype, void *k_out, void *v_out, int32_t *d_err_flag,
                                 kvq_stream stream);

/*
 * kvq_fp8_block_decode_attn -- kvq_decode_attn over an 8-bit block cache:
 *   out[b][h][:] = sum_t softmax_t(softmax_scale * q[b][h] . K^[b][t]) V^[b][t],
 * t = 0 .. d_seq_lens[b] - 1 (a length of 0 gives a zero row).  q enters the
 * products exactly down to 2^-31 of its row's largest element, and off by at
 * most 2^-39 of that below (2^-125 in rows whose largest is under 2^-86); the
 * weights as f16, off by at most 2^-11 of a weight or 2^-25 of the row's
 * largest; sums and softmax statistics are fp32.
 *   num_q_heads  a multiple of num_kv_heads, at most 8 per kv head.
 *   q            device bf16 [batch][num_q_heads][head_dim], 16-byte aligned.
 *   out          device [batch][num_q_heads][head_dim] of out_dtype.
 *   workspace    as kvq_decode_attn's: kvq_decode_workspace_bytes(...) bytes,
 *                not shared by calls that may overlap.
 * Device flags: PAGE_OOB (the page's tokens are left out), BAD_LENGTH,
 * TIMEOUT.
 */
kvq_status kvq_fp8_block_decode_attn(const kvq_cache *cache, int32_t batch, int32_t num_q_heads,
                                     const int32_t *d_seq_lens, const void *q, float softmax_scale, void *out,
                                     int32_t out_dtype, void *workspace, size_t workspace_bytes, int32_t *d_err_flag,
                                     kvq_stream stream);

/*
 * kvq_fp8_block_prefill_attn -- attention of a chunk of new query tokens over
 * an 8-bit block cache that already holds their keys and values: query token i
 * (0 <= i < n_b) of sequence b sits at position T_b - n_b + i and attends
 * positions 0 .. T_b - n_b + i.
 *   d_seq_lens   device int32 [batch]: T_b, the chunk's tokens included.
 *   d_chunk_lens device int32 [batch] or NULL: n_b <= chunk (a padded batch);
 *                NULL: chunk.  Rows i >= n_b of out stay as they were.
 *   num_q_heads  a multiple of num_kv_heads, at most 8 per kv head.
 *   q, out       device [batch][chunk][num_q_heads][head_dim], q bf16, out of
 *                out_dtype; 16-byte aligned.
 * q enters the products exactly down to 2^-9 of its row's largest element, and
 * off by at most 2^-17 of that below (2^-110 in rows whose largest is under
 * 2^-93).  A weight enters the second product times its block's value scale, as
 * f16: off by at most 2^-11 of that, or 2^-24 of the largest such product that
 * the row attends (a block flagged NONFINITE has a scale of 2^120, beside which
 * no other is seen).  A block that a row attends in part can owe its scale to a
 * token behind the row: where the value scales read differ by more than 2^10,
 * the tokens of such a tile of 128 positions have each its own largest value
 * over 2^5 in the place of its block's scale.  Value codes enter exactly; a
 * value scale that is no power of two (the append makes none) is off by at most
 * 2^-11, and so is its product with a code.  No value behind a row's last
 * position, NaN neither, reaches the row, but for what the append made of the
 * block that they share.
 *   workspace    kvq_fp8_block_prefill_workspace_bytes(...) bytes, 16-byte
 *                aligned, not shared by calls that may overlap.
 * Device flags: BAD_LENGTH (n_b outside 0..chunk: the sequence is skipped;
 * T_b < n_b: its n_b rows are written as 0), PAGE_OOB (the page's tokens are
 * left out), TIMEOUT.
 */
size_t kvq_fp8_block_prefill_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                             int32_t head_dim, int32_t chunk);
kvq_status kvq_fp8_block_prefill_attn(const kvq_cache *cache, int32_t batch, int32_t num_q_heads, int32_t chunk,
                                      const int32_t *d_seq_lens, const int32_t *d_chunk_lens, const void *q,
                                      float softmax_scale, void *out, int32_t out_dtype, void *workspace,
                                      size_t workspace_bytes, int32_t *d_err_flag, kvq_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_FP8_BLOCK_H */
