/*
 * token_attention.h -- C ABI of libconv3d.so for attention on the tokens of a
 * convolutional patch embedding, image and video: rotary positions with several
 * axes, a paged cache of keys and values in 8 (or 16) bits, attention of one new
 * token over that cache, and attention within documents packed in one buffer.
 *
 *   rotary_fwd            (a, b) -> (a cos t - b sin t, b cos t + a sin t),
 *                         t = position[axis] * frequency, for pairs of a head
 *   kv_cache_write        rows of new keys and values to their pages, as codes
 *                         with a scale per token and head, or as they are
 *   kv_cache_read         the reverse, to packed rows
 *   paged_attention_fwd   softmax over a sequence's cached tokens, for its last one
 *   packed_attention_fwd  softmax within each document, for all of its tokens
 *
 * Conventions (status codes, conv_last_error, streams and ownership are those of
 * conv3d.h; element types those of token_ops.h):
 *   - Strides are in elements; the elements of a head's row are contiguous.
 *   - Scores, softmax statistics and sums are held in 32 bits.
 *   - Scores: s = scale * (q . k); with cap > 0 s = cap * tanh(s / cap); with
 *     slopes s -= slopes[head] * |i - j|, i and j being the positions of query
 *     and key in their sequence.  A sequence's queries are its last tokens.
 *   - A query at i sees the keys j < length with
 *     (|i - j| < window, if window > 0, and j <= i, if causal) or j < prefix[sequence].
 *     What it does not see takes no part, whatever it holds.  A query that sees
 *     nothing (or whose scores are all -inf) gets zeros.
 *   - BF16 values may be of any size: their weighted sums are held in fp32 below 2^128
 *     for 2^16 keys (2^20 tokens of a paged cache) whatever the scores are.  Results
 *     below 2^-112 lose bits.
 *   - Query head h reads key head h / (heads / kv_heads).
 *   - Rows of an output or of a cache that overlap are refused; outputs overlap no input
 *     (but rotary_fwd's, which may be x itself).
 */
#ifndef TOKEN_ATTENTION_GB300_H
#define TOKEN_ATTENTION_GB300_H

#include "token_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most pairs of a head that rotary_fwd rotates, and most axes. */
#define ROTARY_MAX_PAIRS 128
#define ROTARY_MAX_AXES 8

/* Rotates pairs of each head's elements by their token's positions.
 *   x, out             dtype BF16, F16 or F32, [tokens, heads, width]; out may be x
 *                      itself with the same strides; other overlap is undefined
 *   positions          int32 (position_bytes 4) or int64 (8), [tokens, axes]
 *   axis, frequency    host arrays [pairs]: which position turns a pair, and by
 *                      how many radians for each unit of it
 *   interleaved        pair p is elements (2p, 2p + 1), else (p, p + pairs); the
 *                      elements from 2 * pairs on are copied
 *   inverse            turns back: also the gradient of x from that of out
 * A frequency's turn for each unit of position is held to 2^-65 of a turn (frequencies up to
 * 2^40), so an angle is exact to 2 pi |position| 2^-65 radians, before its sine and cosine
 * are taken in fp32. */
int rotary_fwd(const void* x, int dtype, int64_t x_token_stride, int64_t x_head_stride,
               const void* positions, int position_bytes, int axes, const int* axis,
               const double* frequency, int pairs, int interleaved, int inverse, int64_t tokens,
               int64_t heads, int64_t width, void* out, int64_t out_token_stride,
               int64_t out_head_stride, cudaStream_t stream);

/* A paged cache: k and v are [pages, heads, page_size, width] of one type and the
 * same strides, k_scale and v_scale fp32 [pages, heads, page_size] for INT8 and
 * FP8_E4M3 (NULL for BF16 and F16).  width is a multiple of 16 up to 256; k, v and
 * their strides are multiples of 16 bytes.  Token t of a sequence is row
 * t % page_size of page page_table[sequence][t / page_size].
 * A page outside [0, pages) is never touched: a token in it is not written, reads
 * as NaN, and spoils (NaN) the attention that sees it. */
typedef struct {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int dtype;
    int64_t pages, heads, page_size, width;
    int64_t page_stride, head_stride, row_stride;
    int64_t scale_page_stride, scale_head_stride;
} kv_cache;

/* Rows of k and v [tokens, cache->heads, width] (BF16, F16 or F32; for a BF16 or
 * F16 cache the cache's type) to the cache.  Rows offsets[s] .. offsets[s+1] are
 * tokens starts[s], starts[s] + 1, ... of sequence s; offsets NULL: row s is the
 * one token of sequence s (tokens == sequences).  Rows in no sequence, and tokens
 * below 0 or past the table, are not written.  Codes and scales are those of
 * act_quant_fwd.  A token that two sequences share is written by both, in no
 * given order.  k, v: one pair of strides for both. */
int kv_cache_write(const kv_cache* cache, const void* k, const void* v, int dtype,
                   int64_t token_stride, int64_t head_stride, int64_t tokens,
                   const int32_t* offsets, const int32_t* starts, const int32_t* page_table,
                   int64_t table_stride, int64_t table_pages, int64_t sequences,
                   cudaStream_t stream);

/* The cache's values as rows of k and v [tokens, cache->heads, width] (BF16, F16
 * or F32): rows offsets[s] .. offsets[s+1] from tokens starts[s] (NULL: 0), ...
 * of sequence s.  Rows in no sequence are left as they are. */
int kv_cache_read(const kv_cache* cache, void* k, void* v, int dtype, int64_t token_stride,
                  int64_t head_stride, int64_t tokens, const int32_t* offsets,
                  const int32_t* starts, const int32_t* page_table, int64_t table_stride,
                  int64_t table_pages, int64_t sequences, cudaStream_t stream);

/* Attention of each sequence's last token over its cached ones.
 *   q, out             BF16 or F16 (a BF16 or F16 cache has the same type),
 *                      [sequences, heads, width]; heads a multiple of the cache's
 *   lengths            int32 [sequences]: tokens in the cache, the new one among
 *                      them; 0 or less: nothing to see.  A length past the table
 *                      gives NaN
 *   prefix, slopes     int32 [sequences] or NULL; fp32 [heads] or NULL
 *   workspace          paged_attention_workspace_size bytes, 16-byte aligned; its
 *                      contents before the call do not matter.  Calls that may
 *                      run at the same time need one each.  Where that size is 0,
 *                      NULL or any pointer with 0 bytes; a workspace of more bytes
 *                      is checked for the size of split heads all the same
 * Scales of values have to be positive; those below 2^-100 count as 0. */
int paged_attention_fwd(const void* q, int q_dtype, int64_t q_sequence_stride,
                        int64_t q_head_stride, const kv_cache* cache, const int32_t* page_table,
                        int64_t table_stride, int64_t table_pages, const int32_t* lengths,
                        const int32_t* prefix, const float* slopes, float scale, float cap,
                        int64_t window, int64_t sequences, int64_t heads, void* out,
                        int64_t out_sequence_stride, int64_t out_head_stride, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream);

/* Bytes of workspace paged_attention_fwd needs on the current device (0: none, and
 * NULL will do; or the arguments are invalid). */
size_t paged_attention_workspace_size(int64_t sequences, int64_t heads, int64_t kv_heads,
                                      int64_t width, int64_t page_size, int64_t table_pages);

/* Attention within documents packed one after the other.
 *   q, out             [q_tokens, heads, width], k, v [k_tokens, kv_heads, width], all
 *                      BF16 or all F16; width a multiple of 8 up to 128; k and v
 *                      share their strides; q, k, v and their strides are multiples
 *                      of 16 bytes
 *   q_offsets, k_offsets  int32 [documents + 1]: document s has query rows
 *                      q_offsets[s] .. q_offsets[s+1] and key rows k_offsets[s] ..;
 *                      rows of out in no document are left as they are
 *   causal, window, prefix (int32 [documents]), slopes (fp32 [heads]): as above */
int packed_attention_fwd(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                         const void* k, const void* v, int64_t k_token_stride,
                         int64_t k_head_stride, int dtype, const int32_t* q_offsets,
                         const int32_t* k_offsets, int64_t documents, int64_t q_tokens,
                         int64_t k_tokens, int64_t heads, int64_t kv_heads, int64_t width,
                         int causal, int64_t window, const int32_t* prefix, const float* slopes,
                         float scale, float cap, void* out, int64_t out_token_stride,
                         int64_t out_head_stride, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TOKEN_ATTENTION_GB300_H */
