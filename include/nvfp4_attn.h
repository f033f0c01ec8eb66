/*
 * nvfp4_attn.h - C ABI of the attention operators on a paged key/value cache
 * held in NVFP4, for MI355X (gfx950): norms of queries and keys per head with
 * the position rotation in the same pass, writing keys and values into the
 * cache and reading them back, and attention over it with a sliding window and
 * a few first tokens that stay visible.
 *
 * The cache.  Token slots are numbered page * page_size + offset.  With
 * dp = head_dim rounded up to a multiple of 64:
 *
 *   k_codes, v_codes    uint8 [pages][kv_heads][page_size][dp/2]   two E2M1 codes a
 *                       byte, element 2i in bits 3:0, as in nvfp4_gemv.h
 *   k_scales, v_scales  uint8 [pages][kv_heads][dp/16][page_size]  E4M3 codes, one
 *                       per 16 elements of a token
 *   k_global, v_global  float [kv_heads] or NULL (1)
 *
 * An element stands for e2m1 * e4m3 * global[head].  Elements from head_dim on
 * are zero codes with zero scales: nvfp4_kv_write_launch and
 * nvfp4_qk_norm_rope_launch write them, a cache filled otherwise has to hold
 * them.  Blocks are quantised as nvfp4_quantize.h says, with global[head] as the
 * global scale and one of its rounding rules.
 *
 * Rows.  Q, K, V and the outputs hold tokens x heads rows of head_dim contiguous
 * elements; row (t, h) lies at base + t * token_stride + h * head_stride
 * elements, so that the parts of one QKV projection, or a transposed layout, need
 * no copy.
 *
 * All data pointers are DEVICE pointers owned by the caller (nvfp4_kv_cache_t
 * itself is host memory, read during the call only); the library keeps none of
 * them after the enqueued work.  `stream` is a hipStream_t (NULL = the default
 * stream).  Calls only enqueue work: no device synchronisation, no host read of
 * device memory, no dependence of the launches on device data, so that a captured
 * call serves later lengths, pages and slots.  Every argument is checked before
 * any HIP call; invalid calls return a negative status of nvfp4_gemv.h and enqueue
 * nothing.  What lies on the device (slots, positions, pages, lengths, query
 * starts) is checked by the kernels, as each call says, and never leads out of the
 * buffers.  No C++ exception crosses this interface.
 *
 * Shape rules: head_dim a multiple of 16 from 16 to 256; page_size a power of two
 * from 16 to 1024; pages >= 1, pages * page_size < 2^31; kv_heads from 1 to 1024;
 * heads a multiple of kv_heads, at most 16384; tokens < 2^24 and
 * tokens * (heads + 2 kv_heads) < 2^27 (tokens = 0 does nothing); strides from 0
 * to 2^40 elements, those of outputs such that rows do not overlap.
 * Alignment: rows to their element, codes and scales to 16 bytes, float arrays to
 * 16 (globals to 4), positions and slots to 8, other integers to 4.  Rows that are
 * not 16-byte aligned are read and written element by element.
 */
#ifndef NVFP4_ATTN_H
#define NVFP4_ATTN_H

#include <stddef.h>
#include <stdint.h>

#include "nvfp4_ffn.h"
#include "nvfp4_gemv.h"
#include "nvfp4_quantize.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct nvfp4_kv_cache_t {
    uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    const float *k_global, *v_global;   /* [kv_heads] or NULL (1) */
    int64_t pages, page_size, kv_heads, head_dim;
} nvfp4_kv_cache_t;

/*
 * Writes K and V (x_type NVFP4_OUT_F16 or NVFP4_OUT_BF16, tokens x kv_heads rows)
 * into the slots.  slots int64 [tokens]: a token whose slot is not in
 * [0, pages * page_size) is left out, and nothing else of the cache is touched.
 * A slot may stand there once; twice leaves a mixture of the two tokens there.
 * rule: NVFP4_ROUND_*.
 */
int nvfp4_kv_write_launch(const nvfp4_kv_cache_t *cache, const void *K, int64_t k_token_stride,
                          int64_t k_head_stride, const void *V, int64_t v_token_stride,
                          int64_t v_head_stride, int32_t x_type, const int64_t *slots, int64_t tokens,
                          int32_t rule, void *stream);

/*
 * Reads the slots back: K and V of y_type (NVFP4_OUT_F16, _BF16 or _F32),
 * [tokens][kv_heads][head_dim] contiguous, y( f32( e2m1 * e4m3 * global ) ).  A slot
 * that is not in [0, pages * page_size) gives zeros.
 */
int nvfp4_kv_read_launch(const nvfp4_kv_cache_t *cache, const int64_t *slots, int64_t tokens, void *K,
                         void *V, int32_t y_type, void *stream);

/*
 * Head norms and rotation.  For each row x of Q (heads per token) and of K
 * (kv_heads per token), in fp32:
 *
 *   y = x * w / sqrt( mean(x^2) + eps )           (y = x where the weight is NULL)
 *   pairs (a, b) = (y[i], y[i + rot_dim/2]) or, interleaved, (y[2i], y[2i+1]), for
 *   i < rot_dim/2:  (a cos - b sin, b cos + a sin)   of cos_sin[position][i] and
 *                                                    cos_sin[position][rot_dim/2 + i]
 *
 * and rounded to x_type (fp16 or bf16).  Elements from rot_dim on are not rotated.
 *   q_weight, k_weight  float [head_dim] or NULL
 *   positions           int64 [tokens]; one outside [0, table_rows) gives NaN
 *   cos_sin             float [table_rows][rot_dim], cosines before sines
 *   rot_dim             a multiple of 16 from 0 to head_dim (0: no rotation; then
 *                       positions and cos_sin may be NULL)
 *   Q_out, K_out        of x_type; may be Q, K themselves (same address and strides)
 *
 * With a cache, the rows of K (rounded to x_type) and V go into its slots as
 * nvfp4_kv_write_launch writes them, to the last bit, and K_out has to be NULL;
 * without one, cache, V and slots are NULL.
 */
int nvfp4_qk_norm_rope_launch(const void *Q, int64_t q_token_stride, int64_t q_head_stride,
                              const float *q_weight, void *Q_out, int64_t qo_token_stride,
                              int64_t qo_head_stride, int64_t heads, const void *K,
                              int64_t k_token_stride, int64_t k_head_stride, const float *k_weight,
                              void *K_out, int64_t ko_token_stride, int64_t ko_head_stride,
                              int64_t kv_heads, int64_t head_dim, int32_t x_type,
                              const int64_t *positions, const float *cos_sin, int64_t table_rows,
                              int64_t rot_dim, int32_t interleaved, float eps, int64_t tokens,
                              const nvfp4_kv_cache_t *cache, const void *V, int64_t v_token_stride,
                              int64_t v_head_stride, const int64_t *slots, int32_t rule, void *stream);

/*
 * Attention.  Sequence b has lengths[b] tokens in the cache, token j in page
 * block_table[b][j / page_size] at offset j % page_size, and the queries of tokens
 * query_starts[b] .. query_starts[b+1] of Q; its last query is its last token, so
 * query i of n stands at position p = lengths[b] - n + i.  Query head h reads kv
 * head h / (heads / kv_heads).  Token j is visible to a query at p where j <= p and,
 * with a window, j > p - window or j < sinks, and
 *
 *   out = sum_j softmax_j( scale q . k_j ) v_j      over the visible tokens
 *
 * A query that sees no token, or whose scores are all minus infinity, gives zeros;
 * what stands in the places of other tokens (infinities, NaN) does not matter.
 * Where scale * k_global[head] is not finite in fp32, queries that see a token give NaN.
 *   Q, out        x_type (fp16 or bf16), tokens x heads rows; out is not Q
 *   block_table   int32, row b at block_table + b * table_stride, table_width pages
 *                 each.  A page outside [0, pages) is not read and its tokens are not
 *                 visible (pages that left the window need not be kept)
 *   lengths       int32 [batch], taken to lie in [0, table_width * page_size]
 *   query_starts  int32 [batch + 1], not decreasing, or NULL: tokens / batch queries
 *                 each.  Taken to lie in [0, tokens]; rows of out that belong to no
 *                 sequence are left as they were
 *   max_query     at least the queries of any sequence, 1 .. tokens, and at least
 *                 tokens / batch where query_starts is NULL.  The kernels are chosen by it
 *                 for the whole batch: single tokens that share a call with a prompt take the
 *                 prompt's.  Only that many queries of a sequence are computed
 *   window        0 (all tokens) or the tokens that a query sees, itself included
 *   sinks         first tokens that stay visible outside the window
 *
 * Products of q and k are exact and summed in fp32 (a bf16 row of q is scaled by a
 * power of two to fit fp16, where e2m1 * e4m3 is exact: elements below 2^-31 of the
 * row's largest are rounded to multiples of at most 2^-38 of it); softmax statistics
 * and sums are fp32, and the weights meet v rounded to fp16 after scaling, 2^-11
 * relative.  Results do not depend on other sequences' values; their last bits may
 * depend on the batch's lengths, by which histories are cut into pieces.
 * table_width * page_size < 2^31, batch from 1 to 65535, batch * kv_heads <= 2^18,
 * tokens * heads < 2^30, strides of block_table not negative, scale finite.
 */
size_t nvfp4_kv_attention_workspace_size(const nvfp4_kv_cache_t *cache, int64_t heads, int64_t batch,
                                         int64_t tokens, int64_t max_query, int64_t table_width);

/*
 * With a caller-owned workspace (256-byte aligned, not aliasing any argument, not
 * used by other work that may run concurrently).  Allocates nothing.
 */
int nvfp4_kv_attention_launch_ws(const nvfp4_kv_cache_t *cache, const void *Q, int64_t q_token_stride,
                                 int64_t q_head_stride, void *out, int64_t o_token_stride,
                                 int64_t o_head_stride, int64_t heads, int32_t x_type,
                                 const int32_t *block_table, int64_t table_stride, int64_t table_width,
                                 const int32_t *lengths, const int32_t *query_starts, int64_t batch,
                                 int64_t tokens, int64_t max_query, float scale, int64_t window,
                                 int64_t sinks, void *workspace, size_t workspace_bytes, void *stream);

/* The same with the library-owned workspace, as nvfp4_linear_launch. */
int nvfp4_kv_attention_launch(const nvfp4_kv_cache_t *cache, const void *Q, int64_t q_token_stride,
                              int64_t q_head_stride, void *out, int64_t o_token_stride,
                              int64_t o_head_stride, int64_t heads, int32_t x_type,
                              const int32_t *block_table, int64_t table_stride, int64_t table_width,
                              const int32_t *lengths, const int32_t *query_starts, int64_t batch,
                              int64_t tokens, int64_t max_query, float scale, int64_t window,
                              int64_t sinks, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_ATTN_H */
