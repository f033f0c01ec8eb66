/*
 * nvfp4_ffn.h - C ABI of the feed-forward operators on NVFP4 weights for
 * MI355X (gfx950): the linear layer with bias, activation and residual in its
 * epilogue, and a whole mixture-of-experts (MoE) layer for a few tokens.
 *
 * Both take 16-bit floating-point activations (bf16 or fp16) as they are: a
 * weight element times its block scale, e2m1 * e4m3, has at most 6
 * significant bits and, unless it is 0, lies in 2^-10 .. 2688, so it is exact in
 * either type,
 * the products are exact in fp32 and the sums are fp32 (their order is fixed
 * for a given shape, type, layout and alignment).
 *
 * Linear layer.  For t < n, r < m:
 *
 *   z[t,r] = alpha[0] * sum_kk X[t,kk] w(r,kk) + bias[r]
 *   Y[t,r] = y( residual[t,r] + f(z[t,r]) )
 *
 * and, with NVFP4_ACT_GATED, the weight holds two m x k matrices, gate and up:
 *
 *   u[t,r] = alpha[1] * sum_kk X[t,kk] w(m+r,kk) + bias[m+r]
 *   Y[t,r] = y( residual[t,r] + f(z[t,r]) * u[t,r] )
 *
 * f is the activation; every step up to the rounding y() is in fp32.
 *   X        bf16 or fp16, row t at X + t * ldx elements, k elements each
 *   W        uint8 codes, sfW uint8 block scales: one matrix [m][k/2], [m][k/16]
 *            (gated: two, [2][m][k/2], [2][m][k/16]) with w_layout
 *            NVFP4_W_ROW_MAJOR; with NVFP4_W_PACKED the buffers that
 *            nvfp4_mma_pack_weight writes for groups = 1 (gated: 2)
 *   alpha    float [1] (gated [2]) or NULL (1)
 *   bias     float [m] (gated [2 m]) or NULL (0)
 *   residual y_type, row t at residual + t * ldr elements, or NULL (0).  May be
 *            Y itself (same address and ldr == ldy): the update is in place
 *   Y        y_type, row t at Y + t * ldy elements; only its m elements are written.
 *            No input may share an element with it (but the residual, as above):
 *            rows of X or the residual may lie between Y's where the strides are
 *            the same number of bytes, as column ranges of one matrix do
 *
 * MoE layer.  For token t, with z = X[t] Wr^T over the experts:
 *
 *   s[e]  = softmax(z)[e]  or  1 / (1 + exp(-z[e]))        (scoring)
 *   the topk experts with the largest s[e] + route_bias[e], the lowest index
 *   first among equals (a NaN counts as the least); their weights w[j] = s[e_j],
 *   divided by their sum when renormalize is set, times routed_scale
 *   h_j   = f( alpha13[e_j][0] * gate_{e_j} X[t] ) * ( alpha13[e_j][1] * up_{e_j} X[t] )
 *   Y[t]  = y( residual[t] + sum_j w[j] * alpha2[e_j] * down_{e_j} h_j )
 *
 * Logits and scores are computed in fp64.  Without a route_bias experts are
 * ordered by their logits, so they are chosen as the exact scores say, also where
 * these round to the same number; with one, keys that fp64 does not tell apart
 * (sigmoids of logits from about 37 on are all 1) count as equal.  h is kept with
 * 16 significand bits for a 16-bit Y and with 24 for an fp32 Y; all other sums are
 * fp32.
 *
 * All data pointers are DEVICE pointers owned by the caller (the
 * nvfp4_moe_layer_t itself is host memory, read during the call only); the
 * library keeps none of them after the enqueued work.  `stream` is a
 * hipStream_t (NULL = the default stream).  Calls only enqueue work: no
 * device synchronisation, no host read of device memory, no dependence of the
 * launches on device data.  Every argument is checked before any HIP call;
 * invalid calls return a negative status of nvfp4_gemv.h and enqueue nothing.
 * No C++ exception crosses this interface.
 *
 * Shape rules: k (hidden, inter) a multiple of 16, at least 16 and at most
 * 2^22, and a multiple of 64 with NVFP4_W_PACKED; ldx >= k, at most 2^22;
 * ldy, ldr >= m (hidden), at most 2^31; n, m below 2^31 with
 * ceil(n/16) ceil(m/16) < 2^24; tokens <= 65535 (n = 0 and tokens = 0 do
 * nothing); experts <= 1024, 1 <= topk <= min(experts, 64), experts times
 * ceil(hidden/16) or ceil(inter/16) < 2^24.
 * Alignment: X, Wr, residual and Y to their element, float arrays to 4 bytes,
 * the workspace to 256; packed codes to 16 bytes and packed scales to 4.
 * Row-major codes that are not aligned to 4 bytes take a slower kernel.  More
 * than a few tokens of an X whose rows are not 16-byte aligned are first copied
 * into the workspace by the linear layer.
 */
#ifndef NVFP4_FFN_H
#define NVFP4_FFN_H

#include <stddef.h>
#include <stdint.h>

#include "nvfp4_gemv.h"
#include "nvfp4_mma.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types: NVFP4_OUT_F16 and NVFP4_OUT_BF16 of nvfp4_mma.h (X and Y),
 * and fp32 (Y only). */
#define NVFP4_OUT_F32 2

#define NVFP4_W_ROW_MAJOR 0
#define NVFP4_W_PACKED 1

/* Activation f.  GELU is z (1 + erf(z / sqrt 2)) / 2, GELU_TANH its tanh form
 * z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2, SILU z / (1 + exp(-z)).
 * NVFP4_ACT_GATED is added to one of them for the gated linear layer; the
 * MoE layer is always gated and takes the plain names. */
#define NVFP4_ACT_NONE 0
#define NVFP4_ACT_RELU 1
#define NVFP4_ACT_GELU 2
#define NVFP4_ACT_GELU_TANH 3
#define NVFP4_ACT_SILU 4
#define NVFP4_ACT_GATED 16

#define NVFP4_SCORE_SOFTMAX 0
#define NVFP4_SCORE_SIGMOID 1

/*
 * Bytes of workspace nvfp4_linear_launch_ws needs for this shape, whatever the
 * types, strides and alignment of the operands (0: none; then the workspace
 * may be NULL).  Returns 0 for invalid shapes as well.
 */
size_t nvfp4_linear_workspace_size(int64_t n, int64_t m, int64_t k, int32_t activation);

/*
 * The linear layer above with a caller-owned workspace of `workspace_bytes`
 * bytes (not aliasing any argument, not used by other work that may run
 * concurrently).  Allocates nothing, so it can be captured into a graph.
 * Returns NVFP4_GEMV_OK or a negative status.
 */
int nvfp4_linear_launch_ws(const void *X, int32_t x_type, int64_t ldx,
                           const uint8_t *W, const uint8_t *sfW, int32_t w_layout,
                           const float *alpha, const float *bias,
                           const void *residual, int64_t ldr,
                           void *Y, int32_t y_type, int64_t ldy,
                           int64_t n, int64_t m, int64_t k, int32_t activation,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * The same with the library-owned per-(device, stream) workspace of
 * nvfp4_gemv_launch (grown on first need without synchronising; a call that
 * must grow it while `stream` is being captured returns WORKSPACE: see
 * nvfp4_workspace_reserve; what nvfp4_gemv_launch says of graphs that run at the
 * same time holds here).
 */
int nvfp4_linear_launch(const void *X, int32_t x_type, int64_t ldx,
                        const uint8_t *W, const uint8_t *sfW, int32_t w_layout,
                        const float *alpha, const float *bias,
                        const void *residual, int64_t ldr,
                        void *Y, int32_t y_type, int64_t ldy,
                        int64_t n, int64_t m, int64_t k, int32_t activation, void *stream);

/* What stays the same from call to call of one MoE layer. */
typedef struct nvfp4_moe_layer_t {
    const void *router;        /* [experts][hidden], x_type                               */
    const float *route_bias;   /* [experts] added to the scores for the choice, or NULL   */
    const uint8_t *W13, *sf13; /* gate and up of every expert, [experts][2][inter][hidden] */
                               /* codes and scales (packed: groups = 2 experts)           */
    const float *alpha13;      /* [experts][2] or NULL (1)                                */
    const uint8_t *W2, *sf2;   /* down, [experts][hidden][inter] (packed: groups = experts) */
    const float *alpha2;       /* [experts] or NULL (1)                                   */
    int64_t experts, hidden, inter;
    int32_t topk;
    int32_t x_type;            /* NVFP4_OUT_F16 or NVFP4_OUT_BF16: X and router           */
    int32_t w_layout;          /* NVFP4_W_*                                               */
    int32_t activation;        /* NVFP4_ACT_*, without NVFP4_ACT_GATED                    */
    int32_t scoring;           /* NVFP4_SCORE_*                                           */
    int32_t renormalize;       /* 0 or 1                                                  */
    float routed_scale;
    int32_t reserved;          /* must be 0                                               */
} nvfp4_moe_layer_t;

/*
 * Bytes of workspace nvfp4_moe_layer_launch_ws needs for `tokens` tokens (only
 * the layer's sizes are looked at).  Returns 0 for invalid shapes.
 */
size_t nvfp4_moe_layer_workspace_size(const nvfp4_moe_layer_t *layer, int64_t tokens);

/*
 * The MoE layer above; X as in the linear layer with k = hidden, residual and
 * Y with m = hidden, the workspace as in nvfp4_linear_launch_ws.
 */
int nvfp4_moe_layer_launch_ws(const nvfp4_moe_layer_t *layer, const void *X, int64_t ldx,
                              const void *residual, int64_t ldr, void *Y, int32_t y_type,
                              int64_t ldy, int64_t tokens, void *workspace,
                              size_t workspace_bytes, void *stream);

/* The same with the library-owned workspace, as nvfp4_linear_launch. */
int nvfp4_moe_layer_launch(const nvfp4_moe_layer_t *layer, const void *X, int64_t ldx,
                           const void *residual, int64_t ldr, void *Y, int32_t y_type,
                           int64_t ldy, int64_t tokens, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_FFN_H */
