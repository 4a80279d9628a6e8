/*
 * adam_train.h - C ABI of the operators beside the update that make the
 * gradients it reads: the embedding of tokens with its gradient, attention over
 * packed documents with its gradient, softmax cross entropy over a large
 * vocabulary with its gradient, and activation checkpoints in 8 bits with the
 * backward steps that read them.  They live in libadamw_mi355x.so with the calls of adam.h and
 * share its status codes, dtypes and manner:
 *   - plain pointers and sizes; the caller owns every buffer; nothing is
 *     allocated, nothing is read back and the host never waits, so every
 *     call that takes a stream can be recorded into a HIP graph;
 *   - a call runs on `stream`'s device (the current one for a NULL stream);
 *     every buffer must be usable there;
 *   - results do not depend on timing: no call adds with atomics, so the same
 *     inputs give the same bits;
 *   - a weight gradient is written (or accumulated) in the dtype that a
 *     handle's `g` holds (float, bf16 or fp16), so the buffer given to
 *     adam_tl_build as `g` is the buffer given here;
 *   - matrices are row-major, their rows `stride` elements apart (stride >=
 *     columns; any alignment of the element type).
 * Calls with no rows are valid and do what the sums over no rows say.
 * ADAM_ABI_VERSION counts changes of adam.h; a client that may meet a library
 * from before these calls looks for them by name.
 * Sizes: rows, columns and strides are each below 2^31 and a matrix may be of
 * any total size.  Weight gradients and cross entropy: rows at most 2^30; n, k
 * and hidden at most 2^21, vocab at most 2^21 - 256; and at most 2^22 tiles of
 * 256 x 256 in n x k, in vocab x hidden, and in piece_rows x vocab or hidden.
 */
#ifndef ADAMW_MI355X_ADAM_TRAIN_H
#define ADAMW_MI355X_ADAM_TRAIN_H

#include "adam.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Activation checkpoints in 8 bits
 * ------------------------------------------------------------------------
 * A checkpoint holds a rows x cols matrix as one 8-bit code per element and
 * one 8-bit scale per 32 consecutive elements of a row (the last block of a
 * row may be shorter).  With MAX the format's largest value (448 for e4m3,
 * 57344 for e5m2) and amax the block's largest finite magnitude:
 *   e     = the smallest integer >= -127 with amax <= MAX * 2^e
 *   code  = x * 2^-e rounded to the format (nearest, ties to even)
 *   value = code * 2^e
 * so no finite value is clipped, the scale is exact to apply, and decoding
 * to float or bf16 is exact but for results outside the type's normal range.
 * e4m3 has no infinities: an infinite or NaN element decodes to NaN; in e5m2
 * infinities stay.  A block without finite nonzero elements has e = -127.
 *
 * Layout of a checkpoint buffer (16-byte aligned, adam_act8_bytes long):
 *   codes   rows x P bytes, P = cols rounded up to a multiple of 32 (codes
 *           from cols to P are 0), from offset 0
 *   scales  rows x P/32 bytes, each e + 127, from offset rows * P rounded up
 *           to a multiple of 256
 */
typedef enum {
    ADAM_ACT8_E4M3 = 1, /* OCP 8-bit float: 4 exponent bits, 3 mantissa bits */
    ADAM_ACT8_E5M2 = 2  /* OCP 8-bit float: 5 exponent bits, 2 mantissa bits */
} adam_act8_format;

/* Bytes of a checkpoint of rows x cols (host only).  ADAM_EINVAL for a NULL
 * result or a size out of range. */
int adam_act8_bytes(int64_t rows, int64_t cols, int64_t *bytes);

/* Stores x (rows x cols; F32, BF16 or F16) as a checkpoint.  `ckpt` must not
 * overlap x.  Errors: ADAM_EINVAL (sizes, a NULL pointer with elements, a
 * ckpt that is not 16-byte aligned, an x that is not aligned to its type, an
 * unknown format); ADAM_EDTYPE; ADAM_EHIP. */
int adam_act8_store(const void *x, adam_dtype x_type, int64_t rows, int64_t cols, int64_t x_stride,
                    adam_act8_format format, void *ckpt, hipStream_t stream);

/* Decodes a checkpoint into x (rounded to x's type, nearest even: the value
 * that stands for an fp16 one from 61440 (e5m2) or 63488 (e4m3) on is 65536, inf
 * in fp16).
 * Errors as adam_act8_store. */
int adam_act8_load(const void *ckpt, adam_act8_format format, int64_t rows, int64_t cols, void *x,
                   adam_dtype x_type, int64_t x_stride, hipStream_t stream);

/* Gated activations: h = a(gate) * up.
 *   silu   a(x) = x / (1 + exp(-x))
 *   gelu   a(x) = x/2 * (1 + tanh(sqrt(2/pi) * (x + 0.044715 x^3)))
 * gate, up, h and the gradients share one type (F32, BF16 or F16); the
 * arithmetic is float and each result is rounded once. */
typedef enum { ADAM_ACT_SILU = 1, ADAM_ACT_GELU = 2 } adam_act;

/* h = a(gate) * up, and in the same pass the checkpoints of gate and up
 * (both or neither; h comes from the unrounded inputs).  gate and up are rows
 * `in_stride` apart: two halves of one projection's output, or two buffers.
 * The outputs must not overlap each other or the inputs.  Errors:
 * ADAM_EINVAL (as adam_act8_store, one checkpoint without the other);
 * ADAM_EDTYPE; ADAM_EHIP. */
int adam_glu_forward(const void *gate, const void *up, adam_dtype type, int64_t rows, int64_t cols,
                     int64_t in_stride, adam_act act, void *h, int64_t h_stride, adam_act8_format format,
                     void *ckpt_gate, void *ckpt_up, hipStream_t stream);

/* The backward pass of h = a(gate) * up from the checkpoints, with g and u
 * their decoded values:
 *   dup = dh * a(g),  dgate = dh * u * a'(g),  h = a(g) * u
 * h (rows h_stride apart) and its checkpoint ckpt_h are written where their
 * pointer is not NULL: what the projection behind h needs for its own weight
 * gradient, so h itself need not be kept.  ckpt_h is the checkpoint of the
 * float value, not of the rounded h.  dgate and dup are rows d_stride apart.
 * No output may overlap another buffer, but dgate or dup may be dh itself
 * (the same address and stride).
 * Errors as adam_glu_forward. */
int adam_glu_backward(const void *dh, adam_dtype type, int64_t rows, int64_t cols, int64_t dh_stride,
                      adam_act act, adam_act8_format format, const void *ckpt_gate, const void *ckpt_up,
                      void *dgate, void *dup, int64_t d_stride, void *h, int64_t h_stride, void *ckpt_h,
                      hipStream_t stream);

/* Weight gradient of y = x w^T from the checkpoint of x:
 *   dw[n][k] = (accumulate ? dw[n][k] : 0) + sum over t of dy[t][n] * x^[t][k]
 * dy is rows x n (BF16 or F16), x^ the decoded checkpoint of rows x k.  x^ is
 * taken in dy's type: exact in bf16 (above its subnormals); for fp16 it is
 * halved, so that values of 2^17 and more become inf and those below 2^-20 lose
 * bits, and the sum doubled.  Products and
 * sums are float; dw (F32 or dy's type, n x k) is rounded once.  With no
 * rows the sum is 0.
 *   workspace   device, 256-byte aligned, of at least the bytes that
 *               adam_act8_wgrad_workspace gives for the same arguments; may be
 *               NULL if that is 0.  Its contents do not matter before the call
 *               and mean nothing after it; two calls, or two graphs
 *               that hold one, need two where they may run at once.
 * Errors: ADAM_EINVAL (as adam_act8_store; accumulate not 0/1; a workspace
 * too small or misaligned); ADAM_EDTYPE; ADAM_EHIP. */
int adam_act8_wgrad_workspace(int64_t rows, int64_t n, int64_t k, const void *dy, int64_t dy_stride,
                              int64_t *bytes);
int adam_act8_wgrad(const void *dy, adam_dtype dy_type, int64_t dy_stride, const void *ckpt,
                    adam_act8_format format, int64_t rows, int64_t n, int64_t k, void *dw, adam_dtype dw_type,
                    int64_t dw_stride, int32_t accumulate, void *workspace, int64_t workspace_bytes,
                    hipStream_t stream);

/* ------------------------------------------------------------------------
 * Softmax cross entropy over a large vocabulary
 * ------------------------------------------------------------------------
 * For each row i with hidden state h[i] (hidden elements) and target t[i]:
 *   z     = w h[i]                       (vocab logits)
 *   lse   = log(sum over v of exp(z[v]))
 *   loss  = weight[i] * (lse - z[t[i]])
 * and for the gradient of  L = loss_scale * (sum of loss):
 *   p[v]  = exp(z[v] - lse),   G[i][v] = weight[i] * (p[v] - (v == t[i]))
 *   dh    = loss_scale * G w,   dw = (accumulate ? dw : 0) + loss_scale * G^T h
 * A row whose target is ignore_index has loss 0, lse 0 and dh 0 and adds
 * nothing to dw, whatever its hidden state holds (NaN too); it is not
 * computed.  A row whose target is neither that nor in [0, vocab) has loss
 * NaN and a gradient of NaN, which adam_clip_grad_scale's found-inf flag
 * catches.  Logits may be of any finite size, or -inf.  A row with one of +inf
 * has lse inf and, unless that is the target's, loss inf; one with a NaN has
 * both NaN; the gradient of either is NaN.
 * The logits are never stored: the vocabulary is walked in pieces of 128 with
 * a running maximum and sum.  The gradient holds 16 bits for each logit of
 * `piece_rows` rows at a time: first exp(z - the piece's maximum), with 11
 * significant bits (BF16) or 12 (F16), then G in its place.
 * Products, statistics and sums are float.  G is rounded to h's type for the
 * products that make dh and dw (up to 128 rows, whose roundings would not
 * average out: to a sum of two such values); a float dw keeps that rounding.  In fp16 G is held in units that
 * keep an entry's rounding within 2^-11 of it or 2^-39 of the largest finite
 * |weight| of the computed rows, whichever is more.
 */
typedef struct {
    int64_t rows;         /* >= 0 */
    int64_t hidden;       /* >= 1 */
    int64_t vocab;        /* >= 1 */
    adam_dtype type;      /* of h, w and dh: BF16 or F16 */
    adam_dtype dw_type;   /* of dw: F32, or `type` */
    const void *h;        /* device: rows x hidden */
    int64_t h_stride;
    const void *w;        /* device: vocab x hidden */
    int64_t w_stride;
    const int64_t *target; /* device: rows */
    const float *weight;  /* device: rows, or NULL (all 1) */
    int64_t ignore_index;
    float *loss;          /* device: rows; required */
    float *lse;           /* device: rows, or NULL */
    void *dh;             /* device: rows x hidden, or NULL (not wanted) */
    int64_t dh_stride;
    void *dw;             /* device: vocab x hidden, or NULL (not wanted) */
    int64_t dw_stride;
    int32_t accumulate;   /* 1: dw is added to, 0: dw is overwritten */
    const float *d_loss_scale; /* device float, or NULL (1) */
    int64_t piece_rows;   /* rows held at once: 0 = automatic (loss alone:
                             16384; with gradient: as many as keep the 16-bit
                             G within 1 GiB, at least 256, or all rows where
                             that takes no more workspace than the float sums
                             that a 16-bit dw needs over several pieces); else
                             rounded up to a multiple of 256.  dw may depend
                             on it in the last bits. */
} adam_xent_desc;

/* What a call needs and does (host only; reads from *desc the sizes, types,
 * strides, the alignment of w, and which of dh and dw are given; no device
 * memory). */
typedef struct {
    int64_t workspace_bytes;
    int64_t piece_rows;   /* rows held at once */
    int64_t pieces;       /* pieces the rows are taken in */
} adam_xent_stats;

int adam_xent_plan(const adam_xent_desc *desc, adam_xent_stats *stats);

/* Losses (and, where dh or dw is given, gradients) of all rows.
 *   workspace   device, 256-byte aligned, at least adam_xent_plan's
 *               workspace_bytes for the same *desc; contents as in
 *               adam_act8_wgrad.
 * No output may overlap another buffer.  *desc is not retained.
 * Errors: ADAM_EINVAL (a NULL required pointer, sizes or strides out of
 * range, misaligned buffers, accumulate not 0/1, a workspace too small);
 * ADAM_EDTYPE; ADAM_EHIP. */
int adam_xent(const adam_xent_desc *desc, void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Embedding
 * ------------------------------------------------------------------------
 *   y[t] = scale * w[token[t]]
 * rounded once to y's type (any of F32, BF16, F16, as w's).  A row whose token
 * is ignore_index is 0; one whose token is neither that nor in [0, vocab) is
 * NaN.  w has `vocab` rows of `hidden`.  y must not overlap w or the tokens.
 * Errors: ADAM_EINVAL (sizes, strides, a NULL pointer with elements, misaligned
 * buffers, a scale that is not finite, overlap; with rows, vocab 0);
 * ADAM_EDTYPE; ADAM_EHIP. */
int adam_embed_forward(const int64_t *token, int64_t rows, const void *w, adam_dtype w_type, int64_t vocab,
                       int64_t hidden, int64_t w_stride, float scale, int64_t ignore_index, void *y,
                       adam_dtype y_type, int64_t y_stride, hipStream_t stream);

/* Its gradient, by sorted tokens:
 *   dw[v] = (accumulate ? dw[v] : 0) + scale * sum over t with token[t] == v of dy[t]
 * for every v in [0, vocab): without accumulate rows of dw that no token names
 * become 0, with it they are neither read nor written.  Tokens equal to
 * ignore_index or outside [0, vocab) add nothing, whatever their dy holds.  The
 * sum is float, over the tokens in their order by fixed parts, and dw (F32, BF16
 * or F16, as dy) is rounded once.  scale is applied to the sum.
 *   workspace   device, 256-byte aligned, at least adam_embed_backward_workspace
 *               bytes for the same sizes; contents as in adam_act8_wgrad.
 * rows and hidden at most 2^30 in both.  Errors as adam_embed_forward; ADAM_EINVAL also for
 * accumulate not 0/1 and a workspace too small, misaligned or overlapping. */
int adam_embed_backward_workspace(int64_t rows, int64_t vocab, int64_t hidden, int64_t *bytes);
int adam_embed_backward(const int64_t *token, int64_t rows, const void *dy, adam_dtype dy_type, int64_t dy_stride,
                        float scale, int64_t ignore_index, void *dw, adam_dtype dw_type, int64_t vocab,
                        int64_t hidden, int64_t dw_stride, int32_t accumulate, void *workspace,
                        int64_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Attention over packed documents
 * ------------------------------------------------------------------------
 * `rows` tokens hold documents one behind the other: document d is the rows
 * doc_offsets[d] .. doc_offsets[d + 1] - 1.  Row i of document d sees the keys j
 * of that document
 *   causal            with j <= i
 *   causal, prefix    with j <= i or j < doc_offsets[d] + prefix[d]
 *   causal, window    with i - window < j <= i
 *   not causal        all
 * For each query head h, with key/value head g = h / (heads / kv_heads):
 *   z[i][j] = scale * (q[i][h] . k[j][g])
 *   z[i][j] = softcap * tanh(z[i][j] / softcap)      where softcap > 0
 *   z[i][j] -= slopes[h] * |i - j|                   where slopes are given
 *   lse[h][i] = log(sum over the seen j of exp(z[i][j]))
 *   o[i][h]   = sum over the seen j of exp(z[i][j] - lse[h][i]) v[j][g]
 * and the gradient, for an upstream gradient dout of o:
 *   dp[i][j] = dout[i][h] . v[j][g],   delta = sum over d of dout[i][h][d] o[i][h][d]
 *   ds[i][j] = p[i][j] (dp[i][j] - delta)  (times 1 - tanh^2 where capped)
 *   dq = scale ds k,  dk = scale ds^T q,  dv = p^T dout, dk and dv summed over
 *   the query heads that share the key head; the slopes are constants.
 * Rows of no document (before the first offset, behind the last) are neither
 * read nor written: their o, lse and gradients stay as they were.  What a row
 * does not see never reaches it: not a NaN nor an infinity either.
 * Nothing of the size rows x rows is stored.  Products, sums and statistics are
 * float; p and ds are rounded to the 16-bit type for the products they enter (in
 * F16 in units that follow a row's largest value, so that no gradient's size
 * loses its bits), outputs are rounded once.
 *
 * A tensor's element (row, head, d) lies at row * stride + head * head_stride + d
 * elements; q, dout, o, dq have `heads` heads, k, v, dk, dv `kv_heads`.  So the
 * heads of one token may lie side by side, also as a part of a fused projection's
 * output, or each head's rows may follow each other.
 */
typedef struct {
    int64_t rows;         /* >= 0, at most 2^30 */
    int64_t heads;        /* >= 1, at most 65535; a multiple of kv_heads */
    int64_t kv_heads;     /* >= 1 */
    int64_t head_dim;     /* 1 to 256 */
    adam_dtype type;      /* of q, k, v, o and their gradients: BF16 or F16 */
    const void *q;        /* device; strides of inputs 0 to 2^21, head strides >= 0 */
    int64_t q_stride, q_head_stride;
    const void *k;
    int64_t k_stride, k_head_stride;
    const void *v;
    int64_t v_stride, v_head_stride;
    void *o;              /* written by the forward pass, read by the backward pass */
    int64_t o_stride, o_head_stride;
    float *lse;           /* device: heads x rows; may be NULL in the forward pass */
    const int32_t *doc_offsets; /* device: docs + 1, not decreasing, within [0, rows]
                             (others give unspecified results, but no access
                             outside the buffers); NULL: one document of all rows */
    int64_t docs;         /* documents (without doc_offsets: 1) */
    const int32_t *prefix; /* device: docs, each >= 0 (longer than its document: all
                             of it); or NULL.  Needs causal, and no window */
    int32_t causal;       /* 1 or 0 */
    int64_t window;       /* >= 1, or 0: none; needs causal */
    float scale;          /* > 0, finite */
    float softcap;        /* > 0, finite, or 0: none */
    const float *slopes;  /* device: heads, or NULL */
    const void *dout;     /* backward pass */
    int64_t dout_stride, dout_head_stride;
    void *dq;             /* each of dq, dk, dv is required */
    int64_t dq_stride, dq_head_stride;
    void *dk;
    int64_t dk_stride, dk_head_stride;
    void *dv;
    int64_t dv_stride, dv_head_stride;
} adam_attn_desc;

/* Workspaces of the two passes (host only; reads sizes and types from *desc). */
typedef struct {
    int64_t forward_bytes;
    int64_t backward_bytes;
} adam_attn_stats;

int adam_attn_plan(const adam_attn_desc *desc, adam_attn_stats *stats);

/* The forward pass (the fields behind `slopes` are not read), and the backward
 * pass, which reads o and lse as the forward pass left them for the same q, k, v
 * and mask.  *desc is not retained.
 *   workspace   device, 256-byte aligned, at least the pass's bytes by
 *               adam_attn_plan (NULL where that is 0); contents as in
 *               adam_act8_wgrad.
 * No output may share a byte with another buffer; outputs that lie between each
 * other's rows or heads (equal strides) are fine.
 * Errors: ADAM_EINVAL (a NULL required pointer, sizes, strides or flags out of
 * range, a mask combination above, misaligned buffers, overlap, a workspace too
 * small); ADAM_EDTYPE; ADAM_EHIP. */
int adam_attn_forward(const adam_attn_desc *desc, void *workspace, int64_t workspace_bytes, hipStream_t stream);
int adam_attn_backward(const adam_attn_desc *desc, void *workspace, int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ADAMW_MI355X_ADAM_TRAIN_H */
