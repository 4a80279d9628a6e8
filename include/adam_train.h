/*
 * adam_train.h - C ABI of the operators beside the update that make the
 * gradients it reads: softmax cross entropy over a large vocabulary with its
 * gradient, and activation checkpoints in 8 bits with the backward steps that
 * read them.  They live in libadamw_mi355x.so with the calls of adam.h and
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

#ifdef __cplusplus
}
#endif

#endif /* ADAMW_MI355X_ADAM_TRAIN_H */
