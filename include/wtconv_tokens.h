/*
 * wtconv_tokens.h -- C ABI of libwtconv's token operators (MI355X, gfx950).
 *
 * A pixel of a channels-last plane is a token: B planes of H x W pixels with C
 * channels are B H W rows of C channels.  The operators here are what a block
 * over such tokens needs beside the WTConv layer of wtconv.h:
 *
 *   rms_norm   h = x + residual (as stored), y = h / sqrt(mean_c h^2 + eps) * weight,
 *              forward and backward; or y in 8 bits with one scale per row
 *   rotary     pairs of channels turned by position angles, several axes
 *   attention  softmax(scale Q K^T) V inside each sequence of a pack, full or
 *              causal, grouped heads, forward and backward
 *   dropout    keep / drop from a counter-based generator, no stored mask
 *
 * Conventions (those of wtconv.h):
 *   - Tensor pointers are DEVICE pointers owned by the caller.  Nothing is
 *     allocated, freed or synchronised; calls are asynchronous on `stream`
 *     (a hipStream_t; NULL = default stream).
 *   - Activations are float32 (WTC_FP32) or bfloat16 bits (WTC_BF16); all
 *     sums, statistics and angles are float32.  Parameters, statistics and
 *     parameter gradients are float32.
 *   - Outputs are overwritten, never accumulated; results do not depend on
 *     the order in which workgroups run (no atomics).
 *   - Arguments are checked before any HIP call; a failed check returns a
 *     negative wtc_status and touches nothing.  A failed launch returns
 *     WTC_EHIP.  No C++ exception crosses this interface.
 *   - Counts of rows or tokens may be 0.  Strides are in elements; the last
 *     axis of every tensor is contiguous.
 */
#ifndef WTCONV_TOKENS_H
#define WTCONV_TOKENS_H

#include "wtconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Root-mean-square norm over rows
 * ---------------------------------------------------------------------- */
#define WTC_RMS_MAX_C 16384 /* channels of a row: it is held in registers */

typedef struct {
    long long rows;               /* >= 0                                              */
    long long x_stride, r_stride; /* row strides of x (backward: of h) and the residual */
    long long g_stride;           /* backward: row stride of dy                         */
    int C;                        /* channels, 1 .. WTC_RMS_MAX_C                       */
    int dtype;                    /* wtc_dtype of x, residual, h, dy, dh, dx (and y)    */
    int fp8;                      /* 1: y is e4m3 with a scale per row (forward only)   */
    float eps;                    /* >= 0                                               */
} wtc_rms_desc;

/* h = x + residual rounded to the storage type (what the residual stream
 * holds; without residual, h = x and the argument h is NULL);
 *   rstd = 1 / sqrt(mean_c h^2 + eps),  y = h rstd weight.
 * weight [C] float32; y and h [rows, C] contiguous; rstd [rows] float32 or
 * NULL (kept for the backward pass).
 * fp8 = 1: y is one byte per element (e4m3, largest value 448), scale [rows]
 *   scale = max(max_c |y| / 448, 2^-100),   y8 = e4m3(y / scale)
 * (an all-zero row has y8 = 0; the quotient is y times scale's rounded
 * reciprocal, within two roundings of float32 before the 8 bits' own; a NaN is
 * no maximum: it stays a NaN in y8 alone).  scale is NULL when fp8 = 0. */
int wtconv_rms_norm_forward(const wtc_rms_desc* d, const void* x, const void* residual, const float* weight, void* y,
                            void* h, float* rstd, float* scale, void* stream);

/* Given dy and (or NULL) dh, the gradient that reaches h by its other use:
 *   xh = h rstd,  u = dy weight,  dx = dh + rstd (u - xh mean_c(u xh)),
 *   dw = sum over rows of dy xh.
 * dx [rows, C] contiguous is the gradient of x and of the residual alike; dh
 * contiguous; dw [C].  The workspace holds the rows' partial sums of dw. */
size_t wtconv_rms_norm_backward_workspace(const wtc_rms_desc* d);
int wtconv_rms_norm_backward(const wtc_rms_desc* d, const void* dy, const void* dh, const void* h, const float* weight,
                             const float* rstd, void* dx, float* dw, void* workspace, size_t workspace_bytes,
                             void* stream);

/* ------------------------------------------------------------------------
 * Rotary positions with several axes
 * ---------------------------------------------------------------------- */
#define WTC_ROTARY_MAX_AXES 4

typedef struct {
    long long T;                /* tokens, >= 0                                          */
    long long x_token, x_head;  /* strides of x                                          */
    long long y_token, y_head;  /* strides of y                                          */
    int heads, D;               /* heads and channels per head, >= 1                     */
    int dtype;                  /* wtc_dtype of x and y                                  */
    int axes;                   /* 1 .. WTC_ROTARY_MAX_AXES                              */
    int pairs[WTC_ROTARY_MAX_AXES]; /* pairs turned by each axis; P = their sum <= D / 2 */
    int interleaved;            /* pair p is channels (p, P + p), or with 1 (2p, 2p + 1) */
    int inverse;                /* 1: turned by the negative angles (the backward pass)  */
} wtc_rotary_desc;

/* Pair p, of axis a (the first pairs[0] pairs are axis 0's, and so on), of
 * token t is turned by the angle positions[t * axes + a] * inv_freq[p]
 * (a float32 product):  (u, v) -> (u cos - v sin, u sin + v cos).
 * Channels from 2P on are copied.  positions [T, axes] int32, inv_freq [P]
 * float32.  y may be x (same strides); it must not overlap x otherwise. */
int wtconv_rotary(const wtc_rotary_desc* d, const void* x, const int* positions, const float* inv_freq, void* y,
                  void* stream);

/* ------------------------------------------------------------------------
 * Dropout
 * ---------------------------------------------------------------------- */
/* y[i] = residual[i] + (bits[i] >= r ? x[i] * 65536 / (65536 - r) : 0),
 * r = round(65536 p), for i < n (contiguous tensors of one shape; residual may
 * be NULL, and y may be x or the residual).  bits[i] is half-word i % 8 (low
 * halves first) of the four words of the counter-based generator Philox
 * 4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as
 * 1, 2, 3", 2011) with
 *   counter = (i / 8 low, i / 8 high, offset low, offset high),
 *   key = (seed low, seed high),   rng = {seed, offset} in device memory.
 * The same rng gives the same decisions in every call: the backward pass is
 * this call on dy without a residual, and no mask is stored.  Probabilities
 * are multiples of 2^-16.  A dropped element never reaches y, not even a NaN;
 * 0 <= p <= 1. */
int wtconv_dropout(long long n, int dtype, double p, const void* x, const void* residual,
                   const unsigned long long* rng, void* y, void* stream);

/* ------------------------------------------------------------------------
 * Attention over packed sequences
 * ---------------------------------------------------------------------- */
#define WTC_ATTN_MAX_D 128
#define WTC_ATTN_MAX_TOKEN_STRIDE (1 << 22)

typedef struct {
    long long token, head; /* strides in elements, multiples of 16 bytes;
                              token <= WTC_ATTN_MAX_TOKEN_STRIDE */
} wtc_attn_strides;

typedef struct {
    long long T;   /* tokens of the pack, >= 0, < 2^31                            */
    int n_seq;     /* sequences, >= 0                                             */
    int Hq, Hk;    /* heads of q and of k and v; Hq a multiple of Hk              */
    int D;         /* channels per head: a multiple of 8, 8 .. WTC_ATTN_MAX_D     */
    int dtype;     /* wtc_dtype of every activation                               */
    int causal;    /* 1: a token sees itself and those before it in its sequence  */
    float scale;   /* of the products q . k; finite                               */
    wtc_attn_strides q, k, v, o;         /* inputs and the output                 */
    wtc_attn_strides g, dq, dk, dv;      /* backward: dout and the gradients      */
} wtc_attn_desc;

/* out[i, h] = sum_j softmax_j(scale q[i, h] . k[j, h / group]) v[j, h / group],
 * j over the tokens of i's sequence (causal: j <= i), group = Hq / Hk.
 * cu_seqlens [n_seq + 1] int32: sequence s is the tokens cu_seqlens[s] up to
 * cu_seqlens[s + 1], non-decreasing; entries are clamped to 0 .. T on the
 * device, a sequence may be empty, and tokens that belong to none get zero
 * outputs and zero gradients.  lse [Hq, T] float32 or NULL: the logarithm of
 * each row's sum of exp (+infinity for tokens of no sequence), kept for the
 * backward pass.  out_low [T, Hq, D] bfloat16 contiguous or NULL: what was
 * rounded off out (bfloat16 only), kept for a backward pass whose row sums of
 * dout . out then have 16 bits of out.  Tensors are 16-byte aligned.  A value
 * that is not finite never reaches another sequence; inside its sequence it may
 * reach every row.  float32 values above bfloat16's largest (3.3895e38) count as
 * infinite, and results that an infinity would leave infinite may be NaN.
 * Speed: with few tiles (heads and 128 queries) a tile's keys are shared by
 * workgroups when the mean length T / n_seq is long; leave out empty sequences
 * and those of few tokens where one long sequence should be.
 * The workspace holds partial results where a short pack's keys are split over
 * workgroups (0 bytes, and NULL is taken, where they are not).
 * WTC_ESHAPE: more than about 2^30 / Hq tokens (2^23 workgroups). */
size_t wtconv_attention_forward_workspace(const wtc_attn_desc* d);
int wtconv_attention_forward(const wtc_attn_desc* d, const void* q, const void* k, const void* v,
                             const int* cu_seqlens, void* out, float* lse, void* out_low, void* workspace,
                             size_t workspace_bytes, void* stream);

/* dq, dk, dv from dout and the forward pass's out, lse and out_low (or NULL);
 * dk and dv are summed over the q heads of their group.  Fixed summation order. */
size_t wtconv_attention_backward_workspace(const wtc_attn_desc* d);
int wtconv_attention_backward(const wtc_attn_desc* d, const void* q, const void* k, const void* v, const void* out,
                              const float* lse, const void* out_low, const void* dout, const int* cu_seqlens,
                              void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WTCONV_TOKENS_H */
