/*
 * muon_lm.h - the language-model operators of libmuon.so (MI355X, gfx950):
 * attention with its gradients, the norm and rotation of query and key heads
 * with its gradients, and the embedding with its gradient.  They compute the
 * model around the Muon step of muon.h.
 *
 * Conventions (those of muon.h)
 *  - Device pointers; the caller owns every buffer and the workspace (aligned
 *    to 256 bytes, contents on entry do not matter).  The library allocates
 *    nothing and keeps nothing between calls.
 *  - `stream` is a hipStream_t; work is ordered on it and the call returns
 *    without synchronising.  Every launch is a kernel, so calls can be
 *    captured into a graph.
 *  - Arguments are validated before anything is enqueued: a non-zero status
 *    enqueues nothing, and muon_last_error() describes it.
 *  - What a call writes, the workspace included, must not overlap anything it
 *    reads or writes besides, unless its comment allows that, and elements of
 *    one output must not overlap; the library does not check it.
 *  - The same inputs give the same bits every time: no sum depends on the
 *    order in which workgroups run.
 *  - Values on the device (lengths, positions, tokens, ...) cannot be checked
 *    by the call; each is bounded in the kernels as its field says, so none
 *    makes a kernel read or write out of range.
 */
#ifndef MUON_LM_H
#define MUON_LM_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest head size of attention (multiples of 8) and of the norm with
 * rotation (even). */
#define MUON_ATTENTION_MAX_D 128
#define MUON_QK_NORM_MAX_D 512

/*
 * Attention over bfloat16 heads, and its gradients.
 *
 *   z_ij  = scale q_i . k_j
 *   z_ij  = softcap tanh(z_ij / softcap)            softcap > 0
 *   z_ij -= slopes[head] |p_i - j|                  slopes given
 *   lse_i = log sum_j exp z_ij, out_i = sum_j exp(z_ij - lse_i) v_j
 *
 * over the keys j that query i, at position p_i = starts[batch] + i, sees:
 *   ((not causal or j <= p_i) and (window = 0 or |p_i - j| < window))
 *      or j < prefix[batch]
 *   and documents[batch][p_i] = documents[batch][j]   documents given
 *   and p_i < lengths[batch] and j < lengths[batch]   lengths given
 * A query that sees no key has out = 0, lse = -inf and takes no part in the
 * gradients.  Query head h uses key head h / (heads / kv_heads), and the
 * gradients of a shared key head sum over its query heads.
 *
 * Memory past lengths[batch] may hold anything, NaN included, and so may k and
 * v past the last key that any query of the batch sees (a cache past its last
 * position), and q and dout of a query that sees no key.  (Other NaNs and
 * infinities can reach other rows of the batch through 0 * inf: also of keys in
 * front of every window or of documents that no query has, and with both
 * prefix and documents of queries past the last key's window.)
 *
 * Scores, statistics and sums are float32.  exp(z - lse) and the gradient of
 * the scores are rounded to bfloat16 as operands of the matrix cores; the
 * backward pass takes sum dout out from the rounded out it is given.  A capped
 * score is good to 2^-22 of the cap up to a cap of 64, and to 2^-19 of itself
 * above.
 */
typedef struct muon_attention_args {
    const uint16_t *q;      /* [batch][sq][heads][d], bfloat16 */
    const uint16_t *k;      /* [batch][sk][kv_heads][d] */
    const uint16_t *v;      /* [batch][sk][kv_heads][d] */
    uint16_t *out;          /* [batch][sq][heads][d]; read by the backward pass */
    float *lse;             /* [batch][heads][sq], contiguous; read by the backward pass */
    const uint16_t *dout;   /* backward pass: gradient of out */
    uint16_t *dq, *dk, *dv; /* backward pass: gradients, contiguous, shaped as q, k and v */
    /* strides of (batch, position, head) in elements, multiples of 8 with
     * 16-byte aligned pointers; the last dimension is contiguous */
    int64_t q_strides[3], k_strides[3], v_strides[3], out_strides[3], dout_strides[3];
    const float *slopes;      /* [heads], or NULL */
    const int32_t *documents; /* [batch][sk], rows documents_stride apart, or NULL; p_i is clamped to 0 .. sk - 1 */
    int64_t documents_stride;
    const int32_t *prefix;    /* [batch], or NULL; clamped to 0 .. length */
    const int32_t *lengths;   /* [batch], or NULL; clamped to 0 .. sk */
    const int32_t *starts;    /* [batch], or NULL: sk - sq; clamped to +-2^29 */
    int64_t batch, sq, sk, heads, kv_heads, d;
    int64_t causal;           /* 0 or 1 */
    int64_t window;           /* 0, or 2^29 and more: none */
    double scale;             /* > 0 */
    double softcap;           /* 0: none */
} muon_attention_args;

/* Bytes of workspace (at least 256; 0 for invalid arguments). */
size_t muon_attention_workspace_size(const muon_attention_args *args);
size_t muon_attention_backward_workspace_size(const muon_attention_args *args);

/*
 * out and lse from q, k and v.  out may be q (the same pointer and strides).
 * Errors: MUON_ERR_INVALID_ARG (null pointers, negative sizes, heads not a
 * multiple of kv_heads, misaligned pointers (16 bytes; 4 for lse, slopes and
 * the masks) or strides, a negative documents_stride, a scale that is not
 * positive and finite, a negative softcap or window), MUON_ERR_UNSUPPORTED (d
 * not a multiple of 8 up to 128, sq or sk of 2^29 or more, row strides of
 * 2^24 elements or more, more than 2^31 - 1 workgroups), MUON_ERR_WORKSPACE.
 */
int muon_attention(const muon_attention_args *args, void *workspace, size_t workspace_bytes, void *stream);

/* dq, dk and dv from dout, the forward pass's arguments and its out and lse.
 * dq may be out, and dk and dv may be k and v (one each), where those are
 * contiguous too.  dq is written before q and dout are read for dk and dv. */
int muon_attention_backward(const muon_attention_args *args, void *workspace, size_t workspace_bytes, void *stream);

/*
 * RMS norm over each query and key head and the rotation by position:
 *   r = 1 / sqrt(mean(x^2) + eps), y = x r weight, (a, b) = halves of y,
 *   z = (a cos - b sin, b cos + a sin)
 * with (cos, sin) = table[position][pair].  Computed in float32 and rounded
 * once.  Index 0 of each pair of fields is the queries', 1 the keys'.
 * Positions outside the table give NaN.  out[i] may be x[i] (backward: dz[i]
 * too) where that is contiguous.
 */
typedef struct muon_qk_norm_rope_args {
    const void *x[2];       /* [batch][positions][heads[i]][d] of dtype */
    void *out[2];           /* forward: z; backward: gradient of x; contiguous */
    const void *dz[2];      /* backward: gradient of z, of dtype */
    const float *weight[2]; /* [d], or NULL: ones */
    float *dweight[2];      /* backward: [d], or NULL */
    int64_t x_strides[2][3], dz_strides[2][3]; /* (batch, position, head), in elements */
    int64_t heads[2];
    const float *table;       /* [limit][d / 2][2]: cos, sin */
    int64_t limit;
    const int32_t *positions; /* [batch][s], contiguous, or NULL: 0 .. s - 1 */
    int64_t batch, s, d;
    int64_t dtype;            /* muon_dtype */
    double eps;
} muon_qk_norm_rope_args;

/* Bytes of workspace of the backward pass (at least 256; 0 for invalid sizes). */
size_t muon_qk_norm_rope_backward_workspace_size(const muon_qk_norm_rope_args *args);
int muon_qk_norm_rope(const muon_qk_norm_rope_args *args, void *stream);
int muon_qk_norm_rope_backward(const muon_qk_norm_rope_args *args, void *workspace, size_t workspace_bytes,
                               void *stream);

/*
 * out[i] = scale table[tokens[i]] (float32, rounded once to out's type).  A
 * token outside 0 .. vocab - 1 gives a row of NaN.  n and vocab are below 2^31 -
 * 1 and width up to 2^20 (MUON_ERR_UNSUPPORTED past that).
 *  tokens : [n], int64 (token_bytes 8) or int32 (token_bytes 4).
 *  table  : [vocab][width] of table_type; out: [n][width] of out_type.
 */
int muon_embedding(const void *tokens, int token_bytes, const void *table, int table_type, void *out, int out_type,
                   int64_t n, int64_t vocab, int64_t width, float scale, void *stream);

/* Bytes of workspace of the gradient (0 for invalid sizes). */
size_t muon_embedding_backward_workspace_size(int64_t n, int64_t vocab, int64_t width);

/*
 * dtable[t] = scale * the sum of dout[i] over the i with tokens[i] = t, in
 * float32 and one order, rounded once to table_type; rows of tokens that do
 * not occur are zero, and tokens outside the table take no part.
 */
int muon_embedding_backward(const void *tokens, int token_bytes, const void *dout, int dout_type, void *dtable,
                            int table_type, int64_t n, int64_t vocab, int64_t width, float scale, void *workspace,
                            size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MUON_LM_H */
