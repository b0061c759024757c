/*
 * pamm_positions.h -- C ABI of what stands between a PAMM projection and its
 * attention: rotary positions of queries and keys, and their norm for each
 * head with the rotation in the same pass.  Conventions, tensors and errors
 * as in pamm_block.h.
 */
#ifndef PAMM_POSITIONS_H
#define PAMM_POSITIONS_H

#include "pamm_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * One call.  For each head row x of q and k, with p = the token's position:
 *
 *   n = x                                              without weights
 *   n_e = x_e rstd w_e,  rstd = 1 / sqrt(mean_e x_e^2 + eps)     with them
 *
 *   t_j = p inv_freq[j],  j < rot_dim / 2              (radians, formed in 64 bits)
 *   y_a = magnitude (n_a cos t_j - n_b sin t_j)
 *   y_b = magnitude (n_a sin t_j + n_b cos t_j)
 *     half:         a = j,   b = j + rot_dim / 2
 *     interleaved:  a = 2 j, b = 2 j + 1
 *   y_e = n_e for e >= rot_dim.
 *
 * inverse (without weights) turns by -t_j: the gradient of the rotation.
 *
 * Token (b, s) has the position positions[b, s] (s if NULL) + offset[b] (0 if
 * NULL).  positions holds int64 or int32 elements, position_stride_b and
 * position_stride_s elements apart (0: shared).
 */
typedef struct {
    int32_t dtype;            /* of q, k, the results and the weights */
    int32_t interleaved;      /* 0: half, 1: interleaved */
    int32_t inverse;          /* 0 or 1; 0 with weights */
    int32_t positions_64;     /* positions: 1 int64, 0 int32 */
    int64_t batch, seq, heads_q, heads_k;  /* heads_k 0: no k */
    int64_t head_dim;         /* 1 .. PAMM_MAX_HEAD_DIM, a multiple of 16 bytes */
    int64_t rot_dim;          /* even, 0 .. head_dim */
    float magnitude, eps;     /* finite; eps >= 0 */
    const double *inv_freq;   /* [rot_dim / 2] */
    const void *positions;
    int64_t position_stride_b, position_stride_s;   /* >= 0 */
    const int32_t *offset;    /* [batch] or NULL */
    const void *q_weight, *k_weight;  /* [head_dim] each, 16-byte aligned, or both NULL (k_weight NULL without k) */
    pamm_heads_t q, k;        /* read */
    pamm_heads_t q_out, k_out;/* written; each may be its input itself, and must not meet anything else */
} pamm_rotary_t;

/*
 * Sums and products in 32 bits, each result rounded once; cos and sin are within 4 * 2^-24 for angles of
 * any size that 64 bits hold to that precision.  Rows stand alone: what is not finite in one
 * changes no other.  A row whose sum of squares passes fp32's range has rstd = 0.
 *
 * Errors: PAMM_ERR_NULL, _DTYPE, _SHAPE (sizes out of range, batch * seq beyond 2^31 - 1, a negative
 * or huge stride), _VALUE (a flag that is not 0 or 1, inverse with weights, magnitude or eps out of
 * range), _ALIGN.
 */
int pamm_rotary(const pamm_rotary_t *a_host, void *stream);

/* Bytes of workspace pamm_rotary_backward needs: partial sums of the weights' gradients. */
size_t pamm_rotary_backward_workspace_size(const pamm_rotary_t *a_host);

/*
 * Gradients of pamm_rotary with weights, from those of its results (dq_out, dk_out) and its inputs q, k:
 *
 *   g = the inverse rotation of dy,  u = g w,  xhat = x rstd
 *   dx = rstd (u - xhat mean_e(u xhat)),   dw = sum over tokens and heads of g xhat
 *
 * a->q_out and a->k_out are the gradients dq, dk that are written (they may be dq_out, dk_out themselves);
 * dq_weight, dk_weight [head_dim] fp32, written (dk_weight NULL without k).  Errors as pamm_rotary;
 * _NULL without weights; _WORKSPACE.  Bitwise deterministic.
 */
int pamm_rotary_backward(const pamm_rotary_t *a_host, const pamm_heads_t *dq_out_host,
                         const pamm_heads_t *dk_out_host, float *dq_weight, float *dk_weight, void *ws,
                         size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAMM_POSITIONS_H */
