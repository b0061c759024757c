/*
 * pamm_block.h -- C ABI of the operators around a PAMM projection in a
 * transformer block: attention with a backward pass that recomputes its
 * probabilities, the residual addition with its root-mean-square norm, and
 * the global gradient norm with clipping.  They live in the same library as
 * the calls of pamm.h and follow its conventions:
 *
 *   - Pointers are DEVICE pointers unless the parameter name ends in _host.
 *     The caller owns every buffer, the workspace included; nothing here
 *     allocates, synchronises or keeps state between calls.
 *   - `stream` is a hipStream_t passed as void* (NULL = the legacy default
 *     stream); work is enqueued asynchronously.
 *   - dtype: PAMM_F32 or PAMM_BF16.  Sums, softmax statistics and norms are
 *     held in 32 bits or more.  Results are bitwise deterministic.
 *   - Every call returns a pamm_status_t, validates its arguments before
 *     anything is enqueued, and writes nothing on an error.
 *   - The workspace needs 256-byte alignment; calls that may run
 *     concurrently need workspaces of their own.
 */
#ifndef PAMM_BLOCK_H
#define PAMM_BLOCK_H

#include "pamm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further pamm_status_t: written ranges of one call share memory. */
#define PAMM_ERR_OVERLAP 10

/* Largest head dimension of the attention calls. */
#define PAMM_MAX_HEAD_DIM 128

/* A [batch x sequence x heads x head_dim] tensor: element (b, s, h, e) lies
 * at data + b * stride_b + s * stride_s + h * stride_h + e (strides in
 * elements, >= 0).  Any order of the three outer dimensions is allowed, so a
 * slice of a packed projection output or a [batch x heads x sequence x dim]
 * cache is passed as it is.  data 16-byte aligned and strides multiples of 16
 * bytes.  Strides of 0 (broadcast) are allowed on tensors that are read. */
typedef struct {
    void *data;
    int64_t stride_b, stride_s, stride_h;
} pamm_heads_t;

/*
 * One attention problem.  Query head h uses key/value head h / (heads /
 * heads_kv).  With Lq = q_len[b] (seq_q if q_len is NULL) and Lk = kv_len[b]
 * (seq_k if NULL), query i < Lq of sequence b sees the keys j with
 *
 *   j < Lk,
 *   causal:      j <= i + Lk - Lq   (the last query sees the last key),
 *   window > 0:  j >  i + Lk - Lq - window   (causal only),
 *
 * and no other: K and V at or past Lk are never read.  Lengths outside
 * [0, seq] are clamped into it.
 */
typedef struct {
    int32_t dtype;      /* of q, k, v, o and the gradients */
    int32_t causal;     /* 0 or 1 */
    int64_t batch, seq_q, seq_k;
    int64_t heads, heads_kv;  /* heads_kv >= 1 divides heads */
    int64_t head_dim;   /* 1 .. PAMM_MAX_HEAD_DIM, a multiple of 16 bytes */
    int64_t window;     /* 0: no window */
    float scale;        /* finite; scores are scale * <q, k> */
    const int32_t *q_len, *kv_len;   /* [batch] or NULL */
    pamm_heads_t q, k, v;            /* read */
    pamm_heads_t o;     /* pamm_attention writes it, the backward pass reads it */
    float *lse;         /* [batch x heads x seq_q], contiguous; as o */
} pamm_attention_t;

/* Bytes of workspace pamm_attention needs: 0 unless the keys are split over
 * workgroups because there are few queries (the partial results of each part).
 * Pointers are not looked at, except whether kv_len is given. */
size_t pamm_attention_workspace_size(const pamm_attention_t *a_host);

/*
 *   lse[b, h, i] = log sum_j exp(s_ij)            s_ij = scale * <q_i, k_j>
 *   o[b, i, h]   = sum_j exp(s_ij - lse_i) v_j    over the keys i sees
 *
 * What a mask hides does not come through, not even a NaN or an infinity.
 * A query that sees no key (and every i >= q_len[b]) gets o = 0 and
 * lse = -infinity; so does one whose every score is -infinity.  bf16: products
 * of bf16 values summed in fp32, probabilities rounded to bf16 for the
 * product with V, o rounded once.  fp32: fp32 throughout.  o and lse must not
 * overlap each other or any input; the stride of a dimension with one entry is
 * not looked at.
 *
 * Errors: PAMM_ERR_NULL, _DTYPE, _SHAPE (sizes < 0, heads not a multiple of
 * heads_kv, head_dim out of range, a stride that is negative or spans 2^40
 * elements, seq_q, seq_k or seq_q * heads / heads_kv beyond
 * 2^30 - 512, more workgroups than a grid holds), _VALUE (scale not finite, causal not 0 or 1, window < 0, window > 0
 * without causal), _ALIGN, _UNSUPPORTED (64 rows of one tensor span 2 GiB or
 * more), _WORKSPACE.  With no sequence or no query it does nothing.
 */
int pamm_attention(const pamm_attention_t *a_host, void *ws, size_t ws_bytes, void *stream);

/* Bytes of workspace pamm_attention_backward needs: <do, o> of every row, a
 * mark for every workgroup, and partial sums of dk and dv where few keys are
 * shared by many queries or the device would not be full. */
size_t pamm_attention_backward_workspace_size(const pamm_attention_t *a_host);

/*
 * Gradients of pamm_attention from dout, the gradient of o, and the saved
 * o and lse.  The probabilities are recomputed from q, k and lse:
 *
 *   P_ij = exp(s_ij - lse_i)      dS_ij = P_ij (<do_i, v_j> - <do_i, o_i>)
 *   dv_j = sum_i P_ij do_i        dq_i = scale sum_j dS_ij k_j
 *                                 dk_j = scale sum_i dS_ij q_i
 *
 * The sums over i run over all query heads that share the key/value head.
 * dq, dk and dv are written whole: rows that see or are seen by nothing, and
 * those past the lengths, become 0.  The written tensors must not overlap
 * each other or any input.  Errors as pamm_attention.
 */
int pamm_attention_backward(const pamm_attention_t *a_host, const pamm_heads_t *dout_host,
                            const pamm_heads_t *dq_host, const pamm_heads_t *dk_host, const pamm_heads_t *dv_host,
                            void *ws, size_t ws_bytes, void *stream);

/* Longest row of the norm calls. */
#define PAMM_MAX_NORM_BYTES 65536

/*
 * h = x + r rounded to dtype (h = x if r is NULL),
 * rstd_i = 1 / sqrt(mean_l h_il^2 + eps),
 * y_il = h_il rstd_i w_l.
 *
 *   x, r  [n x d], leading dimensions ldx, ldr                  (read; r may be NULL)
 *   w     [d] dtype                                             (read)
 *   h     [n x d], leading dimension ldh (written if r is given; may be x or
 *         r itself; ignored without r)
 *   y     [n x d] dtype, leading dimension ldy                  (written; may be NULL)
 *   q     [n x d] 8-bit floats (4 exponent and 3 fraction bits, largest 448,
 *         no infinities), leading dimension ldq in bytes        (written; may be NULL)
 *   qscale [n] fp32: max_l |y_il| / 448, at least 2^-126        (written iff q is)
 *         q_il = y_il / qscale_i as 448 h_il w_l / max_l |h_il w_l|, in which rstd
 *         cancels, rounded to nearest even: exactly that for bf16, whose products fp32 holds
 *   rstd  [n] fp32                                              (written; may be NULL)
 *
 * x, r, h, y 16-byte aligned with leading dimensions multiples of 16 bytes;
 * w 16-byte aligned; q 8-byte aligned with ldq a multiple of 8.  A row holds
 * at most PAMM_MAX_NORM_BYTES (32768 bf16 or 16384 fp32 elements).  What is
 * not finite in a row changes that row alone: a NaN makes all of it NaN, an
 * infinity makes its own place NaN and the others 0.  A row whose sum of
 * squares passes fp32's range has rstd = 0.
 *
 * Errors: PAMM_ERR_NULL (x, w; h with r; qscale with q; neither y nor q),
 * _DTYPE, _SHAPE, _VALUE (eps negative, infinite or NaN), _ALIGN.
 */
int pamm_add_rms_norm(const void *x, int64_t ldx, const void *r, int64_t ldr, const void *w, int64_t n, int64_t d,
                      int dtype, float eps, void *h, int64_t ldh, void *y, int64_t ldy, void *q, int64_t ldq,
                      float *qscale, float *rstd, void *stream);

size_t pamm_add_rms_norm_backward_workspace_size(int64_t n, int64_t d, int dtype);

/*
 * Gradients of pamm_add_rms_norm's y with respect to h and w, from the saved
 * h and rstd, with the gradient dh that reaches h by the residual path added:
 *
 *   g = w dy,  dx_il = dh_il + rstd_i (g_il - xhat_il mean_l(g_il xhat_il)),
 *   dw_l = sum_i dy_il xhat_il,   xhat = h rstd
 *
 * dx is the gradient of x and of r alike.  dy, h [n x d] read, dh may be NULL;
 * dx [n x d] dtype written (may be dy or dh itself); dw [d] fp32 written.
 * Alignment as above; workspace of the size above.
 */
int pamm_add_rms_norm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh, const void *w,
                               const float *rstd, const void *dh, int64_t lddh, int64_t n, int64_t d, int dtype,
                               void *dx, int64_t lddx, float *dw, void *ws, size_t ws_bytes, void *stream);

/* One gradient: rows x cols elements, row i at data + i * ld elements.  A
 * contiguous tensor of any shape is one row.  Any element alignment. */
typedef struct {
    const void *data;   /* read */
    void *out;          /* written; data itself to scale in place */
    int64_t rows, cols, ld, ld_out;
    int32_t dtype, out_dtype;
} pamm_grad_t;

size_t pamm_clip_grad_norm_workspace_size(const pamm_grad_t *grads_host, int64_t count);

/*
 * norm = sqrt(sum of squares of all elements of all gradients), summed in
 * 64 bits and rounded to fp32; coef = max_norm / (norm + eps), at most 1 (and
 * 1 if norm + eps is 0); out = coef * data.  Where coef is 1, gradients scaled in place are not
 * touched.  A NaN norm makes every output NaN; an infinite norm gives coef 0
 * (so infinities become NaN and finite values 0).
 *
 *   grads_host  [count] descriptors, read during the call
 *   max_norm    >= 0; +infinity: the norm alone, nothing is written to out
 *   norm        one fp32 (written)
 *
 * The written ranges must not meet each other or another gradient's data
 * (column ranges of one wider matrix may interleave).
 *
 * Errors: PAMM_ERR_NULL, _SHAPE, _DTYPE, _VALUE (max_norm or eps negative or
 * NaN; in place with another out_dtype or ld), _ALIGN (an address that is not
 * a multiple of its element's size), PAMM_ERR_OVERLAP, _WORKSPACE,
 * _TOO_LARGE (no host memory for the list).
 */
int pamm_clip_grad_norm(const pamm_grad_t *grads_host, int64_t count, float max_norm, float eps, float *norm,
                        void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAMM_BLOCK_H */
