/*
 * pamm_cache.h -- C ABI of a cache of keys and values in 8 bits, with a scale
 * for each block of tokens and head, and of the attention over it.
 * Conventions, tensors and errors as in pamm_block.h.
 */
#ifndef PAMM_CACHE_H
#define PAMM_CACHE_H

#include "pamm_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Scales: that of block i of sequence b and head h lies at data + b * stride_b
 * + i * stride_s + h * stride_h (elements, >= 0). */
typedef struct {
    float *data;
    int64_t stride_b, stride_s, stride_h;
} pamm_scales_t;

/*
 * Keys and values of `batch` sequences.  Of a sequence with L tokens the first
 * floor(L / block) * block are held in 8 bits (4 exponent and 3 fraction bits,
 * largest 448), whole blocks at a time: token j of head h as
 *
 *   value = k[b, j, h] * k_scale[b, j / block, h],
 *   most  = max |x| over the block's finite elements, at least 448 * 2^-126,
 *   scale = most / 448 rounded to 32 bits,
 *   k     = 448 x / most rounded to nearest even; NaN where x is not finite.
 *
 * k is a rounding of that quotient, not of x over the rounded scale, which may lie on the other side of a tie.  For
 * bf16 it is the nearest, ties to even; for fp32, where the quotient is within 4 * 2^-24 of it of a tie, either neighbour.
 *
 * The others, fewer than a block, wait in their own type in row j % block of
 * the tail.  So what a cache holds depends on its tokens alone, not on the calls
 * that brought them, and nothing is rounded twice.
 */
typedef struct {
    int32_t dtype;            /* of the tails and of what is appended */
    int64_t batch, room;      /* rows of k and v: tokens a sequence can have */
    int64_t heads_kv;
    int64_t head_dim;         /* a multiple of 16, at most PAMM_MAX_HEAD_DIM */
    int64_t block;            /* 32, 64 or 128 */
    pamm_heads_t k, v;        /* [batch x room x heads_kv x head_dim] of 8 bits, strides in bytes */
    pamm_scales_t k_scale, v_scale;   /* [batch x room / block (rounded down) x heads_kv] */
    pamm_heads_t k_tail, v_tail;      /* [batch x block x heads_kv x head_dim] of dtype */
} pamm_cache8_t;

/*
 * Appends k and v [batch x n x heads_kv x head_dim] of dtype behind the
 * lengths[b] tokens of each sequence: all n, or new_len[b] of them (clamped to
 * [0, n]).  Blocks that become whole go to 8 bits, with what waited of them in
 * the tail; the tokens behind them to the tail.  Nothing else is written: tokens
 * past the room are dropped, rows behind the last token are left as they were.
 * lengths [batch] is clamped to [0, room]; with advance it becomes the new
 * lengths (at most room), else it is left.
 *
 * No written tensor may meet another tensor of the call, or itself.  Errors: PAMM_ERR_NULL, _DTYPE, _SHAPE, _ALIGN
 * (head_dim, addresses or strides off 16 bytes), _VALUE (block, advance), _UNSUPPORTED (64 rows span 2 GiB or more).
 */
int pamm_cache8_append(const pamm_cache8_t *cache_host, const pamm_heads_t *k_host, const pamm_heads_t *v_host,
                       int64_t n, const int32_t *new_len, int32_t *lengths, int32_t advance, void *stream);

/* Bytes of workspace pamm_cache8_attention needs, as for pamm_attention. */
size_t pamm_cache8_attention_workspace_size(const pamm_attention_t *a_host, const pamm_cache8_t *cache_host);

/*
 * pamm_attention over the cache: a_host's k and v are not looked at, its seq_k
 * is the cache's room at most (keys past it are not read), kv_len the lengths
 * (NULL: seq_k).  The lengths have to be those of the cache: the tail holds the tokens behind its last whole
 * block, so a length may be lowered (to take the last tokens back) as far as the end of that block, but a
 * prefix that ends before it cannot be looked at.  Scores are formed of exact 8-bit values and scaled in 32 bits; bf16:
 * each probability times the values' scale is rounded once, to bf16 (where up to 32 query rows share a key/value
 * head, to two bf16 parts).
 * Scales have to be positive, normal numbers.  What a mask hides does not come through, not even a NaN.
 * Errors as pamm_attention; _SHAPE, _DTYPE where the two do not fit each other.
 */
int pamm_cache8_attention(const pamm_attention_t *a_host, const pamm_cache8_t *cache_host, void *ws, size_t ws_bytes,
                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAMM_CACHE_H */
