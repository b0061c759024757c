// pamm_cache_api.hip -- the extern "C" boundary of the cache in 8 bits (declared
// in include/pamm_cache.h): argument validation, workspace carve-up, launches.
// Nothing here allocates, synchronises, or keeps state.
#include <string.h>

#include "pamm_block_checks.hpp"
#include "pamm_cache.h"
#include "pamm_cache_kernels.hpp"

using namespace pamm_checks;

namespace {

int block_log(int64_t block) { return block == 32 ? 5 : block == 64 ? 6 : block == 128 ? 7 : -1; }

int cache_sizes(const pamm_cache8_t* c) {
    if (!c) return PAMM_ERR_NULL;
    if (!dtype_ok(c->dtype)) return PAMM_ERR_DTYPE;
    if (c->batch < 0 || c->batch > kMaxSize || c->room < 0 || c->room > kMaxSequence || c->heads_kv < 1 ||
        c->heads_kv > kMaxSize || c->head_dim < 1 || c->head_dim > PAMM_MAX_HEAD_DIM)
        return PAMM_ERR_SHAPE;
    if (c->head_dim % 16 != 0) return PAMM_ERR_ALIGN;
    return block_log(c->block) < 0 ? PAMM_ERR_VALUE : PAMM_OK;
}

int scales_check(const pamm_scales_t& t, const pamm_cache8_t* c) {
    const int64_t s[3] = {t.stride_b, t.stride_s, t.stride_h}, n[3] = {c->batch, c->room / c->block, c->heads_kv};
    if (c->batch == 0 || n[1] == 0) return PAMM_OK;
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || (n[i] > 1 && mul(n[i] - 1, s[i]) > kMaxSpan)) return PAMM_ERR_SHAPE;
    if (!t.data) return PAMM_ERR_NULL;
    return aligned(t.data, 4) ? PAMM_OK : PAMM_ERR_ALIGN;
}

int cache_check(const pamm_cache8_t* c) {
    if (int e = cache_sizes(c)) return e;
    for (const pamm_heads_t* t : {&c->k, &c->v})
        if (int e = heads_check(*t, c->batch, c->room, c->heads_kv, 1)) return e;
    for (const pamm_heads_t* t : {&c->k_tail, &c->v_tail})
        if (int e = heads_check(*t, c->batch, c->block, c->heads_kv, elem_size(c->dtype))) return e;
    for (const pamm_scales_t* t : {&c->k_scale, &c->v_scale})
        if (int e = scales_check(*t, c)) return e;
    return PAMM_OK;
}

// Strides in bytes; that of a dimension with one entry may be anything.
pamm::HeadsArg heads_of(const pamm_heads_t& t, int64_t batch, int64_t rows, int64_t heads, int64_t e, int64_t D) {
    return {reinterpret_cast<char*>(t.data), batch > 1 && rows > 0 ? t.stride_b * e : 0,
            batch > 0 && rows > 1 ? t.stride_s * e : D * e, batch > 0 && rows > 0 && heads > 1 ? t.stride_h * e : 0};
}
pamm::ScalesArg scales_of(const pamm_scales_t& t, const pamm_cache8_t* c) {
    const int64_t rows = c->room / c->block;
    return {t.data, c->batch > 1 && rows > 0 ? t.stride_b : 0, c->batch > 0 && rows > 1 ? t.stride_s : 0,
            c->batch > 0 && rows > 0 && c->heads_kv > 1 ? t.stride_h : 0};
}

// The attention problem's sizes, and whether the cache is one for it.
int problem_sizes(const pamm_attention_t* a, const pamm_cache8_t* c) {
    if (int e = attention_sizes(a)) return e;
    if (int e = cache_sizes(c)) return e;
    if (a->dtype != c->dtype) return PAMM_ERR_DTYPE;
    return a->batch == c->batch && a->heads_kv == c->heads_kv && a->head_dim == c->head_dim && a->seq_k <= c->room
               ? PAMM_OK
               : PAMM_ERR_SHAPE;
}

int splits_of(const pamm_attention_t* a) {
    return pamm::attention8_splits(a->batch, a->seq_q, a->seq_k, a->heads_kv, a->heads / a->heads_kv,
                                   a->kv_len != nullptr, num_cus());
}

}  // namespace

extern "C" {

int pamm_cache8_append(const pamm_cache8_t* c, const pamm_heads_t* k, const pamm_heads_t* v, int64_t n,
                       const int32_t* new_len, int32_t* lengths, int32_t advance, void* stream) {
    if (int e = cache_check(c)) return e;
    if (!k || !v) return PAMM_ERR_NULL;
    if (n < 0 || n > kMaxSequence) return PAMM_ERR_SHAPE;
    if (advance != 0 && advance != 1) return PAMM_ERR_VALUE;
    const int es = elem_size(c->dtype);
    for (const pamm_heads_t* t : {k, v})
        if (int e = heads_check(*t, c->batch, n, c->heads_kv, es)) return e;
    if (c->batch > 0 && !lengths) return PAMM_ERR_NULL;
    if (!aligned(new_len, 4) || !aligned(lengths, 4)) return PAMM_ERR_ALIGN;
    if (mul(c->batch, c->heads_kv) > kMaxSize) return PAMM_ERR_SHAPE;
    if (c->batch == 0 || n == 0) return PAMM_OK;
    pamm::AppendArgs a;
    memset(&a, 0, sizeof a);
    const int64_t B = c->batch, H = c->heads_kv, D = c->head_dim;
    const pamm_heads_t *x[2] = {k, v}, *to[2] = {&c->k, &c->v}, *tail[2] = {&c->k_tail, &c->v_tail};
    const pamm_scales_t* scale[2] = {&c->k_scale, &c->v_scale};
    for (int i = 0; i < 2; ++i)
        a.t[i] = {heads_of(*x[i], B, n, H, es, D), heads_of(*tail[i], B, c->block, H, es, D),
                  heads_of(*to[i], B, c->room, H, 1, D), scales_of(*scale[i], c)};
    a.new_len = new_len;
    a.lengths = lengths;
    a.B = (int)B;
    a.n = (int)n;
    a.room = (int)c->room;
    a.Hkv = (int)H;
    a.D = (int)D;
    a.block_log = block_log(c->block);
    a.touched = (int)((n + c->block - 2) / c->block + 1);
    a.advance = advance;
    return status(pamm::run_cache8_append(a, c->dtype, reinterpret_cast<hipStream_t>(stream)));
}

size_t pamm_cache8_attention_workspace_size(const pamm_attention_t* a, const pamm_cache8_t* c) {
    if (problem_sizes(a, c) != PAMM_OK) return 0;
    const int n = splits_of(a);
    if (n == 1) return 0;
    const size_t rows = (size_t)(a->batch * a->heads * a->seq_q) * (size_t)n;
    return up256(rows * sizeof(float)) + up256(rows * sizeof(float) * (size_t)a->head_dim);
}

int pamm_cache8_attention(const pamm_attention_t* a, const pamm_cache8_t* c, void* ws, size_t ws_bytes, void* stream) {
    if (int e = problem_sizes(a, c)) return e;
    if (int e = cache_check(c)) return e;
    const int es = elem_size(a->dtype);
    if (int e = heads_check(a->q, a->batch, a->seq_q, a->heads, es)) return e;
    if (int e = heads_check(a->o, a->batch, a->seq_q, a->heads, es)) return e;
    if (a->batch > 0 && a->seq_q > 0 && !a->lse) return PAMM_ERR_NULL;
    if (!aligned(a->lse, 4) || !aligned(a->q_len, 4) || !aligned(a->kv_len, 4)) return PAMM_ERR_ALIGN;
    if (int e = ws_check(ws, ws_bytes, pamm_cache8_attention_workspace_size(a, c))) return e;
    if (a->batch == 0 || a->seq_q == 0) return PAMM_OK;
    pamm_attention_t p = *a;
    memset(&p.k, 0, sizeof p.k);  // not looked at
    memset(&p.v, 0, sizeof p.v);
    pamm::AttnArgs r = attention_args(&p);
    r.k = heads_of(c->k, c->batch, c->room, c->heads_kv, 1, c->head_dim);
    r.v = heads_of(c->v, c->batch, c->room, c->heads_kv, 1, c->head_dim);
    // one query's kernel leaves out the values before its window
    if (r.Sq == 1 && r.G <= pamm::kFewRows) r.hides = false;
    pamm::Cache8Args e;
    memset(&e, 0, sizeof e);
    e.kt = heads_of(c->k_tail, c->batch, c->block, c->heads_kv, es, c->head_dim);
    e.vt = heads_of(c->v_tail, c->batch, c->block, c->heads_kv, es, c->head_dim);
    e.ks = scales_of(c->k_scale, c);
    e.vs = scales_of(c->v_scale, c);
    e.block_log = block_log(c->block);
    r.nsplit = splits_of(a);
    if (r.nsplit > 1) {
        const size_t rows = (size_t)(a->batch * a->heads * a->seq_q) * (size_t)r.nsplit;
        r.part_lse = reinterpret_cast<float*>(ws);
        r.part_o = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + up256(rows * sizeof(float)));
    }
    return status(pamm::run_attention8(r, e, a->dtype, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
