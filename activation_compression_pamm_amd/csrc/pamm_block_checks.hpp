// pamm_block_checks.hpp -- argument checks shared by the C entry points of the
// operators around the projection (host code only).
#pragma once
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "pamm_block.h"
#include "pamm_block_kernels.hpp"

namespace pamm_checks {

constexpr int64_t kMaxSize = 2147483647LL;
constexpr int64_t kMaxSequence = ((int64_t)1 << 30) - 512;  // positions and their sums fit 32 bits
// A grid holds less than 2^32 threads, a workgroup 256.  Cutting an axis into parts is left out
// of the counts below: it is done up to 16 workgroups a unit, for which room is kept.
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 8192;
constexpr int64_t kMaxSpan = (int64_t)1 << 40;  // elements; far beyond any device's memory

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int elem_size(int dtype) { return dtype == PAMM_BF16 ? 2 : 4; }
inline int per16(int dtype) { return 16 / elem_size(dtype); }
inline bool dtype_ok(int dtype) { return dtype == PAMM_F32 || dtype == PAMM_BF16; }
inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

inline int num_cus() {
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 256;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) return 256;
    return cus;
}

// a * b, or a number beyond every limit if that overflows (a, b >= 0)
inline int64_t mul(int64_t a, int64_t b) {
    int64_t r;
    return __builtin_mul_overflow(a, b, &r) ? INT64_MAX : r;
}

// A tensor's pointer and strides.  `tiles`: kernels address 64 of its rows with 32-bit offsets.
inline int heads_check(const pamm_heads_t& t, int64_t batch, int64_t seq, int64_t heads, int elem, bool tiles = true) {
    if (batch == 0 || seq == 0) return PAMM_OK;
    const int64_t s[3] = {t.stride_b, t.stride_s, t.stride_h}, n[3] = {batch, seq, heads};
    int64_t span = PAMM_MAX_HEAD_DIM;
    for (int i = 0; i < 3; ++i) {
        if (s[i] < 0) return PAMM_ERR_SHAPE;
        if (n[i] > 1) span = std::max<int64_t>(span, mul(n[i] - 1, s[i]));
        if (span > kMaxSpan) return PAMM_ERR_SHAPE;
    }
    if (!t.data) return PAMM_ERR_NULL;
    if (!aligned(t.data, 16)) return PAMM_ERR_ALIGN;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && s[i] % (16 / elem) != 0) return PAMM_ERR_ALIGN;
    if (tiles && seq > 1 && mul(t.stride_s, 64 * elem) >= (int64_t)1 << 31) return PAMM_ERR_UNSUPPORTED;
    return PAMM_OK;
}

// Sizes and scalars of an attention problem, without its pointers.
inline int attention_sizes(const pamm_attention_t* a) {
    if (!a) return PAMM_ERR_NULL;
    if (!dtype_ok(a->dtype)) return PAMM_ERR_DTYPE;
    if (a->batch < 0 || a->batch > kMaxSize || a->seq_q < 0 || a->seq_q > kMaxSequence || a->seq_k < 0 ||
        a->seq_k > kMaxSequence || a->heads < 1 || a->heads > kMaxSize || a->heads_kv < 1 || a->heads_kv > a->heads ||
        a->heads % a->heads_kv != 0 || a->head_dim < 1 || a->head_dim > PAMM_MAX_HEAD_DIM)
        return PAMM_ERR_SHAPE;
    if (a->head_dim % per16(a->dtype) != 0) return PAMM_ERR_ALIGN;
    if ((a->causal != 0 && a->causal != 1) || !isfinite(a->scale) || a->window < 0 || (a->window > 0 && !a->causal))
        return PAMM_ERR_VALUE;
    // rows of one key/value head, elements of lse, workgroups of either kernel
    const int64_t rows = mul(a->seq_q, a->heads / a->heads_kv);
    if (rows > kMaxSequence || mul(mul(a->batch, a->heads), a->seq_q) > kMaxSpan) return PAMM_ERR_SHAPE;
    const int64_t heads = mul(a->batch, a->heads_kv);
    if (mul(heads, 64) > kMaxSize || mul(heads, (rows + 127) / 128) > kMaxGroups ||
        mul(heads, (a->seq_k + 127) / 128) > kMaxSize / 64 || mul(heads, a->seq_k) > 4 * kMaxSize ||
        mul(mul(a->batch, a->heads), a->seq_q) > 4 * kMaxSize)
        return PAMM_ERR_SHAPE;
    return PAMM_OK;
}

// Strides in bytes.  That of a dimension with one entry may be anything (it is
// not checked); kernels form addresses past the last row, which bounds turn
// into zeros, so rows get a distance of their own length.
inline pamm::HeadsArg heads_arg(const pamm_heads_t& t, const pamm_attention_t* a, bool query) {
    const int64_t e = elem_size(a->dtype), seq = query ? a->seq_q : a->seq_k, heads = query ? a->heads : a->heads_kv;
    return {reinterpret_cast<char*>(t.data), a->batch > 1 && seq > 0 ? t.stride_b * e : 0,
            a->batch > 0 && seq > 1 ? t.stride_s * e : a->head_dim * e,
            a->batch > 0 && seq > 0 && heads > 1 ? t.stride_h * e : 0};
}

inline pamm::AttnArgs attention_args(const pamm_attention_t* a) {
    pamm::AttnArgs r;
    memset(&r, 0, sizeof r);
    r.q = heads_arg(a->q, a, true);
    r.k = heads_arg(a->k, a, false);
    r.v = heads_arg(a->v, a, false);
    r.o = heads_arg(a->o, a, true);
    r.lse = a->lse;
    r.q_len = a->q_len;
    r.kv_len = a->kv_len;
    r.B = (int)a->batch;
    r.Sq = (int)a->seq_q;
    r.Sk = (int)a->seq_k;
    r.H = (int)a->heads;
    r.Hkv = (int)a->heads_kv;
    r.G = (int)(a->heads / a->heads_kv);
    r.D = (int)a->head_dim;
    r.causal = a->causal;
    r.window = a->window >= a->seq_k ? 0 : (int)a->window;  // a window as long as the keys hides none
    // without a causal mask all queries see the same keys; one query alone sees the last ones, from
    // somewhere inside a block if there is a window
    r.hides = r.causal && (r.Sq > 1 || r.window > 0);
    r.scale = a->scale;
    r.num_cus = num_cus();
    r.nsplit = r.nsplit_kv = 1;
    return r;
}

inline int ws_check(const void* ws, size_t ws_bytes, size_t need) {
    if (need == 0) return PAMM_OK;
    if (!ws || ws_bytes < need) return PAMM_ERR_WORKSPACE;
    return aligned(ws, 256) ? PAMM_OK : PAMM_ERR_ALIGN;
}

inline int status(hipError_t e) { return e == hipSuccess ? PAMM_OK : PAMM_ERR_HIP; }

}  // namespace pamm_checks
