// pamm_block_api.hip -- the extern "C" boundary of the operators around the
// projection (declared in include/pamm_block.h): argument validation,
// workspace carve-up, launches.  Nothing here allocates device memory,
// synchronises, or keeps state.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "pamm_block.h"
#include "pamm_block_checks.hpp"
#include "pamm_block_kernels.hpp"

using namespace pamm_checks;

namespace {

// The backward pass may run its items, tiles of queries and of keys, in one launch.
int backward_sizes(const pamm_attention_t* a) {
    if (int e = attention_sizes(a)) return e;
    const int64_t heads = a->batch * a->heads_kv, rows = a->seq_q * (a->heads / a->heads_kv);
    return heads * ((rows + 127) / 128) + heads * ((a->seq_k + 127) / 128) > kMaxGroups ? PAMM_ERR_SHAPE : PAMM_OK;
}

int attention_check(const pamm_attention_t* a) {
    if (int e = attention_sizes(a)) return e;
    const int64_t B = a->batch, H = a->heads;
    if (int e = heads_check(a->q, B, a->seq_q, H, elem_size(a->dtype))) return e;
    if (int e = heads_check(a->k, B, a->seq_k, a->heads_kv, elem_size(a->dtype))) return e;
    if (int e = heads_check(a->v, B, a->seq_k, a->heads_kv, elem_size(a->dtype))) return e;
    if (int e = heads_check(a->o, B, a->seq_q, H, elem_size(a->dtype))) return e;
    if (B > 0 && a->seq_q > 0 && !a->lse) return PAMM_ERR_NULL;
    if (!aligned(a->lse, 4) || !aligned(a->q_len, 4) || !aligned(a->kv_len, 4)) return PAMM_ERR_ALIGN;
    return PAMM_OK;
}

int splits_of(const pamm_attention_t* a) {
    return pamm::attention_splits(a->batch, a->seq_q, a->seq_k, a->heads_kv, a->heads / a->heads_kv,
                                  a->kv_len != nullptr, num_cus());
}

int dkv_splits_of(const pamm_attention_t* a) {
    return pamm::attention_dkv_splits(a->batch, a->seq_q, a->seq_k, a->heads_kv, a->heads / a->heads_kv, a->dtype,
                                      num_cus());
}

// Workspace of the backward pass: delta, the items' marks, parts of dk and dv.
struct BackwardLayout {
    size_t marks, part_dk, part_dv, total;
    int64_t dq_items;
    int parts;
};
BackwardLayout backward_layout(const pamm_attention_t* a) {
    const int64_t heads = a->batch * a->heads_kv, rows = a->seq_q * (a->heads / a->heads_kv);
    BackwardLayout L;
    L.parts = dkv_splits_of(a);
    L.dq_items = heads * ((rows + 127) / 128);
    const int64_t items = L.dq_items + heads * ((a->seq_k + 127) / 128) * L.parts;
    const size_t part = L.parts > 1 ? up256((size_t)L.parts * (size_t)(heads * a->seq_k * a->head_dim) * sizeof(float)) : 0;
    L.marks = up256((size_t)(a->batch * a->heads * a->seq_q) * sizeof(float));
    L.part_dk = L.marks + up256((size_t)items * 4 * sizeof(int32_t));
    L.part_dv = L.part_dk + part;
    L.total = L.part_dv + part;
    return L;
}

bool rows_ok(int64_t n, int64_t ld, int64_t d) { return ld >= d && ld <= kMaxSpan && n - 1 <= (kMaxSpan - d) / ld; }

// Sizes of the norm calls; their leading dimensions are checked with each matrix.
int norm_sizes(int64_t n, int64_t d, int dtype) {
    if (!dtype_ok(dtype)) return PAMM_ERR_DTYPE;
    if (n < 0 || n > kMaxSize || d < 1 || d > pamm::kMaxNormVectors * per16(dtype))
        return PAMM_ERR_SHAPE;
    return PAMM_OK;
}

int matrix_check(const void* p, int64_t ld, int64_t n, int64_t d, int dtype, bool required) {
    if (!p) return required && n > 0 ? PAMM_ERR_NULL : PAMM_OK;
    if (n == 0) return PAMM_OK;
    if (!rows_ok(n, ld, d)) return PAMM_ERR_SHAPE;
    return aligned(p, 16) && ld % per16(dtype) == 0 ? PAMM_OK : PAMM_ERR_ALIGN;
}

}  // namespace

extern "C" {

size_t pamm_attention_workspace_size(const pamm_attention_t* a) {
    if (attention_sizes(a) != PAMM_OK) return 0;
    const int n = splits_of(a);
    if (n == 1) return 0;
    const size_t rows = (size_t)(a->batch * a->heads * a->seq_q) * (size_t)n;
    return up256(rows * sizeof(float)) + up256(rows * sizeof(float) * (size_t)a->head_dim);
}

int pamm_attention(const pamm_attention_t* a, void* ws, size_t ws_bytes, void* stream) {
    if (int e = attention_check(a)) return e;
    const size_t need = pamm_attention_workspace_size(a);
    if (int e = ws_check(ws, ws_bytes, need)) return e;
    if (a->batch == 0 || a->seq_q == 0) return PAMM_OK;
    pamm::AttnArgs r = attention_args(a);
    // the few-rows kernel's blocks start at the first key that its rows see
    if (r.Sq == 1 && r.G <= pamm::kFewRows) r.hides = false;
    r.nsplit = splits_of(a);
    if (r.nsplit > 1) {
        const size_t rows = (size_t)(a->batch * a->heads * a->seq_q) * (size_t)r.nsplit;
        r.part_lse = reinterpret_cast<float*>(ws);
        r.part_o = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + up256(rows * sizeof(float)));
    }
    return status(pamm::run_attention(r, a->dtype, reinterpret_cast<hipStream_t>(stream)));
}

size_t pamm_attention_backward_workspace_size(const pamm_attention_t* a) {
    return backward_sizes(a) == PAMM_OK ? backward_layout(a).total : 0;
}

int pamm_attention_backward(const pamm_attention_t* a, const pamm_heads_t* dout, const pamm_heads_t* dq,
                            const pamm_heads_t* dk, const pamm_heads_t* dv, void* ws, size_t ws_bytes, void* stream) {
    if (int e = backward_sizes(a)) return e;
    if (int e = attention_check(a)) return e;
    if (!dout || !dq || !dk || !dv) return PAMM_ERR_NULL;
    if (int e = heads_check(*dout, a->batch, a->seq_q, a->heads, elem_size(a->dtype))) return e;
    if (int e = heads_check(*dq, a->batch, a->seq_q, a->heads, elem_size(a->dtype))) return e;
    if (int e = heads_check(*dk, a->batch, a->seq_k, a->heads_kv, elem_size(a->dtype))) return e;
    if (int e = heads_check(*dv, a->batch, a->seq_k, a->heads_kv, elem_size(a->dtype))) return e;
    const size_t need = pamm_attention_backward_workspace_size(a);
    if (int e = ws_check(ws, ws_bytes, need)) return e;
    if (a->batch == 0) return PAMM_OK;
    pamm::AttnArgs r = attention_args(a);
    r.dout = heads_arg(*dout, a, true);
    r.dq = heads_arg(*dq, a, true);
    r.dk = heads_arg(*dk, a, false);
    r.dv = heads_arg(*dv, a, false);
    const BackwardLayout L = backward_layout(a);
    char* at = reinterpret_cast<char*>(ws);
    r.delta = reinterpret_cast<float*>(at);
    r.marks = reinterpret_cast<int32_t*>(at + L.marks);
    r.dq_items = (int)L.dq_items;
    r.nsplit_kv = L.parts;
    r.part_dk = reinterpret_cast<float*>(at + L.part_dk);
    r.part_dv = reinterpret_cast<float*>(at + L.part_dv);
    return status(pamm::run_attention_backward(r, a->dtype, reinterpret_cast<hipStream_t>(stream)));
}

int pamm_add_rms_norm(const void* x, int64_t ldx, const void* r, int64_t ldr, const void* w, int64_t n, int64_t d,
                      int dtype, float eps, void* h, int64_t ldh, void* y, int64_t ldy, void* q, int64_t ldq,
                      float* qscale, float* rstd, void* stream) {
    if (int e = norm_sizes(n, d, dtype)) return e;
    if (!(eps >= 0.0f) || isinf(eps)) return PAMM_ERR_VALUE;
    if (n == 0) return PAMM_OK;
    if (!w || (r && !h) || (q && !qscale) || (!y && !q)) return PAMM_ERR_NULL;
    if (int e = matrix_check(x, ldx, n, d, dtype, true)) return e;
    if (int e = matrix_check(r, ldr, n, d, dtype, false)) return e;
    if (r)
        if (int e = matrix_check(h, ldh, n, d, dtype, true)) return e;
    if (int e = matrix_check(y, ldy, n, d, dtype, false)) return e;
    if (q && !rows_ok(n, ldq, d)) return PAMM_ERR_SHAPE;
    if (!aligned(w, 16) || (q && (!aligned(q, 8) || ldq % 8 != 0)) || !aligned(qscale, 4) || !aligned(rstd, 4))
        return PAMM_ERR_ALIGN;
    const int64_t es = elem_size(dtype);
    pamm::NormArgs a;
    memset(&a, 0, sizeof a);
    a.x = reinterpret_cast<const char*>(x);
    a.r = reinterpret_cast<const char*>(r);
    a.w = reinterpret_cast<const char*>(w);
    a.h = reinterpret_cast<char*>(h);
    a.y = reinterpret_cast<char*>(y);
    a.q = reinterpret_cast<uint8_t*>(q);
    a.qscale = qscale;
    a.rstd = rstd;
    a.ldx = ldx * es;
    a.ldr = r ? ldr * es : 0;  // without its matrix a leading dimension is not checked
    a.ldh = r ? ldh * es : 0;
    a.ldy = y ? ldy * es : 0;
    a.ldq = q ? ldq : 0;
    a.n = n;
    a.d = (int)d;
    a.eps = eps;
    a.num_cus = num_cus();
    return status(pamm::run_add_rms_norm(a, dtype, reinterpret_cast<hipStream_t>(stream)));
}

size_t pamm_add_rms_norm_backward_workspace_size(int64_t n, int64_t d, int dtype) {
    if (norm_sizes(n, d, dtype) != PAMM_OK) return 0;
    return up256((size_t)pamm::norm_backward_blocks(n, d, dtype, num_cus()) * (size_t)d * sizeof(float));
}

int pamm_add_rms_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* w,
                               const float* rstd, const void* dh, int64_t lddh, int64_t n, int64_t d, int dtype,
                               void* dx, int64_t lddx, float* dw, void* ws, size_t ws_bytes, void* stream) {
    if (int e = norm_sizes(n, d, dtype)) return e;
    if (!dw || (n > 0 && (!w || !rstd))) return PAMM_ERR_NULL;
    if (int e = matrix_check(dy, lddy, n, d, dtype, true)) return e;
    if (int e = matrix_check(h, ldh, n, d, dtype, true)) return e;
    if (int e = matrix_check(dh, lddh, n, d, dtype, false)) return e;
    if (int e = matrix_check(dx, lddx, n, d, dtype, true)) return e;
    if (!aligned(w, 16) || !aligned(rstd, 4) || !aligned(dw, 4)) return PAMM_ERR_ALIGN;
    if (int e = ws_check(ws, ws_bytes, pamm_add_rms_norm_backward_workspace_size(n, d, dtype))) return e;
    const int64_t es = elem_size(dtype);
    pamm::NormArgs a;
    memset(&a, 0, sizeof a);
    a.dy = reinterpret_cast<const char*>(dy);
    a.h = reinterpret_cast<char*>(const_cast<void*>(h));
    a.w = reinterpret_cast<const char*>(w);
    a.rstd = const_cast<float*>(rstd);
    a.dh = reinterpret_cast<const char*>(dh);
    a.dx = reinterpret_cast<char*>(dx);
    a.dw = dw;
    a.part = reinterpret_cast<float*>(ws);
    if (n > 0) {  // not checked otherwise, nor used
        a.lddy = lddy * es;
        a.ldh = ldh * es;
        a.lddh = dh ? lddh * es : 0;
        a.lddx = lddx * es;
    }
    a.n = n;
    a.d = (int)d;
    a.num_cus = num_cus();
    return status(pamm::run_add_rms_norm_backward(a, dtype, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// The tensors of a clipping call: empty ones left out, neighbours in memory
// (views of one flat buffer, whose outputs are neighbours too) as one range.
int clip_list(const pamm_grad_t* g, int64_t count, bool write, std::vector<pamm::ClipTensor>& list) {
    for (int64_t i = 0; i < count; ++i) {
        const pamm_grad_t& t = g[i];
        if (!dtype_ok(t.dtype) || (write && !dtype_ok(t.out_dtype))) return PAMM_ERR_DTYPE;
        if (t.rows < 0 || t.cols < 0 || t.rows > kMaxSpan || t.cols > kMaxSpan) return PAMM_ERR_SHAPE;
        if (t.rows == 0 || t.cols == 0) continue;
        if ((t.rows > 1 && (!rows_ok(t.rows, t.ld, t.cols) || (write && !rows_ok(t.rows, t.ld_out, t.cols)))))
            return PAMM_ERR_SHAPE;
        if (!t.data || (write && !t.out)) return PAMM_ERR_NULL;
        if (!aligned(t.data, elem_size(t.dtype)) || (write && !aligned(t.out, elem_size(t.out_dtype))))
            return PAMM_ERR_ALIGN;
        pamm::ClipTensor c;
        c.data = reinterpret_cast<const char*>(t.data);
        c.out = write ? reinterpret_cast<char*>(t.out) : nullptr;
        c.rows = t.rows, c.cols = t.cols, c.ld = t.ld, c.ld_out = t.ld_out;
        c.dtype = t.dtype, c.out_dtype = write ? t.out_dtype : t.dtype;
        if (write && c.out == c.data && (c.dtype != c.out_dtype || (c.rows > 1 && c.ld != c.ld_out)))
            return PAMM_ERR_VALUE;
        if (c.rows > 1 && c.ld == c.cols && (!write || c.ld_out == c.cols)) {
            c.cols *= c.rows;
            c.rows = 1;
        }
        if (!list.empty() && c.rows == 1) {
            pamm::ClipTensor& p = list.back();
            if (p.rows == 1 && p.dtype == c.dtype && p.out_dtype == c.out_dtype &&
                p.data + p.cols * elem_size(p.dtype) == c.data &&
                (!write || p.out + p.cols * elem_size(p.out_dtype) == c.out) && p.cols + c.cols <= kMaxSpan) {
                p.cols += c.cols;
                continue;
            }
        }
        list.push_back(c);
    }
    return PAMM_OK;
}

// Whether a written range meets another tensor's: each element is scaled once.
bool clip_overlap(const pamm_grad_t* g, int64_t count) {
    struct Span {
        uintptr_t begin, end;
        int64_t rows, cols, ld;
        int size;
        bool written;
    };
    std::vector<Span> spans, active;
    spans.reserve(2 * (size_t)count);
    for (int64_t i = 0; i < count; ++i) {
        const pamm_grad_t& t = g[i];
        if (t.rows == 0 || t.cols == 0) continue;
        auto add = [&](const void* p, int64_t ld, int dtype, bool written) {
            const uintptr_t b = reinterpret_cast<uintptr_t>(p);
            const int e = elem_size(dtype);
            spans.push_back({b, b + (uintptr_t)((t.rows > 1 ? (t.rows - 1) * ld : 0) + t.cols) * (uintptr_t)e, t.rows,
                             t.cols, ld, e, written});
        };
        add(t.out, t.ld_out, t.out_dtype, true);
        if (t.out != t.data) add(t.data, t.ld, t.dtype, false);
    }
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
    for (const Span& s : spans) {
        active.erase(std::remove_if(active.begin(), active.end(), [&](const Span& a) { return a.end <= s.begin; }),
                     active.end());
        for (const Span& a : active) {
            if (!a.written && !s.written) continue;
            // columns of one wider matrix interleave without meeting
            const uintptr_t gap = s.begin - a.begin;
            if (a.rows > 1 && s.rows > 1 && a.ld == s.ld && a.size == s.size && gap % (uintptr_t)a.size == 0) {
                const int64_t shift = (int64_t)(gap / (uintptr_t)a.size) % a.ld;
                if (shift >= a.cols && shift + s.cols <= a.ld) continue;
            }
            return true;
        }
        active.push_back(s);
    }
    return false;
}

size_t clip_ws(size_t tensors) {
    const size_t launches = (tensors + pamm::kClipTensors - 1) / pamm::kClipTensors;
    return up256(launches * pamm::kClipBlocks * sizeof(double));
}

}  // namespace

extern "C" {

size_t pamm_clip_grad_norm_workspace_size(const pamm_grad_t* grads, int64_t count) {
    if (count < 0 || count > kMaxSize || (count > 0 && !grads)) return 0;
    // merging neighbours only lowers the count
    return clip_ws(count > 0 ? (size_t)count : 1);
}

int pamm_clip_grad_norm(const pamm_grad_t* grads, int64_t count, float max_norm, float eps, float* norm, void* ws,
                        size_t ws_bytes, void* stream) {
    if (count < 0 || count > kMaxSize) return PAMM_ERR_SHAPE;
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f) || isinf(eps)) return PAMM_ERR_VALUE;
    if (!norm || (count > 0 && !grads)) return PAMM_ERR_NULL;
    if (!aligned(norm, 4)) return PAMM_ERR_ALIGN;
    const bool write = !isinf(max_norm);
    std::vector<pamm::ClipTensor> list;
    try {
        list.reserve((size_t)count);
        if (int e = clip_list(grads, count, write, list)) return e;
        if (write && clip_overlap(grads, count)) return PAMM_ERR_OVERLAP;
    } catch (...) {
        return PAMM_ERR_TOO_LARGE;
    }
    if (int e = ws_check(ws, ws_bytes, pamm_clip_grad_norm_workspace_size(grads, count))) return e;

    const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    double* part = reinterpret_cast<double*>(ws);
    pamm::ClipArgs a;
    bool in_place = true;
    for (const pamm::ClipTensor& t : list) in_place = in_place && t.out == t.data;
    auto fill = [&](size_t first) {
        memset(&a, 0, sizeof a);
        const size_t n = std::min<size_t>(pamm::kClipTensors, list.size() - first);
        for (size_t i = 0; i < n; ++i) {
            a.t[i] = list[first + i];
            a.t[i].first_chunk = a.chunks;
            a.chunks += pamm::clip_chunks(a.t[i]);
        }
        a.count = (int)n;
        a.max_norm = max_norm;
        a.eps = eps;
        a.in_place = in_place;
    };
    int parts = 0;
    for (size_t first = 0; first < list.size(); first += pamm::kClipTensors) {
        fill(first);
        a.parts = (int)std::min<int64_t>(a.chunks, pamm::kClipBlocks);
        a.part = part + parts;
        parts += a.parts;
        const hipError_t e = pamm::run_clip_sum(a, st);
        if (e != hipSuccess) return PAMM_ERR_HIP;
    }
    size_t first = 0;
    do {
        fill(first);
        a.parts = parts;
        a.part = part;
        a.norm = first == 0 ? norm : nullptr;
        const hipError_t e = pamm::run_clip_scale(a, write, st);
        if (e != hipSuccess) return PAMM_ERR_HIP;
        first += pamm::kClipTensors;
    } while (write && first < list.size());
    return PAMM_OK;
}

}  // extern "C"
