// pamm_rotary_api.hip -- the extern "C" boundary of the rotation of queries and
// keys and of their norm (declared in include/pamm_positions.h): argument
// validation, workspace, launches.  Nothing here allocates, synchronises, or
// keeps state.
#include <math.h>
#include <string.h>

#include "pamm_block_checks.hpp"
#include "pamm_positions.h"
#include "pamm_rotary_kernels.hpp"

using namespace pamm_checks;

namespace {

// Sizes, scalars and what there is of weights.
int rotary_sizes(const pamm_rotary_t* a) {
    if (!a) return PAMM_ERR_NULL;
    if (!dtype_ok(a->dtype)) return PAMM_ERR_DTYPE;
    if (a->batch < 0 || a->batch > kMaxSize || a->seq < 0 || a->seq > kMaxSize || mul(a->batch, a->seq) > kMaxSize ||
        a->heads_q < 1 || a->heads_q > kMaxSize / 4 || a->heads_k < 0 || a->heads_k > kMaxSize / 4 || a->head_dim < 1 ||
        a->head_dim > PAMM_MAX_HEAD_DIM || a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 2 != 0)
        return PAMM_ERR_SHAPE;
    if (a->head_dim % per16(a->dtype) != 0) return PAMM_ERR_ALIGN;
    for (int32_t flag : {a->interleaved, a->inverse, a->positions_64})
        if (flag != 0 && flag != 1) return PAMM_ERR_VALUE;
    if (!isfinite(a->magnitude) || !(a->eps >= 0.0f) || isinf(a->eps)) return PAMM_ERR_VALUE;
    return PAMM_OK;
}

int both_check(const pamm_rotary_t* a, const pamm_heads_t& q, const pamm_heads_t& k) {
    const int es = elem_size(a->dtype);
    if (int e = heads_check(q, a->batch, a->seq, a->heads_q, es, false)) return e;
    return a->heads_k > 0 ? heads_check(k, a->batch, a->seq, a->heads_k, es, false) : PAMM_OK;
}

int rotary_check(const pamm_rotary_t* a) {
    if (int e = rotary_sizes(a)) return e;
    if (a->q_weight ? (!a->k_weight != (a->heads_k == 0)) : a->k_weight != nullptr) return PAMM_ERR_NULL;
    if (a->q_weight && a->inverse) return PAMM_ERR_VALUE;
    if (!aligned(a->q_weight, 16) || !aligned(a->k_weight, 16)) return PAMM_ERR_ALIGN;
    if (a->batch == 0 || a->seq == 0) return PAMM_OK;
    if (a->rot_dim > 0 && !a->inv_freq) return PAMM_ERR_NULL;
    if (!aligned(a->inv_freq, 8) || !aligned(a->positions, a->positions_64 ? 8 : 4) || !aligned(a->offset, 4))
        return PAMM_ERR_ALIGN;
    if (a->positions)
        if (a->position_stride_b < 0 || a->position_stride_s < 0 || mul(a->batch - 1, a->position_stride_b) > kMaxSpan ||
            mul(a->seq - 1, a->position_stride_s) > kMaxSpan)
            return PAMM_ERR_SHAPE;
    if (int e = both_check(a, a->q, a->k)) return e;
    return both_check(a, a->q_out, a->k_out);
}

// Strides in bytes; that of a dimension with one entry may be anything, as may all without a token.
pamm::HeadsArg heads_arg(const pamm_rotary_t* a, const pamm_heads_t& t, int64_t heads) {
    const int64_t e = a->batch > 0 && a->seq > 0 ? elem_size(a->dtype) : 0;
    return {reinterpret_cast<char*>(t.data), e && a->batch > 1 ? t.stride_b * e : 0, e && a->seq > 1 ? t.stride_s * e : 0,
            e && heads > 1 ? t.stride_h * e : 0};
}

// What the workspace's size goes by: sizes and the layout alone.
pamm::RotaryArgs sizes_arg(const pamm_rotary_t* a, bool backward, int& blocks) {
    pamm::RotaryArgs r;
    memset(&r, 0, sizeof r);
    r.tokens = a->batch * a->seq;
    r.S = a->seq > 0 ? (int)a->seq : 1;
    r.Hq = (int)a->heads_q;
    r.Hk = (int)a->heads_k;
    r.D = (int)a->head_dim;
    r.R2 = (int)(a->rot_dim / 2);
    r.interleaved = a->interleaved;
    r.num_cus = num_cus();
    blocks = pamm::rotary_shape(r, a->dtype, a->q_weight != nullptr, backward);
    return r;
}

pamm::RotaryArgs rotary_args(const pamm_rotary_t* a, bool backward, int& blocks) {
    pamm::RotaryArgs r = sizes_arg(a, backward, blocks);
    r.q = heads_arg(a, a->q, a->heads_q);
    r.qo = heads_arg(a, a->q_out, a->heads_q);
    if (a->heads_k > 0) {
        r.k = heads_arg(a, a->k, a->heads_k);
        r.ko = heads_arg(a, a->k_out, a->heads_k);
    }
    r.inv_freq = a->inv_freq;
    r.positions = a->positions;
    r.psb = a->batch > 1 ? a->position_stride_b : 0;
    r.pss = a->seq > 1 ? a->position_stride_s : 0;
    r.offset = a->offset;
    r.wq = reinterpret_cast<const char*>(a->q_weight);
    r.wk = reinterpret_cast<const char*>(a->k_weight);
    r.positions_64 = a->positions_64;
    r.inverse = a->inverse;
    r.magnitude = a->magnitude;
    r.eps = a->eps;
    return r;
}

}  // namespace

extern "C" {

int pamm_rotary(const pamm_rotary_t* a, void* stream) {
    if (int e = rotary_check(a)) return e;
    if (a->batch == 0 || a->seq == 0) return PAMM_OK;
    int blocks;
    const pamm::RotaryArgs r = rotary_args(a, false, blocks);
    return status(pamm::run_rotary(r, blocks, a->dtype, reinterpret_cast<hipStream_t>(stream)));
}

size_t pamm_rotary_backward_workspace_size(const pamm_rotary_t* a) {
    if (rotary_sizes(a) != PAMM_OK) return 0;
    int blocks;
    const pamm::RotaryArgs r = sizes_arg(a, true, blocks);
    return up256((size_t)blocks * (size_t)r.D * sizeof(float));
}

int pamm_rotary_backward(const pamm_rotary_t* a, const pamm_heads_t* dq, const pamm_heads_t* dk, float* dwq,
                         float* dwk, void* ws, size_t ws_bytes, void* stream) {
    if (int e = rotary_check(a)) return e;
    if (!a->q_weight || !dq || !dwq || (a->heads_k > 0 && (!dk || !dwk))) return PAMM_ERR_NULL;
    if (int e = both_check(a, *dq, a->heads_k > 0 ? *dk : *dq)) return e;
    if (!aligned(dwq, 4) || !aligned(dwk, 4)) return PAMM_ERR_ALIGN;
    if (int e = ws_check(ws, ws_bytes, pamm_rotary_backward_workspace_size(a))) return e;
    int blocks;
    pamm::RotaryArgs r = rotary_args(a, true, blocks);
    r.dq = heads_arg(a, *dq, a->heads_q);
    if (a->heads_k > 0) r.dk = heads_arg(a, *dk, a->heads_k);
    r.part = reinterpret_cast<float*>(ws);
    r.dwq = dwq;
    r.dwk = a->heads_k > 0 ? dwk : nullptr;
    return status(pamm::run_rotary_backward(r, blocks, a->dtype, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
