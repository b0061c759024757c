// Drives the host side of include/pamm_block.h (validation, workspace layout,
// the lists of the clipping call) with launchers that look at their arguments
// instead of launching, under AddressSanitizer and UBSan.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <vector>

#include "pamm_block.h"
#include "pamm_block_kernels.hpp"

static int launches, parts_sum;
static long long elements;
#define CHECK(x) do { if (!(x)) { printf("%s:%d: %s\n", __FILE__, __LINE__, #x); exit(1); } } while (0)

namespace pamm {
int attention_splits(int64_t, int64_t Sq, int64_t, int64_t, int64_t G, bool, int) { return Sq * G <= kFewRows ? kMaxSplits : 1; }
int attention_dkv_splits(int64_t, int64_t, int64_t, int64_t, int64_t, int, int) { return 8; }
hipError_t run_attention(const AttnArgs& a, int, hipStream_t) {
    ++launches;
    CHECK(a.G * a.Hkv == a.H && (a.nsplit == 1 || (a.part_o && a.part_lse)));
    return hipSuccess;
}
hipError_t run_attention_backward(const AttnArgs& a, int, hipStream_t) {
    ++launches;
    CHECK((a.Sq == 0 && a.Sk == 0) || (a.delta && a.marks && a.part_dk && a.part_dv));
    CHECK(a.window < (a.Sk ? a.Sk : 1));
    return hipSuccess;
}
hipError_t run_add_rms_norm(const NormArgs& a, int, hipStream_t) {
    ++launches;
    CHECK(a.n > 0 && a.d > 0);
    return hipSuccess;
}
int norm_backward_blocks(int64_t n, int64_t, int, int num_cus) { return (int)(n < num_cus ? n : num_cus); }
hipError_t run_add_rms_norm_backward(const NormArgs&, int, hipStream_t) { ++launches; return hipSuccess; }
int64_t clip_chunks(const ClipTensor& t) { return (t.rows * t.cols + 16383) / 16384; }
hipError_t run_clip_sum(const ClipArgs& a, hipStream_t) {
    ++launches;
    CHECK(a.count > 0 && a.count <= kClipTensors && a.parts <= kClipBlocks);
    for (int i = 0; i < a.count; ++i) elements += a.t[i].rows * a.t[i].cols;
    for (int i = 0; i < a.parts; ++i) a.part[i] = 1.0;  // inside the workspace
    parts_sum += a.parts;
    return hipSuccess;
}
hipError_t run_clip_scale(const ClipArgs& a, bool, hipStream_t) {
    ++launches;
    CHECK(a.parts == parts_sum);
    return hipSuccess;
}
}  // namespace pamm

static char* memory() {
    static char* p = (char*)aligned_alloc(256, 1 << 20);
    return p;
}

static pamm_heads_t heads(int64_t S, int64_t H, int64_t D) { return {memory(), S * H * D, H * D, D}; }

static pamm_attention_t problem(int64_t B, int64_t Sq, int64_t Sk, int64_t H, int64_t Hkv, int64_t D) {
    pamm_attention_t a;
    memset(&a, 0, sizeof a);
    a.dtype = PAMM_BF16, a.causal = 1, a.batch = B, a.seq_q = Sq, a.seq_k = Sk, a.heads = H, a.heads_kv = Hkv;
    a.head_dim = D, a.scale = 0.125f;
    a.q = heads(Sq, H, D), a.k = heads(Sk, Hkv, D), a.v = a.k, a.o = a.q, a.lse = (float*)memory();
    return a;
}

static int forward(const pamm_attention_t& a) {
    size_t n = pamm_attention_workspace_size(&a);
    void* ws = n && n < (1u << 28) ? aligned_alloc(256, n) : nullptr;
    const int r = pamm_attention(&a, ws, ws ? n : 0, nullptr);
    free(ws);
    return r;
}

static int backward(const pamm_attention_t& a) {
    size_t n = pamm_attention_backward_workspace_size(&a);
    void* ws = n && n < (1u << 28) ? aligned_alloc(256, n) : nullptr;
    const int r = pamm_attention_backward(&a, &a.q, &a.q, &a.k, &a.k, ws, ws ? n : 0, nullptr);
    free(ws);
    return r;
}

static void attention() {
    const int64_t extremes[] = {INT64_MIN, -1, 0, 1, 7, 128, 2147483647LL, 1LL << 30, 1LL << 40, INT64_MAX};
    pamm_attention_t good = problem(2, 5, 9, 4, 2, 64);
    CHECK(forward(good) == PAMM_OK && backward(good) == PAMM_OK && launches == 2);
    CHECK(forward(problem(0, 5, 9, 4, 2, 64)) == PAMM_OK && forward(problem(2, 0, 9, 4, 2, 64)) == PAMM_OK);
    CHECK(pamm_attention(nullptr, nullptr, 0, nullptr) == PAMM_ERR_NULL);
    CHECK(pamm_attention_workspace_size(nullptr) == 0 && pamm_attention_backward_workspace_size(nullptr) == 0);
    CHECK(pamm_attention_backward(&good, nullptr, &good.q, &good.k, &good.k, nullptr, 0, nullptr) == PAMM_ERR_NULL);
    CHECK(pamm_attention_backward(&good, &good.q, &good.q, &good.k, &good.k, nullptr, 0, nullptr) == PAMM_ERR_WORKSPACE);
    int64_t pamm_attention_t::*sizes[] = {&pamm_attention_t::batch, &pamm_attention_t::seq_q, &pamm_attention_t::seq_k,
                                          &pamm_attention_t::heads, &pamm_attention_t::heads_kv,
                                          &pamm_attention_t::head_dim, &pamm_attention_t::window};
    // every size, then every pair of sizes, at its extremes: an error or a launch, nothing else
    for (auto x : sizes)
        for (auto y : sizes)
            for (int64_t v : extremes)
                for (int64_t w : extremes) {
                    pamm_attention_t a = good;
                    a.*x = v, a.*y = w;
                    const int f = forward(a), b = backward(a);
                    CHECK(f >= 0 && f <= PAMM_ERR_OVERLAP && b >= 0 && b <= PAMM_ERR_OVERLAP);
                }
    for (int64_t v : extremes)
        for (int64_t pamm_heads_t::*s : {&pamm_heads_t::stride_b, &pamm_heads_t::stride_s, &pamm_heads_t::stride_h}) {
            pamm_attention_t a = good;
            a.k.*s = v;
            CHECK(forward(a) >= 0 && (v >= 0 || forward(a) == PAMM_ERR_SHAPE));
        }
    // strides of dimensions with one entry mean nothing
    for (int64_t v : extremes) {
        pamm_attention_t a = problem(1, 1, 1, 1, 1, 64);
        a.q.stride_b = a.q.stride_s = a.q.stride_h = a.k.stride_b = a.k.stride_s = a.k.stride_h = v;
        CHECK(v < 0 || (forward(a) == PAMM_OK && backward(a) == PAMM_OK));
    }
    pamm_attention_t a = good;
    a.scale = NAN;
    CHECK(forward(a) == PAMM_ERR_VALUE);
    a = good, a.causal = 2;
    CHECK(forward(a) == PAMM_ERR_VALUE);
    a = good, a.dtype = 9;
    CHECK(forward(a) == PAMM_ERR_DTYPE);
    a = good, a.v.data = memory() + 2;
    CHECK(forward(a) == PAMM_ERR_ALIGN);
    a = good, a.lse = nullptr;
    CHECK(forward(a) == PAMM_ERR_NULL);
}

static void norm() {
    char* m = memory();
    for (int64_t n : {-1L, 0L, 1L, 3L, 2147483647L, 1L << 40})
        for (int64_t d : {-8L, 0L, 1L, 8L, 17L, 32768L, 32776L, INT64_MAX})
            for (int64_t ld : {INT64_MIN, 0L, 8L, 32L, 32768L, 1L << 40, INT64_MAX}) {
                CHECK(pamm_add_rms_norm(m, ld, m, ld, m, n, d, PAMM_BF16, 1e-6f, m, ld, m, ld, nullptr, 0, nullptr,
                                        (float*)m, nullptr) >= 0);
                CHECK(pamm_add_rms_norm_backward(m, ld, m, ld, m, (float*)m, m, ld, n, d, PAMM_F32, m, ld, (float*)m,
                                                 m, 1 << 20, nullptr) >= 0);
                pamm_add_rms_norm_backward_workspace_size(n, d, PAMM_BF16);
            }
}

static int clip(const std::vector<pamm_grad_t>& g, float limit) {
    const size_t n = pamm_clip_grad_norm_workspace_size(g.data(), (int64_t)g.size());
    char* ws = (char*)aligned_alloc(256, n ? n : 256);
    float out;
    elements = parts_sum = 0;
    const int r = pamm_clip_grad_norm(g.data(), (int64_t)g.size(), limit, 1e-6f, &out, ws, n, nullptr);
    free(ws);
    return r;
}

static void clipping() {
    char* m = memory();
    auto dense = [&](int64_t at, int64_t n, int dt = PAMM_BF16) {
        return pamm_grad_t{m + at, m + at, 1, n, n, n, dt, dt};
    };
    auto rows = [&](int64_t at, int64_t r, int64_t c, int64_t ld) {
        return pamm_grad_t{m + at, m + at, r, c, ld, ld, PAMM_BF16, PAMM_BF16};
    };
    CHECK(clip({}, 1.0f) == PAMM_OK);
    std::vector<pamm_grad_t> many;
    for (int i = 0; i < 400; ++i) many.push_back(dense(2048 * i, 1000 + i % 20));
    CHECK(clip(many, 1.0f) == PAMM_OK && elements == 400 * 1000 + 20 * 190);
    many.clear();
    for (int i = 0; i < 130; ++i) many.push_back(dense(2000 * i, 1000));  // neighbours: one range
    CHECK(clip(many, INFINITY) == PAMM_OK && elements == 130000);
    CHECK(clip({dense(0, 100), dense(199, 10, PAMM_BF16)}, 1.0f) == PAMM_ERR_ALIGN);
    CHECK(clip({dense(0, 100), dense(198, 10)}, 1.0f) == PAMM_ERR_OVERLAP);
    CHECK(clip({dense(0, 100), dense(198, 10)}, INFINITY) == PAMM_OK);
    CHECK(clip({rows(0, 10, 30, 100), rows(60, 10, 70, 100)}, 1.0f) == PAMM_OK);
    CHECK(clip({rows(0, 10, 31, 100), rows(60, 10, 70, 100)}, 1.0f) == PAMM_ERR_OVERLAP);
    CHECK(clip({rows(0, 0, 30, 100), rows(0, 10, 0, 100), dense(0, 5)}, 1.0f) == PAMM_OK && elements == 5);
    for (int64_t v : {INT64_MIN, -1L, 0L, 1L, 1L << 39, 1L << 41, INT64_MAX})
        for (int64_t w : {INT64_MIN, 0L, 3L, 1L << 40, INT64_MAX}) {
            CHECK(clip({rows(0, v, w, 64)}, INFINITY) >= 0);
            CHECK(clip({rows(0, 3, v, w)}, 1.0f) >= 0);
        }
    CHECK(clip({dense(0, 9)}, NAN) == PAMM_ERR_VALUE && clip({dense(0, 9)}, -1.0f) == PAMM_ERR_VALUE);
    CHECK(clip({dense(0, 9, 5)}, 1.0f) == PAMM_ERR_DTYPE);
    float x;
    CHECK(pamm_clip_grad_norm(nullptr, 3, 1.0f, 0.0f, &x, m, 1 << 20, nullptr) == PAMM_ERR_NULL);
    CHECK(pamm_clip_grad_norm(nullptr, -3, 1.0f, 0.0f, &x, m, 1 << 20, nullptr) == PAMM_ERR_SHAPE);
}

int main() {
    attention();
    norm();
    clipping();
    printf("block ABI sanitizer driver ok, %d launches\n", launches);
    return 0;
}
