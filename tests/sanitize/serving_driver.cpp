// Drives the host side of include/pamm_positions.h and include/pamm_cache.h
// (validation, workspace layout) with launchers that look at their arguments
// instead of launching, under AddressSanitizer and UBSan.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "pamm_cache.h"
#include "pamm_cache_kernels.hpp"
#include "pamm_positions.h"
#include "pamm_rotary_kernels.hpp"

static int launches;
#define CHECK(x) do { if (!(x)) { printf("%s:%d: %s\n", __FILE__, __LINE__, #x); exit(1); } } while (0)

namespace pamm {
int attention8_splits(int64_t, int64_t Sq, int64_t, int64_t, int64_t G, bool, int) { return Sq * G <= kFewRows ? kMaxSplits : 1; }
hipError_t run_attention8(const AttnArgs& a, const Cache8Args& c, int, hipStream_t) {
    ++launches;
    CHECK(a.G * a.Hkv == a.H && (a.nsplit == 1 || (a.part_o && a.part_lse)));
    CHECK(c.block_log >= 5 && c.block_log <= 7);
    return hipSuccess;
}
hipError_t run_cache8_append(const AppendArgs& a, int, hipStream_t) {
    ++launches;
    CHECK(a.B > 0 && a.n > 0 && (int64_t)a.touched << a.block_log >= a.n && a.lengths);
    return hipSuccess;
}
int rotary_shape(RotaryArgs& a, int, bool, bool) { return (int)(a.tokens < 512 ? a.tokens : 512); }
hipError_t run_rotary(const RotaryArgs& a, int blocks, int, hipStream_t) {
    ++launches;
    CHECK(a.tokens > 0 && blocks > 0 && a.S > 0 && 2 * a.R2 <= a.D);
    return hipSuccess;
}
hipError_t run_rotary_backward(const RotaryArgs& a, int blocks, int, hipStream_t) {
    ++launches;
    CHECK(a.wq && a.dwq && (blocks == 0 || a.part));
    for (int i = 0; i < blocks * a.D; ++i) a.part[i] = 1.0f;  // inside the workspace
    return hipSuccess;
}
}  // namespace pamm

static const int64_t kExtremes[] = {INT64_MIN, -1, 0, 1, 7, 16, 128, 2147483647LL, 1LL << 30, 1LL << 40, INT64_MAX};

static char* memory() {
    static char* p = (char*)aligned_alloc(256, 1 << 20);
    return p;
}
static pamm_heads_t heads(int64_t S, int64_t H, int64_t D) { return {memory(), S * H * D, H * D, D}; }
static bool known(int status) { return status >= 0 && status <= PAMM_ERR_OVERLAP; }

static pamm_rotary_t rotation() {
    pamm_rotary_t a;
    memset(&a, 0, sizeof a);
    a.dtype = PAMM_BF16, a.batch = 2, a.seq = 5, a.heads_q = 4, a.heads_k = 2, a.head_dim = 64, a.rot_dim = 32;
    a.magnitude = 1.0f, a.eps = 1e-6f;
    a.inv_freq = (double*)memory(), a.positions = memory(), a.offset = (int32_t*)memory();
    a.position_stride_b = 5, a.position_stride_s = 1;
    a.q_weight = a.k_weight = memory();
    a.q = a.q_out = heads(5, 4, 64), a.k = a.k_out = heads(5, 2, 64);
    return a;
}

static int turn(const pamm_rotary_t& a) {
    const int f = pamm_rotary(&a, nullptr);
    const size_t n = pamm_rotary_backward_workspace_size(&a);
    void* ws = n && n < (1u << 28) ? aligned_alloc(256, n) : nullptr;
    const int b = pamm_rotary_backward(&a, &a.q, &a.k, (float*)memory(), (float*)memory(), ws, ws ? n : 0, nullptr);
    free(ws);
    CHECK(known(f) && known(b));
    CHECK(f == PAMM_OK || b != PAMM_OK);
    return f;
}

static void positions() {
    CHECK(turn(rotation()) == PAMM_OK && launches == 2);
    int64_t pamm_rotary_t::*sizes[] = {&pamm_rotary_t::batch, &pamm_rotary_t::seq, &pamm_rotary_t::heads_q,
                                       &pamm_rotary_t::heads_k, &pamm_rotary_t::head_dim, &pamm_rotary_t::rot_dim,
                                       &pamm_rotary_t::position_stride_b, &pamm_rotary_t::position_stride_s};
    for (auto x : sizes)
        for (auto y : sizes)
            for (int64_t v : kExtremes)
                for (int64_t w : kExtremes) {
                    pamm_rotary_t a = rotation();
                    a.*x = v, a.*y = w;
                    turn(a);
                }
    for (int64_t v : kExtremes)
        for (pamm_heads_t pamm_rotary_t::*t : {&pamm_rotary_t::q, &pamm_rotary_t::k, &pamm_rotary_t::q_out})
            for (int64_t pamm_heads_t::*s : {&pamm_heads_t::stride_b, &pamm_heads_t::stride_s, &pamm_heads_t::stride_h}) {
                pamm_rotary_t a = rotation();
                (a.*t).*s = v;
                CHECK(v >= 0 || turn(a) == PAMM_ERR_SHAPE);
                turn(a);
            }
    pamm_rotary_t a = rotation();
    a.q_weight = a.k_weight = nullptr;
    CHECK(pamm_rotary(&a, nullptr) == PAMM_OK);
    a.inverse = 1, a.rot_dim = 0, a.inv_freq = nullptr;
    CHECK(pamm_rotary(&a, nullptr) == PAMM_OK);
    for (int64_t v : kExtremes) {  // without a token, strides mean nothing
        a = rotation(), a.batch = 0;
        a.q = a.k = a.q_out = a.k_out = {memory(), v, v, v};
        CHECK(turn(a) == PAMM_OK);
        a.batch = 3, a.seq = 0;
        CHECK(turn(a) == PAMM_OK);
    }
    a = rotation(), a.heads_k = 0, a.k_weight = nullptr;
    memset(&a.k, 0, sizeof a.k), memset(&a.k_out, 0, sizeof a.k_out);
    CHECK(pamm_rotary(&a, nullptr) == PAMM_OK);
}

static pamm_cache8_t cache() {
    pamm_cache8_t c;
    memset(&c, 0, sizeof c);
    c.dtype = PAMM_BF16, c.batch = 2, c.room = 100, c.heads_kv = 2, c.head_dim = 64, c.block = 32;
    c.k = c.v = heads(100, 2, 64), c.k_tail = c.v_tail = heads(32, 2, 64);
    c.k_scale = c.v_scale = {(float*)memory(), 6, 2, 1};
    return c;
}

static pamm_attention_t problem() {
    pamm_attention_t a;
    memset(&a, 0, sizeof a);
    a.dtype = PAMM_BF16, a.causal = 1, a.batch = 2, a.seq_q = 5, a.seq_k = 100, a.heads = 4, a.heads_kv = 2;
    a.head_dim = 64, a.scale = 0.125f, a.q = a.o = heads(5, 4, 64), a.lse = (float*)memory();
    a.k.stride_b = a.v.stride_s = INT64_MAX;  // not looked at
    return a;
}

static int attend(const pamm_attention_t& a, const pamm_cache8_t& c) {
    const size_t n = pamm_cache8_attention_workspace_size(&a, &c);
    void* ws = n && n < (1u << 28) ? aligned_alloc(256, n) : nullptr;
    const int r = pamm_cache8_attention(&a, &c, ws, ws ? n : 0, nullptr);
    free(ws);
    CHECK(known(r));
    return r;
}

static int append(const pamm_cache8_t& c, int64_t n) {
    const pamm_heads_t x = heads(7, 2, 64);
    const int r = pamm_cache8_append(&c, &x, &x, n, nullptr, (int32_t*)memory(), 1, nullptr);
    CHECK(known(r));
    return r;
}

static void caches() {
    CHECK(attend(problem(), cache()) == PAMM_OK && append(cache(), 7) == PAMM_OK);
    int64_t pamm_cache8_t::*sizes[] = {&pamm_cache8_t::batch, &pamm_cache8_t::room, &pamm_cache8_t::heads_kv,
                                       &pamm_cache8_t::head_dim, &pamm_cache8_t::block};
    for (auto x : sizes)
        for (auto y : sizes)
            for (int64_t v : kExtremes)
                for (int64_t w : kExtremes) {
                    pamm_cache8_t c = cache();
                    c.*x = v, c.*y = w;
                    for (int64_t n : kExtremes) append(c, n);
                    pamm_attention_t a = problem();
                    attend(a, c);
                    a.batch = c.batch, a.heads_kv = c.heads_kv, a.head_dim = c.head_dim, a.seq_k = c.room;
                    attend(a, c);
                }
    for (int64_t v : kExtremes) {
        for (pamm_scales_t pamm_cache8_t::*t : {&pamm_cache8_t::k_scale, &pamm_cache8_t::v_scale})
            for (int64_t pamm_scales_t::*s : {&pamm_scales_t::stride_b, &pamm_scales_t::stride_s, &pamm_scales_t::stride_h}) {
                pamm_cache8_t c = cache();
                (c.*t).*s = v;
                CHECK(v >= 0 || append(c, 7) == PAMM_ERR_SHAPE);
                append(c, 7), attend(problem(), c);
            }
        for (pamm_heads_t pamm_cache8_t::*t : {&pamm_cache8_t::k, &pamm_cache8_t::v_tail})
            for (int64_t pamm_heads_t::*s : {&pamm_heads_t::stride_b, &pamm_heads_t::stride_s, &pamm_heads_t::stride_h}) {
                pamm_cache8_t c = cache();
                (c.*t).*s = v;
                append(c, 7), attend(problem(), c);
            }
        for (int64_t pamm_attention_t::*s : {&pamm_attention_t::seq_q, &pamm_attention_t::seq_k, &pamm_attention_t::window}) {
            pamm_attention_t a = problem();
            a.*s = v;
            attend(a, cache());
        }
    }
}

static void nothing() {
    for (int64_t v : kExtremes) {
        pamm_cache8_t c = cache();
        c.batch = 0;
        c.k = c.v = c.k_tail = c.v_tail = {memory(), v, v, v};
        c.k_scale = c.v_scale = {(float*)memory(), v, v, v};
        pamm_attention_t a = problem();
        a.batch = 0;
        CHECK(append(c, 7) == PAMM_OK && attend(a, c) == PAMM_OK);
    }
}

int main() {
    positions();
    caches();
    nothing();
    printf("serving ABI sanitizer driver ok, %d launches\n", launches);
    return 0;
}
