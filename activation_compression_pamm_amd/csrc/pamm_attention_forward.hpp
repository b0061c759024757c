// pamm_attention_forward.hpp -- what the forward kernels over caches of either
// kind share: running statistics of the softmax, and the joining of a
// workgroup's waves where each takes keys of its own.
#pragma once
#include "pamm_attention_device.hpp"

namespace pamm {

// Running statistics of one row, and its update by 32 keys.
//
// The reference m follows the maximum only when it is exceeded by more than
// 2^kSlack: until then probabilities up to 2^kSlack are summed against the old
// reference, which fp32 sums and bf16 products hold with the same relative
// precision, and the ND x 16 multiplications of a rescale are skipped.
constexpr float kSlack = 8.0f, kMost = 256.0f;  // kMost = 2^kSlack

struct Running {
    float m, l;  // m in log2 units; l: this lane's keys only
};

__device__ __forceinline__ float largest(const f32x16& s) {
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
    return half_max(top);
}

// s (raw products; masked ones already -inf) becomes the probabilities.
template <int ND>
__device__ __forceinline__ void softmax_update(f32x16& s, float c, Running& st, f32x16* acc) {
    const float top = largest(s) * c;
    if (__any(top > st.m + kSlack)) {
        const float m = fmaxf(st.m, top);
        const float f = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
        st.l *= f;
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[db][i] *= f;
        st.m = m;
    }
    const float ref = st.m == -INFINITY ? 0.0f : st.m;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -ref));
        sum += s[i];
    }
    st.l += sum;
}

// The same without looking for the maximum: the sum of the probabilities tells
// whether some are above the slack.  A row that saw nothing yet has the reference
// kUnseen, against which whatever it sees is infinite (or, for a score that low,
// right).  For rows up to 64 in bf16, where the softmax of a block takes longer than
// its products (8192 tokens, 32/8 heads of 64: 4% less time); with heads of 128 it
// gains nothing (4 x 2048 tokens).
constexpr float kUnseen = -3.402823466e38f;

__device__ __forceinline__ float probabilities(f32x16& s, float c, float ref) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -ref));
        sum += s[i];
    }
    return sum;
}

template <int ND>
__device__ __forceinline__ void raise_reference(const f32x16& s, float c, Running& st, f32x16* acc) {
    const float m = fmaxf(st.m, largest(s) * c), f = __builtin_amdgcn_exp2f(st.m - m);
    st.l *= f;
#pragma unroll
    for (int db = 0; db < ND; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[db][i] *= f;
    st.m = m;
}

__device__ __forceinline__ void mask_block(f32x16& s, int key0, const KeyRange& r) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (!sees(key0, i, r)) s[i] = -INFINITY;
}

// Scores' factor in log2 units; its sign is folded into the query operand.
__device__ __forceinline__ float score_factor(float scale) { return fmaxf(fabsf(scale) * kLog2e, 1e-36f); }

// LDS of the kernels for few rows: a V tile a wave, then the merged result.
template <int DT, int ND>
struct FewShared {
    static constexpr int OP = ND * 32 + 4;  // floats between rows of the merged result
    static constexpr int VT = 32 * Tile<DT, ND>::PITCH;
    static constexpr int SH = 4 * VT > 32 * OP * 4 ? 4 * VT : 32 * OP * 4;
    char lds[SH];
    float stat[4][2][32];
};

// Joins the four waves of a kernel for few rows and writes the result (or this
// part's): the common reference first, then the sums in order.
template <int DT, int ND>
__device__ __forceinline__ void join_waves(const AttnArgs& a, FewShared<DT, ND>& shared, const f32x16* acc,
                                           const Running& st, bool marked, int b, int hk, int split) {
    constexpr int OP = FewShared<DT, ND>::OP;
    char* lds = shared.lds;
    auto& stat = shared.stat;
    const int tid = threadIdx.x, l = tid & 63, wave = wave_id();
    const int rows = a.Sq * a.G, row = l & 31, pos = row / a.G, head = hk * a.G + row % a.G;
    const bool live = row < rows;
    const float sum = marked ? NAN : half_sum(st.l);  // makes the joined lse NaN
    if (l < 32) {
        stat[wave][0][l] = sum == 0.0f ? -INFINITY : st.m;
        stat[wave][1][l] = sum;
    }
    __syncthreads();
    float m = -INFINITY, total = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = fmaxf(m, stat[w][0][row]);
    const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int w = 0; w < 4; ++w) total += stat[w][1][row] * __builtin_amdgcn_exp2f(stat[w][0][row] - ref);
    const float f = sum == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(st.m - ref) / total;
    float* merged = reinterpret_cast<float*>(lds);
    for (int w = 0; w < 4; ++w) {
        if (w == wave && live) {
#pragma unroll
            for (int db = 0; db < ND; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float* to = merged + row * OP + 32 * db + 8 * (i >> 2) + 4 * (l >> 5) + (i & 3);
                    const float x = sum == 0.0f ? 0.0f : acc[db][i] * f;
                    *to = w == 0 ? x : *to + x;
                }
        }
        __syncthreads();
    }
    const float lse2 = total == 0.0f ? -INFINITY : m + __builtin_amdgcn_logf(total);
    const int64_t at = ((int64_t)b * a.H + head) * a.Sq + pos;
    if (tid < 32 && live) {
        if (a.nsplit > 1)
            a.part_lse[at * a.nsplit + split] = lse2;
        else
            a.lse[at] = lse2 * kLn2;
    }
    for (int e = tid; e < rows * a.D; e += 256) {
        const int r = e / a.D, x = e % a.D, p = r / a.G, h = hk * a.G + r % a.G;
        const float v = merged[r * OP + x];
        if (a.nsplit > 1) {
            a.part_o[((((int64_t)b * a.H + h) * a.Sq + p) * a.nsplit + split) * a.D + x] = v;
        } else {
            char* o = a.o.p + b * a.o.sb + p * a.o.ss + h * a.o.sh;
            if constexpr (DT == DT_BF16)
                reinterpret_cast<__bf16*>(o)[x] = (__bf16)v;
            else
                reinterpret_cast<float*>(o)[x] = v;
        }
    }
}

// The mark of a wave is the lse of its first row: NaN.  (One that is NaN by
// itself is computed twice, with the same result.)
__device__ __forceinline__ bool is_marked(const AttnArgs& a, const WorkItem& w, int row, int split) {
    if (row >= a.Sq * a.G) return false;
    const int b = w.head / a.Hkv, head = w.head % a.Hkv * a.G + row % a.G, pos = row / a.G;
    const int64_t at = ((int64_t)b * a.H + head) * a.Sq + pos;
    const float v = a.nsplit > 1 ? a.part_lse[at * a.nsplit + split] : a.lse[at];
    return v != v;
}

}  // namespace pamm
