// pamm_cache8.hip -- appending to a cache of keys and values in 8 bits, on
// gfx950.
//
//   scale = max |x| / 448 over a block of tokens of one head, value = e4m3(448 x / max |x|)
//
// Bound by memory and by the vector unit (maxima, quotients with their
// remainders): ragged prompts of 4 x 2048 tokens, 32 heads of 128, blocks of 32,
// bf16, 33 us, 4.2 TB/s with vector issue in 81% of the cycles; a look at each
// element for what is not finite made it 37, and keys and values in
// workgroups of their own 41 of those.  All of 2048 tokens: 40 us, 5.0 TB/s; behind 17 that wait in the
// tail, with a choice of base for each row, 42; in fp32 70.  One token of 64 sequences, 8 heads of 128: 4 us.
//
// One workgroup holds a block of one head, keys and values, in
// registers through the maximum, so each token is read once and written once.
// A block is taken when its last token arrives; its first ones may wait in the
// tail.  The workgroup of the first block that a call touches also writes the
// tail, after it has read it, so nothing waits for another workgroup.
#include <algorithm>

#include "pamm_cache_kernels.hpp"
#include "pamm_device.hpp"

namespace pamm {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int clamped(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// What sequence b has, and what it gets: tokens that fit the room.
struct Extent {
    int have, get;
    __device__ __forceinline__ Extent(const AppendArgs& a, int b) {
        have = clamped(a.lengths[b], 0, a.room);
        get = a.new_len ? clamped(a.new_len[b], 0, a.n) : a.n;
        if (get > a.room - have) get = a.room - have;
    }
};

// The largest |x| of a vector's elements as bits, with what is not finite above all else.
template <int DT>
__device__ __forceinline__ uint32_t top_bits(const uint4& v, uint32_t top) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == DT_BF16) {  // two at a time, each half in place
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        u16x2 t = __builtin_bit_cast(u16x2, top);
#pragma unroll
        for (int i = 0; i < 4; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
        return __builtin_bit_cast(uint32_t, t);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, w[i] & 0x7fffffffu);
        return top;
    }
}

constexpr float kLeast = 1.17549435e-38f;  // of a scale

// A vector's elements as they are stored.
template <int DT, bool FINITE>
__device__ __forceinline__ void eight_bits(const uint4& v, float inv, float part, float seven, uint32_t* o) {
    constexpr int P = Elem<DT>::per16;
    float u[P];
    unpack16<DT>(v, u);
#pragma unroll
    for (int k = 0; k < P; k += 4) {
        float w[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            // at most 448 but for a rounding, which the conversion takes back
            const float n = u[k + m] * seven, q = n * inv;
            w[m] = fmaf(fmaf(-q, part, n), inv, q);
            if (!FINITE && !isfinite(u[k + m])) w[m] = NAN;
        }
        o[k / 4] = __builtin_amdgcn_cvt_pk_fp8_f32(w[2], w[3], __builtin_amdgcn_cvt_pk_fp8_f32(w[0], w[1], 0, false), true);
    }
}

// Keys and values of a block of one head together: twice the loads under way in
// a workgroup, which lives only for one block.
template <int DT, int VPT>
__global__ __launch_bounds__(kThreads) void cache8_append_kernel(AppendArgs a, int64_t items) {
    constexpr int P = Elem<DT>::per16;
    __shared__ uint32_t tops[2][2][kThreads / 64];
    const int tid = threadIdx.x, per_row = a.D / P, block = 1 << a.block_log, vectors = block * per_row;
    const float inv_row = 1.0f / (float)per_row;
    auto row_of = [&](int at) { return (int)(((float)at + 0.5f) * inv_row); };  // at / per_row, for at < 2^20
    int slot = 0;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int h = (int)(item % a.Hkv);
        const int64_t left = item / a.Hkv;
        const int j = (int)(left % a.touched), b = (int)(left / a.touched);
        const Extent e(a, b);
        const int first = (e.have >> a.block_log) + j, start = first << a.block_log, end = e.have + e.get;
        const char* x[2];  // the new tokens
        char* tail[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            x[t] = a.t[t].x.p + b * a.t[t].x.sb + h * a.t[t].x.sh;
            tail[t] = a.t[t].tail.p + b * a.t[t].tail.sb + h * a.t[t].tail.sh;
        }
        if (e.get > 0 && start + block <= end) {
            // rows of the block that wait in the tail; those behind them begin at this token of the call's
            const int waiting = e.have > start ? e.have - start : 0, from = start + waiting - e.have;
            uint4 v[2][VPT];
            uint32_t top[2] = {0, 0};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const char* rows = x[t] + (from - waiting) * a.t[t].x.ss;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int at = tid + i * kThreads, r = row_of(at), c = at - r * per_row;
                    v[t][i] = make_uint4(0, 0, 0, 0);
                    if (at >= vectors) continue;
                    // a row's distance, 128 times, is below 2^32
                    if (waiting == 0)
                        v[t][i] = *reinterpret_cast<const uint4*>(rows + ((uint32_t)r * (uint32_t)a.t[t].x.ss + c * 16));
                    else
                        v[t][i] = *reinterpret_cast<const uint4*>((r < waiting ? tail[t] + r * a.t[t].tail.ss
                                                                               : rows + r * a.t[t].x.ss) + c * 16);
                }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) top[t] = top_bits<DT>(v[t][i], top[t]);
                if constexpr (DT == DT_BF16) top[t] = max(top[t] & 0xffffu, top[t] >> 16) << 16;
#pragma unroll
                for (int m = 1; m < 64; m <<= 1) top[t] = max(top[t], (uint32_t)shfl_xor((int)top[t], m));
                if ((tid & 63) == 0) tops[slot][t][tid >> 6] = top[t];
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t bits = tops[slot][t][0];
#pragma unroll
                for (int k = 1; k < kThreads / 64; ++k) bits = max(bits, tops[slot][t][k]);
                const bool finite = bits < 0x7f800000u;
                if (!finite) {  // rarely: the largest of the others, by every wave for itself
                    float most = 0.0f;
                    const char* rows = x[t] + (from - waiting) * a.t[t].x.ss;
                    for (int at = tid & 63; at < vectors; at += 64) {
                        const int r = row_of(at), c = at - r * per_row;
                        float u[P];
                        unpack16<DT>(*reinterpret_cast<const uint4*>((r < waiting ? tail[t] + r * a.t[t].tail.ss
                                                                                  : rows + r * a.t[t].x.ss) + c * 16), u);
#pragma unroll
                        for (int k = 0; k < P; ++k) most = fmaxf(most, isfinite(u[k]) ? fabsf(u[k]) : 0.0f);
                    }
#pragma unroll
                    for (int m = 1; m < 64; m <<= 1) most = fmaxf(most, shfl_xor(most, m));
                    bits = __float_as_uint(most);
                }
                // 448 x / most = (7/8 x) / (most / 512): a quotient and its correction by the remainder, which for
                // bf16 (products of 3 and 8 bits) is rounded as the definition is; tiny numbers are raised by a power
                // of two first, below which the products would lose bits
                const float most = fmaxf(__uint_as_float(bits), 448.0f * kLeast), raise = most < 0x1p-60f ? 0x1p64f : 1.0f;
                const float inv = 512.0f / (most * raise), part = most * raise * (1.0f / 512.0f), seven = 0.875f * raise;
                const ScalesArg& sc = a.t[t].scale;
                if (tid == 0) sc.p[b * sc.sb + first * sc.ss + h * sc.sh] = most / 448.0f;
                const HeadsArg& out = a.t[t].to;
                char* to = out.p + b * out.sb + h * out.sh + start * out.ss;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int at = tid + i * kThreads, r = row_of(at), c = at - r * per_row;
                    if (at >= vectors) continue;
                    uint32_t o[P / 4];
                    if (finite)
                        eight_bits<DT, true>(v[t][i], inv, part, seven, o);
                    else
                        eight_bits<DT, false>(v[t][i], inv, part, seven, o);
                    char* place = to + ((uint32_t)r * (uint32_t)out.ss + c * P);
                    if constexpr (P == 8)
                        *reinterpret_cast<uint2*>(place) = make_uint2(o[0], o[1]);
                    else
                        *reinterpret_cast<uint32_t*>(place) = o[0];
                }
            }
            slot ^= 1;           // the next block's maxima: between two uses of one place lies a barrier
            if (waiting > 0) __syncthreads();  // the tail is written below: every wave has read it, also for a second time
        }
        // the tokens behind the last whole block
        const int rest = end >> a.block_log << a.block_log, behind = e.have > rest ? e.have : rest;
        if (j == 0 && behind < end) {
            const int n = (end - behind) * per_row;
            for (int i = tid; i < 2 * n; i += kThreads) {
                const bool second = i >= n;
                const int at = second ? i - n : i, r = row_of(at), c = at - r * per_row;
                const int64_t ts = second ? a.t[1].tail.ss : a.t[0].tail.ss, xs = second ? a.t[1].x.ss : a.t[0].x.ss;
                *reinterpret_cast<uint4*>((second ? tail[1] : tail[0]) + (behind - rest + r) * ts + c * 16) =
                    *reinterpret_cast<const uint4*>((second ? x[1] : x[0]) + (behind - e.have + r) * xs + c * 16);
            }
        }
    }
}

__global__ __launch_bounds__(kThreads) void cache8_advance_kernel(AppendArgs a) {
    for (int64_t b = blockIdx.x * (int64_t)kThreads + threadIdx.x; b < a.B; b += (int64_t)gridDim.x * kThreads) {
        const Extent e(a, (int)b);
        a.lengths[b] = e.have + e.get;
    }
}

}  // namespace

hipError_t run_cache8_append(const AppendArgs& a, int dtype, hipStream_t st) {
    const int64_t items = (int64_t)a.B * a.Hkv * a.touched;
    const dim3 grid((unsigned)std::min<int64_t>(items, (int64_t)1 << 20));
    const int vectors = (a.D / (dtype == DT_BF16 ? 8 : 4)) << a.block_log;
#define PAMM_CASE(V)                                                                                     \
    if (vectors <= V * kThreads) {                                                                       \
        auto* kernel = dtype == DT_BF16 ? cache8_append_kernel<DT_BF16, V> : cache8_append_kernel<DT_F32, V>; \
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, a, items);                               \
    } else
    PAMM_CASE(1) PAMM_CASE(2) PAMM_CASE(4) PAMM_CASE(8) PAMM_CASE(16) return hipErrorInvalidValue;
#undef PAMM_CASE
    if (a.advance)
        hipLaunchKernelGGL(cache8_advance_kernel, dim3((unsigned)std::min((a.B + kThreads - 1) / kThreads, 1024)),
                           dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace pamm
