// pamm_cache8.hip -- appending to a cache of keys and values in 8 bits, on
// gfx950.
//
//   scale = max |x| / 448 over a block of tokens of one head, value = e4m3(x / scale)
//
// Bound by memory: one workgroup holds a block of one head, keys and values, in
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

// Keys and values of a block of one head together: twice the loads under way in
// a workgroup, which lives only for one block.
template <int DT, int VPT>
__global__ __launch_bounds__(kThreads) void cache8_append_kernel(AppendArgs a, int64_t items) {
    constexpr int P = Elem<DT>::per16;
    __shared__ float tops[2][2][kThreads / 64];
    const int tid = threadIdx.x, per_row = a.D / P, block = 1 << a.block_log, vectors = block * per_row;
    int slot = 0;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int h = (int)(item % a.Hkv);
        const int64_t left = item / a.Hkv;
        const int j = (int)(left % a.touched), b = (int)(left / a.touched);
        const Extent e(a, b);
        const int first = (e.have >> a.block_log) + j, start = first << a.block_log, end = e.have + e.get;
        const char* x[2];
        char* tail[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            // row of token p: x + p * ss
            x[t] = a.t[t].x.p + b * a.t[t].x.sb + h * a.t[t].x.sh - e.have * a.t[t].x.ss;
            tail[t] = a.t[t].tail.p + b * a.t[t].tail.sb + h * a.t[t].tail.sh;
        }
        if (e.get > 0 && start + block <= end) {
            uint4 v[2][VPT];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int at = tid + i * kThreads, r = at / per_row, c = at - r * per_row;
                    v[t][i] = make_uint4(0, 0, 0, 0);
                    if (at < vectors)
                        v[t][i] = *reinterpret_cast<const uint4*>((start + r < e.have ? tail[t] + r * a.t[t].tail.ss
                                                                                      : x[t] + (start + r) * a.t[t].x.ss) +
                                                                  c * 16);
                }
            float top[2] = {0.0f, 0.0f};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    float u[P];
                    unpack16<DT>(v[t][i], u);
#pragma unroll
                    for (int k = 0; k < P; ++k) top[t] = fmaxf(top[t], isfinite(u[k]) ? fabsf(u[k]) : 0.0f);
                }
#pragma unroll
                for (int m = 1; m < 64; m <<= 1) top[t] = fmaxf(top[t], shfl_xor(top[t], m));
                if ((tid & 63) == 0) tops[slot][t][tid >> 6] = top[t];
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float most = tops[slot][t][0];
#pragma unroll
                for (int k = 1; k < kThreads / 64; ++k) most = fmaxf(most, tops[slot][t][k]);
                // 448 x / most = (7/8 x) / (most / 512): a quotient and its correction by the remainder, which for
                // bf16 (products of 3 and 8 bits) is rounded as the definition is; tiny numbers are raised by a power
                // of two first, below which the products would lose bits
                constexpr float kLeast = 1.17549435e-38f;
                most = fmaxf(most, 448.0f * kLeast);
                const float raise = most < 0x1p-60f ? 0x1p64f : 1.0f;
                const float inv = 512.0f / (most * raise), part = most * raise * (1.0f / 512.0f), seven = 0.875f * raise;
                const ScalesArg& sc = a.t[t].scale;
                if (tid == 0) sc.p[b * sc.sb + first * sc.ss + h * sc.sh] = most / 448.0f;
                const HeadsArg& out = a.t[t].to;
                char* to = out.p + b * out.sb + h * out.sh + start * out.ss;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int at = tid + i * kThreads, r = at / per_row, c = at - r * per_row;
                    if (at >= vectors) continue;
                    float u[P];
                    unpack16<DT>(v[t][i], u);
                    uint32_t o[P / 4];
#pragma unroll
                    for (int k = 0; k < P; k += 4) {
                        float w[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const float n = u[k + m] * seven, q = n * inv, f = fmaf(fmaf(-q, part, n), inv, q);
                            w[m] = isfinite(u[k + m]) ? fminf(fmaxf(f, -448.0f), 448.0f) : NAN;
                        }
                        o[k / 4] = __builtin_amdgcn_cvt_pk_fp8_f32(
                            w[2], w[3], __builtin_amdgcn_cvt_pk_fp8_f32(w[0], w[1], 0, false), true);
                    }
                    if constexpr (P == 8)
                        *reinterpret_cast<uint2*>(to + r * out.ss + c * P) = make_uint2(o[0], o[1]);
                    else
                        *reinterpret_cast<uint32_t*>(to + r * out.ss + c * P) = o[0];
                }
            }
            slot ^= 1;  // the next block's maxima: between two uses of one place lies a barrier
        }
        // the tokens behind the last whole block
        const int rest = end >> a.block_log << a.block_log, from = e.have > rest ? e.have : rest;
        if (j == 0 && from < end) {
            const int n = (end - from) * per_row;
            for (int i = tid; i < 2 * n; i += kThreads) {
                const bool second = i >= n;
                const int at = second ? i - n : i, r = at / per_row, c = at - r * per_row;
                const int64_t ts = second ? a.t[1].tail.ss : a.t[0].tail.ss, xs = second ? a.t[1].x.ss : a.t[0].x.ss;
                *reinterpret_cast<uint4*>((second ? tail[1] : tail[0]) + (from - rest + r) * ts + c * 16) =
                    *reinterpret_cast<const uint4*>((second ? x[1] : x[0]) + (from + r) * xs + c * 16);
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
