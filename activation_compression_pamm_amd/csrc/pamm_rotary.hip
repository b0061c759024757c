// pamm_rotary.hip -- rotary positions of queries and keys, with their norm for
// each head in the same pass, and its gradients, on gfx950.
//
//   n = x rstd w (or x),  y = rotation of n by p inv_freq          forward
//   g = rotation of dy by -p inv_freq,  u = g w,  xhat = x rstd
//   dx = rstd (u - xhat mean(u xhat)),  dw = sum g xhat            backward
//
// Bound by memory: a head row is read once, held by `lanes` neighbouring lanes
// (two 16-byte vectors each, in the half layout the two that are rotated with
// each other) and written once.  The angles are the same for all heads of a
// token: a workgroup forms its tokens' cosines and sines once, one pair a
// thread, into LDS, and each lane keeps those of its elements while it goes
// over the token's heads.
#include <algorithm>

#include "pamm_device.hpp"
#include "pamm_rotary_kernels.hpp"

namespace pamm {

namespace {

constexpr int kThreads = 256;
constexpr int kTablePairs = 1024;
constexpr int kMaxHeadDim = 128;

enum : int { PAIRS_INTER = 0, PAIRS_HALF = 1, PAIRS_FAR = 2 };  // FAR: half, R2 not a whole number of vectors

// cos and sin of p * f radians.  The angle in turns and its reduction to
// within an eighth of one are exact to 64 bits, so that positions of millions
// lose nothing; the rest is the series of both functions up to pi / 4, whose
// first omitted terms are 1.8e-9 and 1.1e-10.
__device__ __forceinline__ float2 turn(double p, double f, float magnitude) {
    const double t = p * (f * 0.15915494309189533577);
    const double u = t - rint(t), q = rint(u * 4.0);
    const float x = (float)((u - q * 0.25) * 6.28318530717958647693), z = x * x;
    float s = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);  // 1/9!, -1/7!
    s = fmaf(z, s, 8.33333333e-3f);                      // 1/5!
    s = fmaf(z, s, -1.66666667e-1f);                     // -1/3!
    s = fmaf(x * z, s, x);
    float c = fmaf(z, -2.75573192e-7f, 2.48015873e-5f);  // -1/10!, 1/8!
    c = fmaf(z, c, -1.38888889e-3f);                     // -1/6!
    c = fmaf(z, c, 4.16666667e-2f);                      // 1/4!
    c = fmaf(z, c, -0.5f);
    c = fmaf(z, c, 1.0f);
    const int n = (int)q & 3;
    const float a = n & 1 ? s : c, b = n & 1 ? c : s;
    return make_float2((n == 1 || n == 2 ? -a : a) * magnitude, (n & 2 ? -b : b) * magnitude);
}

__device__ __forceinline__ double position(const RotaryArgs& a, int64_t token) {
    const int64_t b = token / a.S, s = token - b * a.S;
    int64_t p = s;
    if (a.positions) {
        const int64_t at = b * a.psb + s * a.pss;
        p = a.positions_64 ? reinterpret_cast<const int64_t*>(a.positions)[at]
                           : (int64_t)reinterpret_cast<const int32_t*>(a.positions)[at];
    }
    // two's complement sums of any positions are defined for unsigned numbers
    if (a.offset) p = (int64_t)((uint64_t)p + (uint64_t)(int64_t)a.offset[b]);
    return (double)p;
}

// The cosines and sines of the tokens [first, first + 2^tokens_log).
__device__ __forceinline__ void fill_table(const RotaryArgs& a, int64_t first, float2* table) {
    const int n = a.R2 << a.tokens_log;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int tk = i / a.R2, j = i - tk * a.R2;
        const int64_t token = first + tk;
        if (token < a.tokens) table[i] = turn(position(a, token), a.inv_freq[j], a.magnitude);
    }
}

// What a lane has of a head row: vectors `at[0]` and `at[1]`, the elements of
// them, and how they are rotated.
template <int DT, int PAIRS>
struct Row {
    static constexpr int P = Elem<DT>::per16;
    int at[2];   // vector of the row, or -1
    int lane, base;  // lane of the row; the lane group's first element in the exchange buffer
    float c[2 * P], s[2 * P];  // per element (FAR), per pair of the two vectors (HALF), per pair (INTER)

    __device__ __forceinline__ Row(const RotaryArgs& a) {
        const int nv = a.D / P;
        lane = threadIdx.x & ((1 << a.lanes_log) - 1);
        base = (threadIdx.x >> a.lanes_log) * a.D;
        if (PAIRS == PAIRS_HALF) {
            const int r = a.R2 / P;
            at[0] = lane < r ? lane : 2 * lane;
            at[1] = lane < r ? lane + r : 2 * lane + 1;
        } else {
            at[0] = 2 * lane, at[1] = 2 * lane + 1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (at[i] >= nv) at[i] = -1;
    }

    // The cosines and sines of this lane's elements; 1 and 0 where nothing is rotated.
    __device__ __forceinline__ void angles(const RotaryArgs& a, const float2* table, float sign) {
        auto take = [&](int i, int j, bool turned) {
            const float2 t = turned ? table[j] : make_float2(1.0f, 0.0f);
            c[i] = t.x, s[i] = sign * t.y;
        };
        if constexpr (PAIRS == PAIRS_HALF) {
#pragma unroll
            for (int e = 0; e < P; ++e) take(e, lane * P + e, lane < a.R2 / P);
        } else if constexpr (PAIRS == PAIRS_INTER) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int j = lane * P + i;
                take(i, j, j < a.R2);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2 * P; ++i) {
                const int e = 2 * lane * P + i;
                take(i, e < a.R2 ? e : e - a.R2, e < 2 * a.R2);
                if (e < a.R2) s[i] = -s[i];
            }
        }
    }

    __device__ __forceinline__ void load(const char* row, float* x) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = at[i] >= 0 ? *reinterpret_cast<const uint4*>(row + at[i] * 16) : make_uint4(0, 0, 0, 0);
            unpack16<DT>(v, x + i * P);
        }
    }
    // The same without unpacking, from a row that can be read in any case.
    __device__ __forceinline__ void fetch(const char* row, uint4 (&v)[2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = *reinterpret_cast<const uint4*>(row + (at[i] >= 0 ? at[i] * 16 : 0));
    }
    __device__ __forceinline__ void unpack(const uint4 (&v)[2], float* x) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) unpack16<DT>(at[i] >= 0 ? v[i] : make_uint4(0, 0, 0, 0), x + i * P);
    }
    __device__ __forceinline__ void store(char* row, const float* x) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (at[i] >= 0) *reinterpret_cast<uint4*>(row + at[i] * 16) = pack16<DT>(x + i * P);
    }

    // Rotates this lane's elements.  `exchange` holds a row for each group of
    // lanes: in the FAR layout an element's partner is in another lane.  All
    // lanes of the wave take part.
    __device__ __forceinline__ void rotate(const RotaryArgs& a, float* x, float* exchange) const {
        if constexpr (PAIRS == PAIRS_HALF) {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float u = x[e], v = x[P + e];
                x[e] = fmaf(u, c[e], -(v * s[e]));
                x[P + e] = fmaf(u, s[e], v * c[e]);
            }
        } else if constexpr (PAIRS == PAIRS_INTER) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float u = x[2 * i], v = x[2 * i + 1];
                x[2 * i] = fmaf(u, c[i], -(v * s[i]));
                x[2 * i + 1] = fmaf(u, s[i], v * c[i]);
            }
        } else {
            const int first = 2 * lane * P;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // what the row before was read for
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 2 * P; ++i)
                if (at[i / P] >= 0) exchange[base + first + i] = x[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 2 * P; ++i) {
                const int e = first + i;
                if (e >= 2 * a.R2) continue;
                const float other = exchange[base + (e < a.R2 ? e + a.R2 : e - a.R2)];
                x[i] = fmaf(x[i], c[i], other * s[i]);
            }
        }
    }
};

// Sum over the lanes of a row (up to 16), the same in each: with the neighbour,
// the neighbouring pair, four and eight.
template <int CTRL>
__device__ __forceinline__ float with_lane(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lanes_sum(float v, int lanes_log) {
    if (lanes_log > 0) v = with_lane<0xb1>(v);   // lanes 1, 0, 3, 2 of each four
    if (lanes_log > 1) v = with_lane<0x4e>(v);   // 2, 3, 0, 1
    if (lanes_log > 2) v = with_lane<0x141>(v);  // 7, 6, ... of each eight: the other four
    if (lanes_log > 3) v = with_lane<0x140>(v);  // 15, 14, ... of each sixteen: the other eight
    return v;
}

// Which part of the work a thread has: of the workgroup's 2^tokens_log tokens
// the one `token`, of its heads every `step`th from `head` on.
struct Share {
    int64_t token, b, s;
    int head, step, tk;
    bool live;
    __device__ __forceinline__ Share(const RotaryArgs& a, int64_t first) {
        const int group = threadIdx.x >> a.lanes_log, per_log = 8 - a.lanes_log - a.tokens_log;
        step = 1 << per_log;
        tk = group >> per_log, head = group & (step - 1);
        token = first + tk;
        live = token < a.tokens;
        b = token / a.S, s = token - b * a.S;
    }
};

__device__ __forceinline__ char* head_row(const HeadsArg& t, const Share& w, int h) {
    return t.p + w.b * t.sb + w.s * t.ss + h * t.sh;
}

template <int DT, int PAIRS, bool NORM>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a) {
    constexpr int P = Elem<DT>::per16;
    __shared__ float2 table[kTablePairs];
    __shared__ float exchange[PAIRS == PAIRS_FAR ? kThreads * 2 * P : 1];
    Row<DT, PAIRS> row(a);
    const int heads = a.Hq + a.Hk;
    float wq[NORM ? 2 * P : 1], wk[NORM ? 2 * P : 1];
    if constexpr (NORM) {
        row.load(a.wq, wq);
        row.load(a.Hk ? a.wk : a.wq, wk);
    }
    const int64_t step = (int64_t)gridDim.x << a.tokens_log;
    for (int64_t first = (int64_t)blockIdx.x << a.tokens_log; first < a.tokens; first += step) {
        fill_table(a, first, table);
        __syncthreads();
        const Share w(a, first);
        row.angles(a, table + w.tk * a.R2, a.inverse ? -1.0f : 1.0f);
        // every lane goes round as often: sums and exchanges take all lanes of a row's wave
        for (int h0 = 0; h0 < heads; h0 += w.step) {
            const int h = h0 + w.head;
            const bool live = w.live && h < heads, second = h >= a.Hq;
            float x[2 * P];
            if (live) {
                row.load(second ? head_row(a.k, w, h - a.Hq) : head_row(a.q, w, h), x);
            } else {
#pragma unroll
                for (int i = 0; i < 2 * P; ++i) x[i] = 0.0f;
            }
            if constexpr (NORM) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 2 * P; ++i) ss = fmaf(x[i], x[i], ss);
                const float rstd = 1.0f / sqrtf(lanes_sum(ss, a.lanes_log) / (float)a.D + a.eps);
#pragma unroll
                for (int i = 0; i < 2 * P; ++i) x[i] = x[i] * rstd * (second ? wk[i] : wq[i]);
            }
            row.rotate(a, x, exchange);
            if (live) row.store(second ? head_row(a.ko, w, h - a.Hq) : head_row(a.qo, w, h), x);
        }
        __syncthreads();  // the table is filled again
    }
}

// Workgroups a unit, all of which are resident: 168 registers a thread, 128 in fp32.
template <int DT> constexpr int kBackwardGroups = DT == DT_BF16 ? 3 : 4;

// The first `blocks_q` workgroups take the queries' heads, the others the keys':
// one weight's sums a thread, which leaves three waves a SIMD instead of two.
template <int DT, int PAIRS>
__global__ __launch_bounds__(kThreads, kBackwardGroups<DT>) void rotary_backward_kernel(RotaryArgs a) {
    constexpr int P = Elem<DT>::per16;
    __shared__ float2 table[kTablePairs];
    __shared__ float exchange[PAIRS == PAIRS_FAR ? kThreads * 2 * P : 1];
    __shared__ float sums[kThreads / 64][kMaxHeadDim];
    Row<DT, PAIRS> row(a);
    const bool keys = (int)blockIdx.x >= a.blocks_q;
    const int lanes = 1 << a.lanes_log, heads = keys ? a.Hk : a.Hq, block = blockIdx.x - (keys ? a.blocks_q : 0);
    const HeadsArg x_in = keys ? a.k : a.q, g_in = keys ? a.dk : a.dq, out = keys ? a.ko : a.qo;
    float dw[2 * P], wt[2 * P];
    row.load(keys ? a.wk : a.wq, wt);
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) dw[i] = 0.0f;
    const int64_t step = (int64_t)(keys ? gridDim.x - a.blocks_q : a.blocks_q) << a.tokens_log;
    // the next row's loads are under way while a row is worked on, also from one
    // group of tokens to the next; lanes without a row read the first one
    uint4 nx[2], ng[2];
    auto fetch = [&](const Share& w, int h) {
        const bool live = w.live && h < heads;
        row.fetch(live ? head_row(x_in, w, h) : x_in.p, nx);
        row.fetch(live ? head_row(g_in, w, h) : g_in.p, ng);
    };
    Share w(a, (int64_t)block << a.tokens_log);
    fetch(w, w.head);
    for (int64_t first = (int64_t)block << a.tokens_log; first < a.tokens; first += step) {
        fill_table(a, first, table);
        __syncthreads();
        row.angles(a, table + w.tk * a.R2, -1.0f);
        for (int h = w.head, h0 = 0; h0 < heads; h0 += w.step, h += w.step) {
            const Share now = w;
            const bool live = w.live && h < heads;
            float x[2 * P], g[2 * P];
            row.unpack(nx, x);
            row.unpack(ng, g);
            if (h0 + w.step >= heads) w = Share(a, first + step);
            fetch(w, h0 + w.step >= heads ? w.head : h + w.step);
            row.rotate(a, g, exchange);
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < 2 * P; ++i) {
                ss = fmaf(x[i], x[i], ss);
                dot = fmaf(g[i] * wt[i], x[i], dot);
            }
            ss = lanes_sum(ss, a.lanes_log), dot = lanes_sum(dot, a.lanes_log);
            const float rstd = 1.0f / sqrtf(ss / (float)a.D + a.eps), mean = dot * rstd / (float)a.D;
#pragma unroll
            for (int i = 0; i < 2 * P; ++i) {
                const float xhat = x[i] * rstd;
                if (live) dw[i] = fmaf(g[i], xhat, dw[i]);
                x[i] = rstd * fmaf(-xhat, mean, g[i] * wt[i]);
            }
            if (live) row.store(head_row(out, now, h), x);
        }
        __syncthreads();
    }
    // the weight's gradient of this workgroup: over the wave's rows by a fixed tree, then over the waves in order
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) {
        float v = dw[i];
        for (int m = lanes; m < 64; m <<= 1) v += shfl_xor(v, m);
        if ((threadIdx.x & 63) < lanes && row.at[i / P] >= 0) sums[threadIdx.x >> 6][row.at[i / P] * P + i % P] = v;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.D; e += kThreads) {
        float v = sums[0][e];
#pragma unroll
        for (int k = 1; k < kThreads / 64; ++k) v += sums[k][e];
        a.part[(int64_t)blockIdx.x * a.D + e] = v;
    }
}

// The weights' gradients: 64 lanes of 16 columns each take every 64th of the
// partial rows of their weight, then add up in order.
__global__ __launch_bounds__(1024) void rotary_dw_kernel(RotaryArgs a, int blocks) {
    __shared__ float sums[64][17];
    const int c = threadIdx.x & 15, g = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
    const bool keys = blockIdx.y != 0;
    const int from = keys ? a.blocks_q : 0, to = keys ? blocks : a.blocks_q;
    float s = 0.0f;
    if (col < a.D)
        for (int b = from + g; b < to; b += 64) s += a.part[(int64_t)b * a.D + col];
    sums[g][c] = s;
    __syncthreads();
    if (g == 0 && col < a.D) {
        for (int i = 1; i < 64; ++i) s += sums[i][c];
        (keys ? a.dwk : a.dwq)[col] = s;
    }
}

int pairs_of(const RotaryArgs& a, int dtype) {
    return a.interleaved ? PAIRS_INTER : a.R2 % (dtype == DT_BF16 ? 8 : 4) == 0 ? PAIRS_HALF : PAIRS_FAR;
}

int64_t token_groups(const RotaryArgs& a) { return ((a.tokens - 1) >> a.tokens_log) + 1; }

}  // namespace

// A row's vectors two a lane.  Tokens a workgroup: as many as leave each token
// enough groups of lanes for its heads in about four rounds (the angles are
// formed once a token, and a lane's share of them is fetched once), but no
// fewer workgroups than two a unit, and no more angles than the table holds.  In the
// backward pass, whose workgroups stay, no fewer groups of tokens than eight a unit.
void rotary_shape(RotaryArgs& a, int dtype, bool backward) {
    const int nv = a.D / (dtype == DT_BF16 ? 8 : 4), need = (nv + 1) / 2;
    a.lanes_log = 0;
    while ((1 << a.lanes_log) < need) ++a.lanes_log;
    const int groups = kThreads >> a.lanes_log, heads = a.Hq + a.Hk;
    a.tokens_log = 0;
    while ((2 << a.tokens_log) <= groups && (a.R2 << (a.tokens_log + 1)) <= kTablePairs &&
           (groups >> a.tokens_log) * 4 > heads && (a.tokens >> (a.tokens_log + 1)) >= (backward ? 8 : 2) * a.num_cus)
        ++a.tokens_log;
}

hipError_t run_rotary(const RotaryArgs& a, int dtype, hipStream_t st) {
    const int pairs = pairs_of(a, dtype);
    const bool norm = a.wq != nullptr;
    const dim3 grid((unsigned)std::min<int64_t>(token_groups(a), (int64_t)1 << 20));
#define PAMM_CASE(DT, PAIRS)                                                                                    \
    if (dtype == DT && pairs == PAIRS) {                                                                        \
        auto* kernel = norm ? rotary_kernel<DT, PAIRS, true> : rotary_kernel<DT, PAIRS, false>;                 \
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, a);                                             \
    }
#define PAMM_CASES                                                                                              \
    PAMM_CASE(DT_BF16, PAIRS_INTER) PAMM_CASE(DT_BF16, PAIRS_HALF) PAMM_CASE(DT_BF16, PAIRS_FAR)                \
    PAMM_CASE(DT_F32, PAIRS_INTER) PAMM_CASE(DT_F32, PAIRS_HALF) PAMM_CASE(DT_F32, PAIRS_FAR)
    PAMM_CASES
#undef PAMM_CASE
    return hipGetLastError();
}

// Each workgroup leaves a row of partial sums of its weight: as many as are
// resident, looping over their tokens, dealt to queries and keys as they have heads.
int rotary_backward_blocks(RotaryArgs& a, int dtype) {
    if (a.tokens == 0) return a.blocks_q = 0;
    const int64_t groups = token_groups(a);
    const int64_t most = (int64_t)a.num_cus * (dtype == DT_BF16 ? kBackwardGroups<DT_BF16> : kBackwardGroups<DT_F32>);
    if (a.Hk == 0) return a.blocks_q = (int)std::min(groups, most);
    const int64_t keys = std::min(groups, std::max<int64_t>(1, most * a.Hk / (a.Hq + a.Hk)));
    a.blocks_q = (int)std::min(groups, std::max<int64_t>(1, most - keys));
    return a.blocks_q + (int)keys;
}

hipError_t run_rotary_backward(RotaryArgs a, int dtype, hipStream_t st) {
    const int blocks = rotary_backward_blocks(a, dtype), pairs = pairs_of(a, dtype);
    if (blocks > 0) {
#define PAMM_CASE(DT, PAIRS)                                                                                    \
    if (dtype == DT && pairs == PAIRS)                                                                          \
        hipLaunchKernelGGL((rotary_backward_kernel<DT, PAIRS>), dim3(blocks), dim3(kThreads), 0, st, a);
        PAMM_CASES
#undef PAMM_CASE
    }
    hipLaunchKernelGGL(rotary_dw_kernel, dim3((a.D + 15) / 16, a.Hk > 0 ? 2 : 1), dim3(1024), 0, st, a, blocks);
    return hipGetLastError();
}
#undef PAMM_CASES

}  // namespace pamm
