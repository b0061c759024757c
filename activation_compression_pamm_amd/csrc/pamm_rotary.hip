// pamm_rotary.hip -- rotary positions of queries and keys, with their norm for
// each head in the same pass, and its gradients, on gfx950.
//
//   n = x rstd w (or x),  y = rotation of n by p inv_freq          forward
//   g = rotation of dy by -p inv_freq,  u = g w,  xhat = x rstd
//   dx = rstd (u - xhat mean(u xhat)),  dw = sum g xhat            backward
//
// Bound by memory: a head row is read once, held by `lanes` neighbouring lanes
// (two 16-byte vectors each, in the half layout the two that are rotated with
// each other) and written once.  A workgroup takes the heads of some tokens of
// one of the two tensors, row after row over all of them, with the next row's
// loads under way; the angles, the same for all heads of a token, it forms once,
// a pair a thread, into LDS, with where each token's rows lie.
#include <algorithm>

#include "pamm_device.hpp"
#include "pamm_rotary_kernels.hpp"

namespace pamm {

namespace {

constexpr int kThreads = 256;
constexpr int kTablePairs = 2048, kTokens = 64;  // of a workgroup at a time
constexpr int kMaxHeadDim = 128;

// FAR: either layout, R2 not a whole number of vectors, so that a lane's elements are rotated in part.  (A choice for
// each pair in the interleaved kernel took norm and rotation of 4 x 2048 tokens, 32/8 heads of 128, from 32 to 38 us.)
enum : int { PAIRS_INTER = 0, PAIRS_HALF = 1, PAIRS_FAR = 2 };

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
    const uint32_t b = (uint32_t)token / (uint32_t)a.S, s = (uint32_t)token - b * (uint32_t)a.S;
    int64_t p = s;
    if (a.positions) {
        const int64_t at = (int64_t)b * a.psb + (int64_t)s * a.pss;
        p = a.positions_64 ? reinterpret_cast<const int64_t*>(a.positions)[at]
                           : (int64_t)reinterpret_cast<const int32_t*>(a.positions)[at];
    }
    // two's complement sums of any positions are defined for unsigned numbers
    if (a.offset) p = (int64_t)((uint64_t)p + (uint64_t)(int64_t)a.offset[b]);
    return (double)p;
}

// The tokens of a workgroup: cosines and sines, `width` a token of which those
// from R2 on are 1 and 0, and offsets of the tokens' rows in each of N tensors.
template <int N>
struct Tokens {
    __attribute__((aligned(16))) float2 table[kTablePairs];
    int64_t at[N][kTokens];
    __device__ __forceinline__ void fill(const RotaryArgs& a, int64_t first, int n, const HeadsArg* const (&t)[N]) {
        const float inv = 1.0f / (float)a.width;
        for (int i = threadIdx.x; i < n * a.width; i += kThreads) {
            const int tk = quotient(i, inv), j = i - tk * a.width;
            table[i] = j < a.R2 ? turn(position(a, first + tk), a.inv_freq[j], a.magnitude) : make_float2(1.0f, 0.0f);
        }
        if ((int)threadIdx.x < n) {
            const uint32_t token = (uint32_t)first + threadIdx.x, b = token / (uint32_t)a.S, s = token - b * (uint32_t)a.S;
#pragma unroll
            for (int i = 0; i < N; ++i) at[i][threadIdx.x] = b * t[i]->sb + s * t[i]->ss;
        }
    }
    // i / d for i < 2^20, given 1 / d
    __device__ static __forceinline__ int quotient(int i, float inv) { return (int)(((float)i + 0.5f) * inv); }
};

// What a lane has of a head row: vectors `at[0]` and `at[1]`, the elements of
// them, and how they are rotated.
template <int DT, int PAIRS>
struct Row {
    static constexpr int P = Elem<DT>::per16;
    int at[2];   // vector of the row, or -1
    bool full;   // every lane of a row has two vectors
    int lane, base;  // lane of the row; the lane group's first element in the exchange buffer
    int angle;       // where this lane's cosines and sines begin in a token's
    float c[2 * P], s[2 * P];  // per element (FAR), per pair of the two vectors (HALF), per pair (INTER)

    __device__ __forceinline__ Row(const RotaryArgs& a) {
        const int nv = a.D / P;
        lane = threadIdx.x & ((1 << a.lanes_log) - 1);
        base = (threadIdx.x >> a.lanes_log) * a.D;
        full = nv == 2 << a.lanes_log;
        if (PAIRS == PAIRS_HALF) {
            const int r = a.R2 / P;
            at[0] = lane < r ? lane : 2 * lane;
            at[1] = lane < r ? lane + r : 2 * lane + 1;
            angle = lane < r ? lane * P : a.R2;
        } else {
            at[0] = 2 * lane, at[1] = 2 * lane + 1;
            angle = lane * P;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (at[i] >= nv) at[i] = -1;
    }

    // The cosines and sines of this lane's elements of a token.
    __device__ __forceinline__ void angles(const RotaryArgs& a, const float2* table, float sign) {
        if constexpr (PAIRS == PAIRS_FAR) {
#pragma unroll
            for (int i = 0; i < 2 * P; ++i) {
                const int e = 2 * lane * P + i;
                const bool first = a.interleaved ? e % 2 == 0 : e < a.R2;
                const float2 t = table[e >= 2 * a.R2 ? a.R2 : a.interleaved ? e / 2 : first ? e : e - a.R2];
                c[i] = t.x, s[i] = first ? -sign * t.y : sign * t.y;
            }
        } else {
            const float4* from = reinterpret_cast<const float4*>(table + angle);
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float4 t = from[i / 2];
                c[i] = t.x, s[i] = sign * t.y, c[i + 1] = t.z, s[i + 1] = sign * t.w;
            }
        }
    }

    // The vectors of a row that can be read in any case.
    __device__ __forceinline__ void fetch(const char* row, uint4 (&v)[2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = *reinterpret_cast<const uint4*>(row + (at[i] >= 0 ? at[i] * 16 : 0));
    }
    __device__ __forceinline__ void unpack(uint4 (&v)[2], float* x) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!full && at[i] < 0) v[i] = make_uint4(0, 0, 0, 0);
            unpack16<DT>(v[i], x + i * P);
        }
    }
    __device__ __forceinline__ void load(const char* row, float* x) const {
        uint4 v[2];
        fetch(row, v);
        unpack(v, x);
    }
    __device__ __forceinline__ void store(char* row, const float* x) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (at[i] >= 0) *reinterpret_cast<uint4*>(row + at[i] * 16) = pack16<DT>(x + i * P);
    }

    // Rotates this lane's elements; those past the rotated ones are left alone, as what is not
    // finite in one of them must not reach another.  `exchange` holds a row for each group of
    // lanes: in the FAR layout an element's partner may be in another lane.  All
    // lanes of the wave take part.
    __device__ __forceinline__ void rotate(const RotaryArgs& a, float* x, float* exchange) const {
        auto turned = [&](float& u0, float& v0, int i) {
            const float u = u0, v = v0;
            u0 = fmaf(u, c[i], -(v * s[i]));
            v0 = fmaf(u, s[i], v * c[i]);
        };
        if constexpr (PAIRS == PAIRS_HALF) {
            if (lane * P >= a.R2) return;
#pragma unroll
            for (int e = 0; e < P; ++e) turned(x[e], x[P + e], e);
        } else if constexpr (PAIRS == PAIRS_INTER) {
            if (lane * P >= a.R2) return;
#pragma unroll
            for (int i = 0; i < P; ++i) turned(x[2 * i], x[2 * i + 1], i);
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
                const float other = exchange[base + (a.interleaved ? e ^ 1 : e < a.R2 ? e + a.R2 : e - a.R2)];
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

// Workgroups a unit of the backward pass, all of which are resident: 168 registers
// a thread, 128 in fp32.
template <int DT> constexpr int kBackwardGroups = DT == DT_BF16 ? 3 : 4;

// Which tensor a workgroup takes, and of which tokens: the first `blocks_q`
// workgroups the queries, the others the keys.
struct Part {
    bool keys;
    int heads, block, blocks;
    __device__ __forceinline__ Part(const RotaryArgs& a) {
        keys = (int)blockIdx.x >= a.blocks_q;
        heads = keys ? a.Hk : a.Hq;
        block = (int)blockIdx.x - (keys ? a.blocks_q : 0);
        blocks = keys ? (int)gridDim.x - a.blocks_q : a.blocks_q;
    }
};

template <int DT, int PAIRS, bool NORM>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a) {
    constexpr int P = Elem<DT>::per16;
    __shared__ Tokens<2> tokens;
    __shared__ float exchange[PAIRS == PAIRS_FAR ? kThreads * 2 * P : 1];
    Row<DT, PAIRS> row(a);
    const Part part(a);
    const HeadsArg in = part.keys ? a.k : a.q, out = part.keys ? a.ko : a.qo;
    const float sign = a.inverse ? -1.0f : 1.0f, inv_d = 1.0f / (float)a.D, inv_heads = 1.0f / (float)part.heads;
    float w[NORM ? 2 * P : 1];
    if constexpr (NORM) row.load(part.keys ? a.wk : a.wq, w);
    const int group = threadIdx.x >> a.lanes_log, groups = kThreads >> a.lanes_log;
    for (int64_t first = (int64_t)part.block * a.T; first < a.tokens; first += (int64_t)part.blocks * a.T) {
        const int n = a.tokens - first < a.T ? (int)(a.tokens - first) : a.T, rows = n * part.heads;
        const HeadsArg* const both[2] = {&in, &out};
        tokens.fill(a, first, n, both);
        __syncthreads();
        // every lane goes round as often: sums and exchanges take all lanes of a row's wave
        if constexpr (NORM) {
            int tk, h;
            uint4 next[2];
            auto fetch = [&](int r) {  // lanes without a row read the first one
                const int some = r < rows ? r : 0;
                tk = a.T > 1 ? tokens.quotient(some, inv_heads) : 0, h = some - tk * part.heads;
                row.fetch(in.p + tokens.at[0][tk] + h * in.sh, next);
            };
            fetch(group);
            for (int r = group, r0 = 0; r0 < rows; r0 += groups, r += groups) {
                float x[2 * P];
                row.unpack(next, x);
                row.angles(a, tokens.table + tk * a.width, sign);
                char* to = out.p + tokens.at[1][tk] + h * out.sh;
                if (r0 + groups < rows) fetch(r + groups);
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 2 * P; ++i) ss = fmaf(x[i], x[i], ss);
                const float rstd = 1.0f / sqrtf(lanes_sum(ss, a.lanes_log) * inv_d + a.eps);
#pragma unroll
                for (int i = 0; i < 2 * P; ++i) x[i] = x[i] * rstd * w[i];
                row.rotate(a, x, exchange);
                if (r < rows) row.store(to, x);
            }
        } else {
            // the rotation alone does little for a row: each group of lanes stays with one token, whose angles
            // it keeps (4 x 2048 tokens, 64 heads of 128: 45 us; 49 with rows as above)
            const int per = groups / a.T, tk = group / per, h0 = group - tk * per, some = tk < n ? tk : 0;
            row.angles(a, tokens.table + some * a.width, sign);
            const char* from = in.p + tokens.at[0][some] + h0 * in.sh;
            char* to = out.p + tokens.at[1][some] + h0 * out.sh;
            const int64_t in_step = per * in.sh, out_step = per * out.sh;
            for (int h = h0, i = 0; i < part.heads; i += per, h += per, from += in_step, to += out_step) {
                const bool live = tk < n && h < part.heads;
                float x[2 * P];
                row.load(live ? from : in.p, x);
                row.rotate(a, x, exchange);
                if (live) row.store(to, x);
            }
        }
        __syncthreads();  // the table is filled again
    }
}

template <int DT, int PAIRS>
__global__ __launch_bounds__(kThreads, kBackwardGroups<DT>) void rotary_backward_kernel(RotaryArgs a) {
    constexpr int P = Elem<DT>::per16;
    __shared__ Tokens<3> tokens;
    __shared__ float exchange[PAIRS == PAIRS_FAR ? kThreads * 2 * P : 1];
    __shared__ float sums[kThreads / 64][kMaxHeadDim];
    Row<DT, PAIRS> row(a);
    const Part part(a);
    const HeadsArg x_in = part.keys ? a.k : a.q, g_in = part.keys ? a.dk : a.dq, out = part.keys ? a.ko : a.qo;
    const float inv_d = 1.0f / (float)a.D, inv_heads = 1.0f / (float)part.heads;
    float dw[2 * P], wt[2 * P];
    row.load(part.keys ? a.wk : a.wq, wt);
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) dw[i] = 0.0f;
    const int group = threadIdx.x >> a.lanes_log, groups = kThreads >> a.lanes_log;
    for (int64_t first = (int64_t)part.block * a.T; first < a.tokens; first += (int64_t)part.blocks * a.T) {
        const int n = a.tokens - first < a.T ? (int)(a.tokens - first) : a.T, rows = n * part.heads;
        const HeadsArg* const three[3] = {&x_in, &g_in, &out};
        tokens.fill(a, first, n, three);
        __syncthreads();
        int tk, h;
        uint4 nx[2], ng[2];
        auto fetch = [&](int r) {  // lanes without a row read the first one
            const int some = r < rows ? r : 0;
            tk = a.T > 1 ? tokens.quotient(some, inv_heads) : 0, h = some - tk * part.heads;
            row.fetch(x_in.p + tokens.at[0][tk] + h * x_in.sh, nx);
            row.fetch(g_in.p + tokens.at[1][tk] + h * g_in.sh, ng);
        };
        fetch(group);
        for (int r = group, r0 = 0; r0 < rows; r0 += groups, r += groups) {
            float x[2 * P], g[2 * P];
            row.unpack(nx, x);
            row.unpack(ng, g);
            row.angles(a, tokens.table + tk * a.width, -1.0f);
            char* to = out.p + tokens.at[2][tk] + h * out.sh;
            if (r0 + groups < rows) fetch(r + groups);
            row.rotate(a, g, exchange);
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < 2 * P; ++i) {
                ss = fmaf(x[i], x[i], ss);
                dot = fmaf(g[i] * wt[i], x[i], dot);
            }
            ss = lanes_sum(ss, a.lanes_log), dot = lanes_sum(dot, a.lanes_log);
            const float rstd = 1.0f / sqrtf(ss * inv_d + a.eps), mean = dot * rstd * inv_d;
            if (r < rows) {
#pragma unroll
                for (int i = 0; i < 2 * P; ++i) {
                    const float xhat = x[i] * rstd;
                    dw[i] = fmaf(g[i], xhat, dw[i]);
                    x[i] = rstd * fmaf(-xhat, mean, g[i] * wt[i]);
                }
                row.store(to, x);
            }
        }
        __syncthreads();
    }
    // the weight's gradient of this workgroup: over the wave's rows by a fixed tree, then over the waves in order
    for (int m = 1 << a.lanes_log; m < 64; m <<= 1)
#pragma unroll
        for (int i = 0; i < 2 * P; ++i) dw[i] += shfl_xor(dw[i], m);
    if ((threadIdx.x & 63) < 1 << a.lanes_log)
#pragma unroll
        for (int i = 0; i < 2 * P; ++i)
            if (row.at[i / P] >= 0) sums[threadIdx.x >> 6][row.at[i / P] * P + i % P] = dw[i];
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
    return a.R2 % (dtype == DT_BF16 ? 8 : 4) != 0 ? PAIRS_FAR : a.interleaved ? PAIRS_INTER : PAIRS_HALF;
}

}  // namespace

// A row's vectors two a lane.
//
// Forward: tokens for about eight rows a group of lanes, so that there are many
// workgroups of which some load while others form angles, but at least two a unit
// (4 x 2048 tokens, 64 heads of 128: 50 us with five workgroups a unit that stay).
// Backward: workgroups that stay, as each leaves a row of partial sums: as many as are
// resident, dealt to queries and keys as they have heads, each with its tokens in as few
// equal parts as the table holds, so that all end together (8 x 1024 tokens, 12 heads of
// 64: 19 us; 24 with parts of four tokens).
int rotary_shape(RotaryArgs& a, int dtype, bool norm, bool backward) {
    const int per16 = dtype == DT_BF16 ? 8 : 4, nv = a.D / per16, pairs = pairs_of(a, dtype);
    a.lanes_log = 0;
    while ((2 << a.lanes_log) < nv) ++a.lanes_log;
    a.width = pairs == PAIRS_HALF ? a.R2 + per16 : pairs == PAIRS_INTER ? per16 << a.lanes_log : a.R2 + 1;
    const int64_t heads = std::max(a.Hq, a.Hk), most_tokens = std::max<int64_t>(
        1, std::min<int64_t>({kTokens, kTablePairs / a.width, ((int64_t)1 << 20) / heads}));
    const int groups = kThreads >> a.lanes_log;
    if (!backward && !norm) {  // a power of two, that divides the groups of lanes; about four rows a group
        a.T = 1;
        while (2 * a.T <= std::min<int64_t>(groups, most_tokens) && groups / a.T * 4 > a.Hq &&
               a.tokens / (2 * a.T) >= 2 * a.num_cus)
            a.T *= 2;
    } else if (!backward) {
        a.T = (int)std::max<int64_t>(1, std::min<int64_t>({most_tokens, 8 * groups / a.Hq,
                                                           a.tokens / (2 * a.num_cus)}));
    }
    if (!backward) {
        const int64_t all = (a.tokens + a.T - 1) / a.T;
        a.blocks_q = (int)std::min<int64_t>(all, (int64_t)1 << 20);
        if (a.Hk == 0) return a.blocks_q;
        return a.blocks_q + (int)std::max<int64_t>(all > 0, std::min<int64_t>(a.blocks_q, all * a.Hk / a.Hq));
    }
    const int64_t blocks = (int64_t)a.num_cus * (dtype == DT_BF16 ? kBackwardGroups<DT_BF16> : kBackwardGroups<DT_F32>);
    const int64_t keys = a.Hk == 0 ? 0 : std::max<int64_t>(1, blocks * a.Hk / (a.Hq + a.Hk));
    const int64_t queries = std::max<int64_t>(1, blocks - keys);
    // tokens a workgroup of the queries has, in equal parts
    const int64_t share = std::max<int64_t>(1, (a.tokens + queries - 1) / queries);
    const int64_t parts = (share + most_tokens - 1) / most_tokens;
    a.T = (int)((share + parts - 1) / parts);
    const int64_t all = (a.tokens + a.T - 1) / a.T;
    a.blocks_q = (int)std::min(all, queries);
    return a.blocks_q + (int)std::min(all, keys);
}

hipError_t run_rotary(const RotaryArgs& a, int blocks, int dtype, hipStream_t st) {
    const int pairs = pairs_of(a, dtype);
    const bool norm = a.wq != nullptr;
    const dim3 grid((unsigned)blocks);
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

hipError_t run_rotary_backward(const RotaryArgs& a, int blocks, int dtype, hipStream_t st) {
    const int pairs = pairs_of(a, dtype);
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
