// pamm_norm.hip -- residual addition with the root-mean-square norm, its
// backward pass and its 8-bit output, on gfx950.
//
//   h = x + r,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   g = w dy,   dx = dh + rstd (g - xhat mean(g xhat)),  dw = sum_i dy xhat
//
// Bound by memory: each row is read once, held in registers (VPT 16-byte
// vectors a thread, TPR threads a row) through its reductions, and written
// once.  Workgroups loop over rows, so w is loaded once each, and in the
// backward pass each thread sums dw for its columns over all its rows.
#include "pamm_block_kernels.hpp"
#include "pamm_device.hpp"

namespace pamm {

// Store the 16-byte group of element `col` of a row that holds d elements.
// Results are written past the caches: what reads them comes a whole matrix
// later (32768 x 4096 bf16 with the 8-bit output: 6% more time without this hint).
template <int DT>
__device__ __forceinline__ void store16_tail(char* row, int col, int d, const uint4& v) {
    constexpr int P = Elem<DT>::per16;
    if (col + P <= d) {
        const u32x4 t = {v.x, v.y, v.z, v.w};
        __builtin_nontemporal_store(t, reinterpret_cast<u32x4*>(row + (int64_t)col * Elem<DT>::size));
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    for (int e = 0; e < P && col + e < d; ++e) {
        if constexpr (DT == DT_BF16)
            reinterpret_cast<uint16_t*>(row)[col + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        else
            reinterpret_cast<uint32_t*>(row)[col + e] = w[e];
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += shfl_xor(v, m);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, shfl_xor(v, m));
    return v;
}

// Sum (or maximum) over the TPR threads of a row.  `slot` alternates between
// calls, so that one barrier a call is enough.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float (*buf)[16], int& slot) {
    v = MAX ? wave_max(v) : wave_sum(v);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) buf[slot][wave] = v;
        __syncthreads();
        v = buf[slot][0];
#pragma unroll
        for (int i = 1; i < W; ++i) v = MAX ? fmaxf(v, buf[slot][i]) : v + buf[slot][i];
        slot ^= 1;
    }
    return v;
}

template <int TPR> constexpr int kNormThreads = TPR < 256 ? 256 : TPR;

// Q: the 8-bit output is asked for.
template <int DT, int TPR, int VPT, bool Q>
__global__ __launch_bounds__(kNormThreads<TPR>) void add_rms_norm_kernel(NormArgs a) {
    constexpr int P = Elem<DT>::per16, RPB = kNormThreads<TPR> / TPR;
    __shared__ float buf[2][16];
    int slot = 0;
    const int tid = threadIdx.x % TPR, d = a.d;
    uint4 w[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) w[i] = load16_tail<DT>(a.w, (tid + i * TPR) * P, d);
    const int64_t step = (int64_t)gridDim.x * RPB;
    // the next row's loads are issued before this row's reductions; with more
    // than a wave a row, every thread takes part in every barrier of the loop
    uint4 x[VPT], r[VPT];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            x[i] = load16_tail<DT>(a.x + row * a.ldx, (tid + i * TPR) * P, d);
            if (a.r) r[i] = load16_tail<DT>(a.r + row * a.ldr, (tid + i * TPR) * P, d);
        }
    };
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (row < a.n) fetch(row);
    for (; row < a.n; row += step) {
        float v[VPT][P];
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            unpack16<DT>(x[i], v[i]);
            if (a.r) {
                float u[P];
                unpack16<DT>(r[i], u);
#pragma unroll
                for (int e = 0; e < P; ++e) u[e] += v[i][e];
                x[i] = pack16<DT>(u);  // h as it is stored is what the norm and the backward pass see
                unpack16<DT>(x[i], v[i]);
                if ((tid + i * TPR) * P < d) store16_tail<DT>(a.h + row * a.ldh, (tid + i * TPR) * P, d, x[i]);
            }
        }
        if (row + step < a.n) fetch(row + step);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < P; ++e) ss = fmaf(v[i][e], v[i][e], ss);
        ss = row_reduce<TPR, false>(ss, buf, slot);
        const float rstd = 1.0f / sqrtf(ss / (float)d + a.eps);
        if (a.rstd && tid == 0) a.rstd[row] = rstd;
        if (a.y) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float g[P];
                unpack16<DT>(w[i], g);
#pragma unroll
                for (int e = 0; e < P; ++e) g[e] *= v[i][e] * rstd;
                if ((tid + i * TPR) * P < d)
                    store16_tail<DT>(a.y + row * a.ldy, (tid + i * TPR) * P, d, pack16<DT>(g));
            }
        }
        if constexpr (!Q) continue;
        // y / scale = 448 p / max|p| for p = h w 2^k, with rstd = 2^k t, 1 <= t < 2: t
        // cancels, and for bf16 p is exact, so that elements half way between two
        // 8-bit values (1 of 3000, whose quotient fp32 holds) are rounded to even as
        // they should be and not by the errors of rstd, scale and 1 / scale.
        const uint32_t bits = __float_as_uint(rstd);
        const float t = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
        const float power = isfinite(rstd) ? __uint_as_float(bits & 0x7f800000u) : NAN;
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float g[P];
            unpack16<DT>(w[i], g);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                v[i][e] = v[i][e] * power * g[e];
                top = fmaxf(top, fabsf(v[i][e]));
            }
        }
        top = row_reduce<TPR, true>(top, buf, slot);
        // the scale is at least the smallest normal number, so that inverses are finite
        constexpr float kLeast = 1.17549435e-38f;
        if (tid == 0) a.qscale[row] = fmaxf(top * t / 448.0f, kLeast);
        // 448 p / most = (7/8 p) / (most / 512): a quotient and its correction by the remainder
        const float most = fmaxf(top, 448.0f * kLeast / t), inv = 512.0f / most;
        const float part = isinf(most) ? 0.0f : most * (1.0f / 512.0f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (tid + i * TPR) * P;
            if (col >= d) continue;
            uint32_t o[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < P; e += 2) {
                float u[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float n = v[i][e + j] * 0.875f, q = n * inv;
                    u[j] = fmaf(fmaf(-q, part, n), inv, q);  // NaN stays NaN below
                    u[j] = u[j] > 448.0f ? 448.0f : u[j] < -448.0f ? -448.0f : u[j];
                }
                if (e & 2)
                    o[e >> 2] = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], o[e >> 2], true);
                else
                    o[e >> 2] = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], o[e >> 2], false);
            }
            uint8_t* to = a.q + row * a.ldq + col;
            if (col + P <= d) {
                if constexpr (P == 8)
                    *reinterpret_cast<uint2*>(to) = make_uint2(o[0], o[1]);
                else
                    *reinterpret_cast<uint32_t*>(to) = o[0];
            } else {
                for (int e = 0; e < P && col + e < d; ++e) to[e] = (uint8_t)(o[e >> 2] >> (8 * (e & 3)));
            }
        }
    }
}

template <int DT, int TPR, int VPT>
__global__ __launch_bounds__(kNormThreads<TPR>) void add_rms_norm_backward_kernel(NormArgs a) {
    constexpr int P = Elem<DT>::per16, RPB = kNormThreads<TPR> / TPR;
    __shared__ float buf[2][16];
    __shared__ float cols[RPB > 1 ? VPT * TPR * P : 1];
    int slot = 0;
    const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR, d = a.d;
    uint4 w[VPT];
    float dw[VPT][P];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        w[i] = load16_tail<DT>(a.w, (tid + i * TPR) * P, d);
#pragma unroll
        for (int e = 0; e < P; ++e) dw[i][e] = 0.0f;
    }
    const int64_t step = (int64_t)gridDim.x * RPB;
    uint4 nh[VPT], ny[VPT], nd[VPT];
    float nr = 0.0f;
    auto fetch = [&](int64_t row) {
        nr = a.rstd[row];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            nh[i] = load16_tail<DT>(a.h + row * a.ldh, (tid + i * TPR) * P, d);
            ny[i] = load16_tail<DT>(a.dy + row * a.lddy, (tid + i * TPR) * P, d);
            if (a.dh) nd[i] = load16_tail<DT>(a.dh + row * a.lddh, (tid + i * TPR) * P, d);
        }
    };
    int64_t row = (int64_t)blockIdx.x * RPB + sub;
    if (row < a.n) fetch(row);
    for (; row < a.n; row += step) {
        uint4 h[VPT], dy[VPT], dh[VPT];
        float dot = 0.0f;
        const float rstd = nr;
#pragma unroll
        for (int i = 0; i < VPT; ++i) h[i] = nh[i], dy[i] = ny[i], dh[i] = nd[i];
        if (row + step < a.n) fetch(row + step);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float x[P], y[P], g[P];
            unpack16<DT>(h[i], x);
            unpack16<DT>(dy[i], y);
            unpack16<DT>(w[i], g);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float t = y[e] * (x[e] * rstd);
                dw[i][e] += t;
                dot = fmaf(t, g[e], dot);
            }
        }
        dot = row_reduce<TPR, false>(dot, buf, slot) / (float)d;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (tid + i * TPR) * P;
            if (col >= d) continue;
            float x[P], y[P], g[P], o[P];
            unpack16<DT>(h[i], x);
            unpack16<DT>(dy[i], y);
            unpack16<DT>(w[i], g);
#pragma unroll
            for (int e = 0; e < P; ++e) o[e] = rstd * (g[e] * y[e] - x[e] * rstd * dot);
            if (a.dh) {
                unpack16<DT>(dh[i], x);
#pragma unroll
                for (int e = 0; e < P; ++e) o[e] += x[e];
            }
            store16_tail<DT>(a.dx + row * a.lddx, col, d, pack16<DT>(o));
        }
    }
    // the workgroup's rows of partial sums, added in order
    if constexpr (RPB > 1) {
        for (int s = 0; s < RPB; ++s) {
            if (s == sub) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < P; ++e) {
                        float* to = cols + (tid + i * TPR) * P + e;
                        dw[i][e] = s == 0 ? dw[i][e] : *to + dw[i][e];
                        *to = dw[i][e];
                    }
            }
            __syncthreads();
        }
        if (sub != RPB - 1) return;
    }
    float* part = a.part + (int64_t)blockIdx.x * d;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) {
            const int col = (tid + i * TPR) * P + e;
            if (col < d) part[col] = dw[i][e];
        }
}

// dw = the sum of `blocks` rows of partial sums: 16 lanes of 64 columns each
// take every 16th row, then add up in order.  512 rows of 4096: 5 us, the latency
// of 32 loads a thread and the launch.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* part, int blocks, int d, float* dw) {
    __shared__ float sums[16][64];
    const int col = blockIdx.x * 64 + (threadIdx.x & 63), g = threadIdx.x >> 6;
    float s = 0.0f;
    if (col < d)
#pragma unroll 4
        for (int b = g; b < blocks; b += 16) s += part[(int64_t)b * d + col];
    sums[g][threadIdx.x & 63] = s;
    __syncthreads();
    if (g == 0 && col < d) {
        for (int i = 1; i < 16; ++i) s += sums[i][threadIdx.x];
        dw[col] = s;
    }
}

namespace {

struct NormShape {
    int tpr, vpt;
};

// Threads and vectors a row: as few threads as hold the row in 4 vectors each
// (a wave needs no barrier, and 8 vectors take half of the registers); more
// where there are too few rows to fill the device, so that a row's latency falls.
NormShape norm_shape(int64_t n, int64_t d, int dtype, int num_cus) {
    const int64_t vec = (d + (dtype == DT_BF16 ? 7 : 3)) / (dtype == DT_BF16 ? 8 : 4);
    int tpr = vec <= 64 * 4 ? 64 : vec <= 256 * 4 ? 256 : 1024;
    if (n < 4 * num_cus) {
        if (tpr == 64 && vec > 64) tpr = 256;
        if (tpr == 256 && vec > 512) tpr = 1024;
    }
    int vpt = 1;
    while ((int64_t)vpt * tpr < vec) vpt *= 2;
    return {tpr, vpt};
}

// Two workgroups a unit, looping over rows with the next row's loads under way
// (32768 x 4096 bf16: 171 us, 5.5 TB/s, with the 8-bit output, 177 with 8 a
// unit; backward 189 us, 5.7 TB/s, 210 with 4); one of 1024 threads where it
// also holds sums.
int norm_blocks(int64_t n, const NormShape& s, bool sums, int num_cus) {
    const int rpb = s.tpr < 256 ? 256 / s.tpr : 1, per_cu = sums && s.tpr == 1024 ? 1 : 2;
    const int64_t all = (n + rpb - 1) / rpb, most = (int64_t)num_cus * per_cu;
    return (int)(all < most ? all : most);
}

}  // namespace

#define PAMM_NORM_CASES(RUN) \
    RUN(64, 1) RUN(64, 2) RUN(64, 4) RUN(256, 1) RUN(256, 2) RUN(256, 4) RUN(1024, 1) RUN(1024, 2) RUN(1024, 4)

hipError_t run_add_rms_norm(const NormArgs& a, int dtype, hipStream_t st) {
    const NormShape s = norm_shape(a.n, a.d, dtype, a.num_cus);
    const dim3 grid((unsigned)norm_blocks(a.n, s, false, a.num_cus));
#define PAMM_RUN(T, V)                                                                                           \
    if (s.tpr == T && s.vpt == V) {                                                                              \
        auto* kernel = dtype == DT_BF16 ? (a.q ? add_rms_norm_kernel<DT_BF16, T, V, true>                        \
                                               : add_rms_norm_kernel<DT_BF16, T, V, false>)                      \
                                        : (a.q ? add_rms_norm_kernel<DT_F32, T, V, true>                         \
                                               : add_rms_norm_kernel<DT_F32, T, V, false>);                      \
        hipLaunchKernelGGL(kernel, grid, dim3(kNormThreads<T>), 0, st, a);                                       \
    }
    PAMM_NORM_CASES(PAMM_RUN)
#undef PAMM_RUN
    return hipGetLastError();
}

int norm_backward_blocks(int64_t n, int64_t d, int dtype, int num_cus) {
    const NormShape s = norm_shape(n, d, dtype, num_cus);
    return norm_blocks(n, s, true, num_cus);
}

hipError_t run_add_rms_norm_backward(const NormArgs& a, int dtype, hipStream_t st) {
    const NormShape s = norm_shape(a.n, a.d, dtype, a.num_cus);
    const int blocks = norm_backward_blocks(a.n, a.d, dtype, a.num_cus);
    if (blocks > 0) {
#define PAMM_RUN(T, V)                                                                                               \
    if (s.tpr == T && s.vpt == V) {                                                                                  \
        if (dtype == DT_BF16)                                                                                        \
            hipLaunchKernelGGL((add_rms_norm_backward_kernel<DT_BF16, T, V>), dim3(blocks), dim3(kNormThreads<T>), 0, \
                               st, a);                                                                               \
        else                                                                                                         \
            hipLaunchKernelGGL((add_rms_norm_backward_kernel<DT_F32, T, V>), dim3(blocks), dim3(kNormThreads<T>), 0, \
                               st, a);                                                                               \
    }
        PAMM_NORM_CASES(PAMM_RUN)
#undef PAMM_RUN
    }
    hipLaunchKernelGGL(norm_dw_kernel, dim3((a.d + 63) / 64), dim3(1024), 0, st, a.part, blocks, a.d, a.dw);
    return hipGetLastError();
}

}  // namespace pamm
