// pamm_clip.hip -- the global norm of many gradients, and clipping by it, on
// gfx950.
//
//   norm = sqrt(sum g^2),  coef = min(1, max_norm / (norm + eps)),  g *= coef
//
// Bound by memory: one read for the sum, one read and one write for the
// scaling.  The tensors of a launch travel as kernel arguments and are cut
// into chunks; workgroup b takes chunks b, b + grid, ...  Squares are summed
// in 64 bits: no bf16 or fp32 gradient overflows or vanishes in it, and the
// order is fixed, so the norm is bitwise repeatable.
#include "pamm_block_kernels.hpp"
#include "pamm_device.hpp"

namespace pamm {

constexpr int kClipThreads = 256;
constexpr int kClipChunk = 16384;  // elements

// Vectors at any element alignment (global memory takes them unaligned).
template <int DT> struct ClipVec;
template <> struct ClipVec<DT_BF16> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2))); };
template <> struct ClipVec<DT_F32> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4))); };

template <int DT>
__device__ __forceinline__ float load_one(const char* p, int64_t i) {
    if constexpr (DT == DT_BF16)
        return bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
    else
        return reinterpret_cast<const float*>(p)[i];
}
template <int DT>
__device__ __forceinline__ void store_one(char* p, int64_t i, float v) {
    if constexpr (DT == DT_BF16)
        reinterpret_cast<__bf16*>(p)[i] = (__bf16)v;
    else
        reinterpret_cast<float*>(p)[i] = v;
}

// f(element offset, values, how many) for the elements [begin, end) of a dense range.
template <int DT, typename F>
__device__ __forceinline__ void each_vector(const char* data, int64_t begin, int64_t end, F&& f) {
    typedef typename ClipVec<DT>::type vec;
    constexpr int P = Elem<DT>::per16, U = 4;
    int64_t i = begin + threadIdx.x * P;
    for (; i + (U - 1) * kClipThreads * P + P <= end; i += U * kClipThreads * P) {
        uint4 r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const vec v = *reinterpret_cast<const vec*>(data + (i + u * kClipThreads * P) * Elem<DT>::size);
            r[u] = make_uint4(v.x, v.y, v.z, v.w);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[P];
            unpack16<DT>(r[u], x);
            f(i + u * kClipThreads * P, x, P);
        }
    }
    for (; i < end; i += kClipThreads * P) {
        float x[P];
        const int m = end - i < P ? (int)(end - i) : P;
        if (m == P) {
            const vec v = *reinterpret_cast<const vec*>(data + i * Elem<DT>::size);
            unpack16<DT>(make_uint4(v.x, v.y, v.z, v.w), x);
        } else {
#pragma unroll
            for (int e = 0; e < P; ++e) x[e] = e < m ? load_one<DT>(data, i + e) : 0.0f;
        }
        f(i, x, m);
    }
}

// The tensor a chunk belongs to.
__device__ __forceinline__ int clip_tensor(const ClipArgs& a, int64_t chunk) {
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.t[mid].first_chunk <= chunk)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double sums[kClipThreads / 64];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sums[0];
#pragma unroll
    for (int i = 1; i < kClipThreads / 64; ++i) v += sums[i];
    return v;
}

template <int DT>
__device__ __forceinline__ double chunk_squares(const ClipTensor& t, int64_t chunk) {
    double s = 0.0;
    const int64_t total = t.rows * t.cols;
    const int64_t begin = chunk * kClipChunk, end = begin + kClipChunk < total ? begin + kClipChunk : total;
    if (t.rows == 1) {
        each_vector<DT>(t.data, begin, end, [&](int64_t, const float* x, int m) {
#pragma unroll
            for (int e = 0; e < Elem<DT>::per16; ++e)
                if (e < m) s = fma((double)x[e], (double)x[e], s);
        });
    } else {
        for (int64_t i = begin + threadIdx.x; i < end; i += kClipThreads) {
            const int64_t r = i / t.cols;
            const double x = load_one<DT>(t.data, r * t.ld + (i - r * t.cols));
            s = fma(x, x, s);
        }
    }
    return s;
}

__global__ __launch_bounds__(kClipThreads) void clip_sum_kernel(ClipArgs a) {
    double s = 0.0;
    for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        const ClipTensor& t = a.t[clip_tensor(a, c)];
        s += t.dtype == DT_BF16 ? chunk_squares<DT_BF16>(t, c - t.first_chunk)
                                : chunk_squares<DT_F32>(t, c - t.first_chunk);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) a.part[blockIdx.x] = s;
}

template <int DT, int DO>
__device__ __forceinline__ void chunk_scale(const ClipTensor& t, int64_t chunk, float coef) {
    typedef typename ClipVec<DO>::type vec;
    const int64_t total = t.rows * t.cols;
    const int64_t begin = chunk * kClipChunk, end = begin + kClipChunk < total ? begin + kClipChunk : total;
    if (t.rows == 1) {
        each_vector<DT>(t.data, begin, end, [&](int64_t i, const float* x, int m) {
            constexpr int P = Elem<DT>::per16, Q = Elem<DO>::per16;
            if constexpr (P >= Q) {
                if (m == P) {
#pragma unroll
                    for (int q = 0; q < P; q += Q) {
                        vec v;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            if constexpr (DO == DT_BF16) {
                                typedef __bf16 b2 __attribute__((ext_vector_type(2)));
                                b2 p;
                                p[0] = (__bf16)(x[2 * w] * coef), p[1] = (__bf16)(x[2 * w + 1] * coef);
                                v[w] = __builtin_bit_cast(uint32_t, p);
                            } else {
                                v[w] = __float_as_uint(x[q + w] * coef);
                            }
                        }
                        *reinterpret_cast<vec*>(t.out + (i + q) * Elem<DO>::size) = v;
                    }
                    return;
                }
            }
#pragma unroll
            for (int e = 0; e < P; ++e)
                if (e < m) store_one<DO>(t.out, i + e, x[e] * coef);
        });
    } else {
        for (int64_t i = begin + threadIdx.x; i < end; i += kClipThreads) {
            const int64_t r = i / t.cols, c = i - r * t.cols;
            store_one<DO>(t.out, r * t.ld_out + c, load_one<DT>(t.data, r * t.ld + c) * coef);
        }
    }
}

// Every workgroup adds up all partial sums (in the same order), so the norm
// needs no launch of its own.
__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(ClipArgs a) {
    double s = 0.0;
    for (int i = threadIdx.x; i < a.parts; i += kClipThreads) s += a.part[i];
    const float norm = (float)sqrt(block_sum(s));
    if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
    const float size = norm + a.eps;
    float coef = size == 0.0f ? 1.0f : a.max_norm / size;  // all gradients are 0: not 0 / 0 of them
    if (coef > 1.0f) coef = 1.0f;                          // NaN stays
    if (coef == 1.0f && a.in_place) return;
    for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        const ClipTensor& t = a.t[clip_tensor(a, c)];
        if (coef == 1.0f && t.out == t.data) continue;
        const int64_t k = c - t.first_chunk;
        if (t.dtype == DT_BF16)
            t.out_dtype == DT_BF16 ? chunk_scale<DT_BF16, DT_BF16>(t, k, coef) : chunk_scale<DT_BF16, DT_F32>(t, k, coef);
        else
            t.out_dtype == DT_BF16 ? chunk_scale<DT_F32, DT_BF16>(t, k, coef) : chunk_scale<DT_F32, DT_F32>(t, k, coef);
    }
}

int64_t clip_chunks(const ClipTensor& t) { return (t.rows * t.cols + kClipChunk - 1) / kClipChunk; }

hipError_t run_clip_sum(const ClipArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(clip_sum_kernel, dim3((unsigned)a.parts), dim3(kClipThreads), 0, st, a);
    return hipGetLastError();
}

hipError_t run_clip_scale(const ClipArgs& a, bool write, hipStream_t st) {
    ClipArgs b = a;
    if (!write) b.chunks = 0;
    const int64_t grid = b.chunks < 1 ? 1 : b.chunks < kClipBlocks ? b.chunks : kClipBlocks;
    hipLaunchKernelGGL(clip_scale_kernel, dim3((unsigned)grid), dim3(kClipThreads), 0, st, b);
    return hipGetLastError();
}

}  // namespace pamm
