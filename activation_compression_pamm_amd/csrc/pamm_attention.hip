// pamm_attention.hip -- attention forward on gfx950.
//
//   s_ij = scale <q_i, k_j>,  lse_i = log sum_j exp(s_ij),
//   o_i = sum_j exp(s_ij - lse_i) v_j
//
// in one pass over the keys with a running maximum m and sum l: a block of
// keys whose scores exceed m rescales what was summed by exp(m_old - m_new).
// All exponentials are powers of two (scores carry log2 e).
//
// Scores are formed transposed, S^T = K Q^T: a lane then owns one query, its
// statistics are two registers, the maximum needs one exchange between the
// wave's halves, and the probabilities leave the softmax in the register
// order that O^T = V^T P^T takes them in (pamm_attention_device.hpp).
//
// Queries of the heads that share a key/value head are rows of one problem:
// row r is position r / G of head r % G.
#include <algorithm>

#include "pamm_attention_forward.hpp"

namespace pamm {

// ---------------------------------------------------------------- many rows

// Four waves of 32 rows share tiles of 64 keys (32 in fp32 and for rows above 64,
// where 64 leave two waves a SIMD instead of three: 4 x 2048 tokens, 32 heads of
// 128, 5% more time), which two LDS buffers hold: while one is used, the next tile
// travels through registers into the other.
//
// No single unit bounds it: at that size the matrix unit is busy 41% of the
// cycles, vector instructions issue in 52%, waves wait 29% of theirs, and the clock
// falls below 2 GHz; without loads, barriers or softmax it is 3%, 3% and 0% faster.
// A wave has one chain of products, exponentials and products, and each operand
// read from LDS feeds one product.  174 us, 788 TFLOP/s of the pairs that the mask
// leaves; 8192 tokens, 32/8 heads of 64: 322 us, 854; 8 x 1024, 12 heads of 64: 30
// us, 428, whose 768 workgroups, all resident at once, end at very different times.
template <int DT, int ND>
struct RowsShared {
    static constexpr int BK = DT == DT_BF16 && ND <= 2 ? 64 : 32;
    char tile[2][2][BK * Tile<DT, ND>::PITCH];
};

template <int DT, int ND, bool SAFE>
__device__ __forceinline__ void attention_rows(const AttnArgs& a, int id, int row_tiles, RowsShared<DT, ND>& shared) {
    using T = Tile<DT, ND>;
    constexpr int BK = RowsShared<DT, ND>::BK;
    constexpr bool BY_SUM = DT == DT_BF16 && ND <= 2;
    auto& lds = shared.tile;
    const int tid = threadIdx.x, l = tid & 63, wave = wave_id();

    const WorkItem w = work_item(id, a.B * a.Hkv, row_tiles * a.nsplit, a.causal);
    const int split = w.item % a.nsplit, b = w.head / a.Hkv, hk = w.head % a.Hkv;
    const int tile = row_tiles - 1 - w.item / a.nsplit;  // the last rows see the most keys: they start first
    const int Lq = valid_length(a.q_len, b, a.Sq), Lk = valid_length(a.kv_len, b, a.Sk);
    const int rows = a.Sq * a.G;

    // what this lane's row, this wave's rows and this workgroup's rows see
    const int r0 = tile * 128, w0 = r0 + wave * 32, row = w0 + (l & 31);
    const int pos = row / a.G, head = hk * a.G + row % a.G;
    const bool live = row < rows;
    KeyRange mine = key_range(a, live ? pos : Lq, Lq, Lk);
    if (mine.hi < mine.lo) mine.hi = mine.lo;
    const RowsRange wr = rows_range(a, w0, 32, rows, Lq, Lk), br = rows_range(a, r0, 128, rows, Lq, Lk);

    int t0 = br.begin / BK, t1 = (br.end + BK - 1) / BK;
    if (t1 < t0) t1 = t0;
    if (a.nsplit > 1) {
        const int per = (t1 - t0 + a.nsplit - 1) / a.nsplit;
        const int s0 = t0 + split * per;
        t1 = s0 + per < t1 ? s0 + per : t1;
        t0 = s0 < t1 ? s0 : t1;
    }

    const char* kbase = a.k.p + b * a.k.sb + hk * a.k.sh;
    const char* vbase = a.v.p + b * a.v.sb + hk * a.v.sh;
    uint4 qf[T::NS];
    load_row_operand<DT, ND>(qf, a.q.p + b * a.q.sb + pos * a.q.ss + head * a.q.sh, live && pos < Lq, a.D);
    if (a.scale < 0.0f)
#pragma unroll
        for (int s = 0; s < T::NS; ++s) qf[s] = negate16<DT>(qf[s]);
    arrived(qf);
    const float c = score_factor(a.scale);

    f32x16 acc[ND];
#pragma unroll
    for (int db = 0; db < ND; ++db) acc[db] = f32x16{};
    Running st{BY_SUM ? kUnseen : -INFINITY, 0.0f};

    TileCopy<DT, ND, BK, 256> kc, vc;
    if (t0 < t1) {
        kc.fetch(kbase + t0 * BK * a.k.ss, (int)a.k.ss, Lk - t0 * BK, a.D, tid);
        vc.fetch(vbase + t0 * BK * a.v.ss, (int)a.v.ss, Lk - t0 * BK, a.D, tid);
        kc.put(lds[0][0], tid);
        vc.put(lds[0][1], tid);
    }
    __syncthreads();
    int cur = 0;
    for (int t = t0; t < t1; ++t, cur ^= 1) {
        const bool more = t + 1 < t1;
        if (more) {
            kc.fetch(kbase + (t + 1) * BK * a.k.ss, (int)a.k.ss, Lk - (t + 1) * BK, a.D, tid);
            vc.fetch(vbase + (t + 1) * BK * a.v.ss, (int)a.v.ss, Lk - (t + 1) * BK, a.D, tid);
        }
        const int rb = opaque(row_base<DT, ND>()), tb = opaque(trans_base<DT, ND>());
#pragma unroll
        for (int kb = 0; kb < BK / 32; ++kb) {
            const int key0 = t * BK + kb * 32;
            if (key0 >= wr.end || key0 + 32 <= wr.begin) continue;
            const bool part = key0 < wr.all_lo || key0 + 32 > wr.all_hi;
            auto scores = [&] {
                f32x16 s{};
#pragma unroll
                for (int i = 0; i < T::NS; ++i)
                    s = mma_step<DT>(row_operand<DT, ND>(lds[cur][0], kb * 32, rb, i), qf[i], s);
                settle<DT>(s);
                if (part) mask_block(s, key0, mine);
                return s;
            };
            f32x16 s = scores();
            if constexpr (BY_SUM) {
                float sum = probabilities(s, c, st.m);
                if (__any(sum > kMost)) {  // the first block of a row, then rarely: form the scores again
                    s = scores();
                    raise_reference<ND>(s, c, st, acc);
                    sum = probabilities(s, c, st.m);
                }
                st.l += sum;
            } else {
                softmax_update<ND>(s, c, st, acc);
            }
            Packed<DT> p;
            p.set(s);
            trans_product<DT, ND, true, SAFE>(lds[cur][1], kb * 32, tb, p, part, key0, mine, acc);
        }
        if (more) {
            kc.put(lds[cur ^ 1][0], tid);
            vc.put(lds[cur ^ 1][1], tid);
        }
        __syncthreads();
    }

#pragma unroll
    for (int db = 0; db < ND; ++db) settle<DT>(acc[db]);
    const bool marked = !SAFE && a.hides && !sums_finite<ND>(acc);
    if (!live) return;
    const float sum = half_sum(st.l);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    float lse2 = sum == 0.0f ? -INFINITY : st.m + __builtin_amdgcn_logf(sum);
    if (marked) lse2 = NAN;
    const int64_t at = ((int64_t)b * a.H + head) * a.Sq + pos;
    if (a.nsplit > 1) {
        store_rows<DT_F32, ND>(reinterpret_cast<char*>(a.part_o + (at * a.nsplit + split) * a.D), acc, inv, sum == 0.0f, a.D);
        if (l < 32) a.part_lse[at * a.nsplit + split] = lse2;
    } else {
        store_rows<DT, ND>(a.o.p + b * a.o.sb + pos * a.o.ss + head * a.o.sh, acc, inv, sum == 0.0f, a.D);
        if (l < 32) a.lse[at] = lse2 * kLn2;
    }
}

template <int DT, int ND>
__global__ __launch_bounds__(256, DT == DT_BF16 ? 3 : 1) void attention_kernel(AttnArgs a, int row_tiles) {
    __shared__ __attribute__((aligned(16))) RowsShared<DT, ND> shared;
    attention_rows<DT, ND, false>(a, blockIdx.x, row_tiles, shared);
}

template <int DT, int ND>
__global__ __launch_bounds__(256, 1) void attention_again_kernel(AttnArgs a, int row_tiles, int items) {
    __shared__ __attribute__((aligned(16))) RowsShared<DT, ND> shared;
    each_marked(
        items,
        [&](int id) {
            const WorkItem w = work_item(id, a.B * a.Hkv, row_tiles * a.nsplit, a.causal);
            const int row = (row_tiles - 1 - w.item / a.nsplit) * 128, split = w.item % a.nsplit;
            bool any = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) any |= is_marked(a, w, row + 32 * i, split);
            return any;
        },
        [&](int id) { attention_rows<DT, ND, true>(a, __builtin_amdgcn_readfirstlane(id), row_tiles, shared); });
}

// ----------------------------------------------------------------- few rows

// At most 32 rows (single tokens): every wave takes the same rows and 32-key
// blocks of its own, wave w the blocks w, w + 4, ... of this part, so nothing
// waits for another wave until the end.  A lane reads its K operand straight
// from memory (16 bytes of one key a step, the wave 32 keys), V goes through
// the wave's own LDS tile; the next block's loads are issued as soon as the
// registers of the current one are used.  Blocks are counted from the first key
// that a row sees, so a query alone never meets a key outside its window.
//
// Bound by reading K and V: 64 sequences of 64 to 8192 keys, 8 heads of 128, 1.11
// GB: 224 us, 4.95 TB/s (a large copy reaches 4.75), and 5 us for the join.  130
// keys of 12 heads: 6 us, one block's latency and the launch.
template <int DT, int ND, bool SAFE>
__device__ __forceinline__ void attention_few(const AttnArgs& a, int id, FewShared<DT, ND>& shared) {
    using T = Tile<DT, ND>;
    constexpr int VT = FewShared<DT, ND>::VT;
    char* lds = shared.lds;
    const int l = threadIdx.x & 63, wave = wave_id();

    const WorkItem w = work_item(id, a.B * a.Hkv, a.nsplit, false);
    const int split = w.item, b = w.head / a.Hkv, hk = w.head % a.Hkv;
    const int Lq = valid_length(a.q_len, b, a.Sq), Lk = valid_length(a.kv_len, b, a.Sk);
    const int rows = a.Sq * a.G;
    const int row = l & 31, pos = row / a.G, head = hk * a.G + row % a.G;
    const bool live = row < rows;
    KeyRange mine = key_range(a, live ? pos : Lq, Lq, Lk);
    if (mine.hi < mine.lo) mine.hi = mine.lo;
    const RowsRange br = rows_range(a, 0, rows, rows, Lq, Lk);
    const int first = br.begin, n = br.end > first ? (br.end - first + 31) / 32 : 0;
    const int per = (n + a.nsplit - 1) / a.nsplit, p0 = split * per, p1 = p0 + per < n ? p0 + per : n;

    const char* kbase = a.k.p + b * a.k.sb + hk * a.k.sh;
    const char* vbase = a.v.p + b * a.v.sb + hk * a.v.sh;
    uint4 qf[T::NS], kf[T::NS];
    load_row_operand<DT, ND>(qf, a.q.p + b * a.q.sb + pos * a.q.ss + head * a.q.sh, live && pos < Lq, a.D);
    if (a.scale < 0.0f)
#pragma unroll
        for (int s = 0; s < T::NS; ++s) qf[s] = negate16<DT>(qf[s]);
    arrived(qf);
    const float c = score_factor(a.scale);
    f32x16 acc[ND];
#pragma unroll
    for (int db = 0; db < ND; ++db) acc[db] = f32x16{};
    Running st{-INFINITY, 0.0f};
    char* vt = lds + wave * VT;
    TileCopy<DT, ND, 32, 64> vc;

    auto fetch = [&](int key0) {
        const RowView view(kbase + key0 * a.k.ss, (int)a.k.ss, Lk - key0, 32, a.D * T::ES);
#pragma unroll
        for (int i = 0; i < T::NS; ++i) {
            const int g = 2 * i + (l >> 5);
            kf[i] = view.load(g * T::PE < a.D ? row * (int)a.k.ss + g * 16 : kOutside);
        }
        vc.fetch(vbase + key0 * a.v.ss, (int)a.v.ss, Lk - key0, a.D, l);
    };
    int t = p0 + wave;
    if (t < p1) fetch(first + t * 32);
    for (; t < p1; t += 4) {
        const int key0 = first + t * 32;
        f32x16 s{};
#pragma unroll
        for (int i = 0; i < T::NS; ++i) s = mma_step<DT>(kf[i], qf[i], s);
        settle<DT>(s);
        __builtin_amdgcn_wave_barrier();
        vc.put(vt, l);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (t + 4 < p1) fetch(key0 + 128);
        const bool part = key0 < br.all_lo || key0 + 32 > br.all_hi;
        if (part) mask_block(s, key0, mine);
        softmax_update<ND>(s, c, st, acc);
        Packed<DT> p;
        p.set(s);
        trans_product<DT, ND, true, SAFE>(vt, 0, opaque(trans_base<DT, ND>()), p, part, key0, mine, acc);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }

#pragma unroll
    for (int db = 0; db < ND; ++db) settle<DT>(acc[db]);
    const bool marked = !SAFE && a.hides && !sums_finite<ND>(acc);

    join_waves<DT, ND>(a, shared, acc, st, marked, b, hk, split);
}

template <int DT, int ND>
__global__ __launch_bounds__(256, DT == DT_BF16 ? 2 : 1) void attention_few_kernel(AttnArgs a) {
    __shared__ __attribute__((aligned(16))) FewShared<DT, ND> shared;
    attention_few<DT, ND, false>(a, blockIdx.x, shared);
}

template <int DT, int ND>
__global__ __launch_bounds__(256, 1) void attention_few_again_kernel(AttnArgs a, int items) {
    __shared__ __attribute__((aligned(16))) FewShared<DT, ND> shared;
    each_marked(
        items,
        [&](int id) {
            const WorkItem w = work_item(id, a.B * a.Hkv, a.nsplit, false);
            return is_marked(a, w, 0, w.item);
        },
        [&](int id) { attention_few<DT, ND, true>(a, __builtin_amdgcn_readfirstlane(id), shared); });
}

// Joins the parts of one row: weights 2^(lse_part - lse).  Half a wave a row:
// lane s holds the weights of parts s and s + 32 (there are at most 64), then
// every lane adds up four columns, eight parts' loads at a time.  Bound by
// reading the parts: 3 of 32768 rows of 128, 59 MB in all, 12.2 us, 4.8 TB/s (a
// wave a row with 4 bytes a lane: 17 us with 2 parts).
template <int DT>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
    const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const bool live = at < (int64_t)a.B * a.H * a.Sq;
    const int l = threadIdx.x & 31, n = live ? a.nsplit : 0;
    const float* part = a.part_lse + at * a.nsplit;
    const float lse0 = l < n ? part[l] : -INFINITY, lse1 = l + 32 < n ? part[l + 32] : -INFINITY;
    float m = fmaxf(lse0, lse1);
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) m = fmaxf(m, shfl_xor(m, x));
    const float ref = m == -INFINITY ? 0.0f : m;
    const float w0 = __builtin_amdgcn_exp2f(lse0 - ref), w1 = __builtin_amdgcn_exp2f(lse1 - ref);
    float total = w0 + w1;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) total += shfl_xor(total, x);
    // parts that saw nothing hold zeros
    const float4* po = reinterpret_cast<const float4*>(a.part_o + at * a.nsplit * a.D) + l;
    const bool mine = 4 * l < a.D;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < a.nsplit; s += 8) {
        float4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = mine && s + i < n ? po[(s + i) * (a.D / 4)] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = __shfl(s < 32 ? w0 : w1, (s + i) & 31, 32);
            sum.x = fmaf(u, x[i].x, sum.x), sum.y = fmaf(u, x[i].y, sum.y);
            sum.z = fmaf(u, x[i].z, sum.z), sum.w = fmaf(u, x[i].w, sum.w);
        }
    }
    if (!live) return;
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    const int64_t pos = at % a.Sq, bh = at / a.Sq;
    char* o = a.o.p + (bh / a.H) * a.o.sb + pos * a.o.ss + (bh % a.H) * a.o.sh;
    if (mine) {
        if constexpr (DT == DT_BF16) {
            bf16x2 u, v;
            u[0] = (__bf16)(sum.x * inv), u[1] = (__bf16)(sum.y * inv);
            v[0] = (__bf16)(sum.z * inv), v[1] = (__bf16)(sum.w * inv);
            *reinterpret_cast<uint2*>(o + 8 * l) =
                make_uint2(__builtin_bit_cast(uint32_t, u), __builtin_bit_cast(uint32_t, v));
        } else {
            *reinterpret_cast<float4*>(o + 16 * l) =
                make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
        }
    }
    if (l == 0) a.lse[at] = total == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(total)) * kLn2;
}

void launch_attention_join(const AttnArgs& a, int dtype, hipStream_t st) {
    const dim3 grid((unsigned)(((int64_t)a.B * a.H * a.Sq + 7) / 8));
    auto* kernel = dtype == DT_BF16 ? attention_join_kernel<DT_BF16> : attention_join_kernel<DT_F32>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, a);
}

// Single tokens are bound by reading K and V once.  Where the keys' lengths are
// given they differ, unknown to the host, so the parts are made small enough to
// even them out: 8 workgroups a unit (64 sequences of up to 8192, 8 heads of
// 128: 229 us, against 245 with 4 and 272 with 2).  Equal lengths need no more
// than fill the device (369 us with 2, 389 with 4, 394 with 8).  A part is at
// least 256 keys, two blocks a wave; 512 for a tile of many rows, of which 3
// workgroups a unit run at once (2 x 512 queries over 8192 keys, 32/8 heads of
// 128: 166 us, 169 with 2, 177 with 4; 2048 of 2048, 16 heads of 128: 50, 53
// and 58; against 4 x 128 over 4096: 64, 61 and 73).
int attention_splits(int64_t B, int64_t Sq, int64_t Sk, int64_t Hkv, int64_t G, bool lengths, int num_cus) {
    const int64_t rows = Sq * G;
    const bool few = rows <= kFewRows;
    const int64_t tiles = few ? 1 : (rows + 127) / 128;
    const int64_t blocks = B * Hkv * tiles, want = (!few ? 3 : lengths ? 8 : 2) * (int64_t)num_cus, least = few ? 256 : 512;
    if (blocks == 0 || blocks >= want) return 1;
    int64_t n = (want + blocks - 1) / blocks;
    n = std::min(n, (Sk + least - 1) / least);
    return (int)std::max<int64_t>(1, std::min<int64_t>(n, kMaxSplits));
}

template <int DT, int ND>
static void launch_attention(const AttnArgs& a, hipStream_t st) {
    const int64_t rows = (int64_t)a.Sq * a.G, tiles = rows <= kFewRows ? 1 : (rows + 127) / 128;
    const int items = (int)((int64_t)a.B * a.Hkv * tiles * a.nsplit);
    const dim3 grid((unsigned)items), again((unsigned)std::min(items, a.num_cus));
    if (rows <= kFewRows) {
        hipLaunchKernelGGL((attention_few_kernel<DT, ND>), grid, dim3(256), 0, st, a);
        if (a.hides) hipLaunchKernelGGL((attention_few_again_kernel<DT, ND>), again, dim3(256), 0, st, a, items);
    } else {
        hipLaunchKernelGGL((attention_kernel<DT, ND>), grid, dim3(256), 0, st, a, (int)tiles);
        if (a.hides) hipLaunchKernelGGL((attention_again_kernel<DT, ND>), again, dim3(256), 0, st, a, (int)tiles, items);
    }
    if (a.nsplit > 1) launch_attention_join(a, DT, st);
}

hipError_t run_attention(const AttnArgs& a, int dtype, hipStream_t st) {
    const int nd = (a.D + 31) / 32;
#define PAMM_CASE(DT, ND) \
    if (dtype == DT && nd == ND) launch_attention<DT, ND>(a, st)
    PAMM_CASE(DT_BF16, 1);
    PAMM_CASE(DT_BF16, 2);
    PAMM_CASE(DT_BF16, 3);
    PAMM_CASE(DT_BF16, 4);
    PAMM_CASE(DT_F32, 1);
    PAMM_CASE(DT_F32, 2);
    PAMM_CASE(DT_F32, 3);
    PAMM_CASE(DT_F32, 4);
#undef PAMM_CASE
    return hipGetLastError();
}

}  // namespace pamm
