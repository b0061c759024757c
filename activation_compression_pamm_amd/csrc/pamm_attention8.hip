// pamm_attention8.hip -- attention over a cache held in 8 bits with a scale for
// each block of tokens and head, on gfx950.
//
//   s_ij = (scale ks_j) <q_i, k_j>,  o_i = sum_j (exp(s_ij - lse_i) vs_j) v_j
//
// The forward pass of attention (same tiles, running statistics, order of
// operands and joins), whose keys and values arrive as 8-bit floats: these are
// exact in bf16 and fp32, into which they are widened on their way, and 32 keys
// lie in one block, so that their scales are two numbers a tile.  Keys behind
// the last whole block come from the tail, in the queries' type.
#include <algorithm>

#include "pamm_attention_forward.hpp"
#include "pamm_cache_kernels.hpp"

namespace pamm {

// 16 8-bit floats as 16 / per16 vectors of the type; exact.
template <int DT>
__device__ __forceinline__ void widen16(const uint4& r, uint4* out) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (DT == DT_BF16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                u[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * i + j], 1.0f, false));
                u[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * i + j], 1.0f, true));
            }
            out[i] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
            out[i] = make_uint4(__float_as_uint(lo[0]), __float_as_uint(lo[1]), __float_as_uint(hi[0]),
                                __float_as_uint(hi[1]));
        }
    }
}

// Where 16-byte groups of 8-bit rows (2 ND of them, D / 16 in use) become
// vectors of the type.
template <int DT, int ND>
struct Wide {
    using T = Tile<DT, ND>;
    static constexpr int PER = 16 / T::PE;  // vectors of one group
    static constexpr int GROUPS = 2 * ND;
    static constexpr int N = 32 * GROUPS;   // groups of a tile
    // Writes group c of row r to a tile.
    __device__ static __forceinline__ void put(char* tile, int r, int c, const uint4& raw) {
        uint4 v[PER];
        widen16<DT>(raw, v);
#pragma unroll
        for (int i = 0; i < PER; ++i) *reinterpret_cast<uint4*>(tile + T::offset(r, PER * c + i)) = v[i];
    }
};

__device__ __forceinline__ float scale_of(const ScalesArg& s, int b, int block, int h) {
    return s.p[b * s.sb + block * s.ss + h * s.sh];
}

// The start of the tail.
__device__ __forceinline__ int whole_blocks(const Cache8Args& c, int Lk) { return Lk >> c.block_log << c.block_log; }

// ---------------------------------------------------------------- many rows

// As attention_rows: four waves of 32 rows share tiles of 32 keys in two LDS
// buffers, the next tile under way in registers.
template <int DT, int ND>
struct Rows8Shared {
    char tile[2][2][32 * Tile<DT, ND>::PITCH];
};

template <int DT, int ND, bool SAFE>
__device__ __forceinline__ void attention8_rows(const AttnArgs& a, const Cache8Args& c8, int id, int row_tiles,
                                                Rows8Shared<DT, ND>& shared) {
    using T = Tile<DT, ND>;
    using W = Wide<DT, ND>;
    auto& lds = shared.tile;
    const int tid = threadIdx.x, l = tid & 63, wave = wave_id();

    const WorkItem w = work_item(id, a.B * a.Hkv, row_tiles * a.nsplit, a.causal);
    const int split = w.item % a.nsplit, b = w.head / a.Hkv, hk = w.head % a.Hkv;
    const int tile = row_tiles - 1 - w.item / a.nsplit;
    const int Lq = valid_length(a.q_len, b, a.Sq), Lk = valid_length(a.kv_len, b, a.Sk), whole = whole_blocks(c8, Lk);
    const int rows = a.Sq * a.G;

    const int r0 = tile * 128, w0 = r0 + wave * 32, row = w0 + (l & 31);
    const int pos = row / a.G, head = hk * a.G + row % a.G;
    const bool live = row < rows;
    KeyRange mine = key_range(a, live ? pos : Lq, Lq, Lk);
    if (mine.hi < mine.lo) mine.hi = mine.lo;
    const RowsRange wr = rows_range(a, w0, 32, rows, Lq, Lk), br = rows_range(a, r0, 128, rows, Lq, Lk);

    int t0 = br.begin / 32, t1 = (br.end + 31) / 32;
    if (t1 < t0) t1 = t0;
    if (a.nsplit > 1) {
        const int per = (t1 - t0 + a.nsplit - 1) / a.nsplit;
        const int s0 = t0 + split * per;
        t1 = s0 + per < t1 ? s0 + per : t1;
        t0 = s0 < t1 ? s0 : t1;
    }

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
    Running st{-INFINITY, 0.0f};

    // a tile on its way: 8 bits in the first vector of each copy, or the tail's rows
    const char* kbase = a.k.p + b * a.k.sb + hk * a.k.sh;
    const char* vbase = a.v.p + b * a.v.sb + hk * a.v.sh;
    const char* ktail = c8.kt.p + b * c8.kt.sb + hk * c8.kt.sh;
    const char* vtail = c8.vt.p + b * c8.vt.sb + hk * c8.vt.sh;
    TileCopy<DT, ND, 32, 256> kc, vc;
    float ks = 1.0f, vs = 1.0f, next_ks = 1.0f, next_vs = 1.0f;
    const int group_row = tid / W::GROUPS, group = tid % W::GROUPS;
    const bool takes = (W::N >= 256 || tid < W::N) && group * 16 < a.D;
    auto fetch = [&](int t) {
        const int key0 = t * 32;
        if (key0 < whole) {
            kc.r[0] = RowView(kbase + key0 * a.k.ss, (int)a.k.ss, 32, 32, a.D)
                          .load(takes ? group_row * (int)a.k.ss + group * 16 : kOutside);
            vc.r[0] = RowView(vbase + key0 * a.v.ss, (int)a.v.ss, 32, 32, a.D)
                          .load(takes ? group_row * (int)a.v.ss + group * 16 : kOutside);
            next_ks = scale_of(c8.ks, b, key0 >> c8.block_log, hk);
            next_vs = scale_of(c8.vs, b, key0 >> c8.block_log, hk);
        } else {
            const int at = key0 - whole;
            kc.fetch(ktail + at * c8.kt.ss, (int)c8.kt.ss, Lk - key0, a.D, tid);
            vc.fetch(vtail + at * c8.vt.ss, (int)c8.vt.ss, Lk - key0, a.D, tid);
            next_ks = next_vs = 1.0f;
        }
    };
    auto put = [&](int t, int to) {
        if (t * 32 < whole) {
            if (W::N >= 256 || tid < W::N) {
                W::put(lds[to][0], group_row, group, kc.r[0]);
                W::put(lds[to][1], group_row, group, vc.r[0]);
            }
        } else {
            kc.put(lds[to][0], tid);
            vc.put(lds[to][1], tid);
        }
        ks = next_ks, vs = next_vs;
    };
    if (t0 < t1) {
        fetch(t0);
        put(t0, 0);
    }
    __syncthreads();
    int cur = 0;
    for (int t = t0; t < t1; ++t, cur ^= 1) {
        const bool more = t + 1 < t1;
        if (more) fetch(t + 1);
        const int rb = opaque(row_base<DT, ND>()), tb = opaque(trans_base<DT, ND>());
        const int key0 = t * 32;
        if (key0 < wr.end && key0 + 32 > wr.begin) {
            const bool part = key0 < wr.all_lo || key0 + 32 > wr.all_hi;
            f32x16 s{};
#pragma unroll
            for (int i = 0; i < T::NS; ++i) s = mma_step<DT>(row_operand<DT, ND>(lds[cur][0], 0, rb, i), qf[i], s);
            settle<DT>(s);
            if (part) mask_block(s, key0, mine);
            softmax_update<ND>(s, c * ks, st, acc);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] *= vs;
            Packed<DT> p;
            p.set(s);
            trans_product<DT, ND, true, SAFE>(lds[cur][1], 0, tb, p, part, key0, mine, acc);
        }
        if (more) put(t + 1, cur ^ 1);
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
__global__ __launch_bounds__(256, DT == DT_BF16 ? 3 : 1) void attention8_kernel(AttnArgs a, Cache8Args c, int row_tiles) {
    __shared__ __attribute__((aligned(16))) Rows8Shared<DT, ND> shared;
    attention8_rows<DT, ND, false>(a, c, blockIdx.x, row_tiles, shared);
}

template <int DT, int ND>
__global__ __launch_bounds__(256, 1) void attention8_again_kernel(AttnArgs a, Cache8Args c, int row_tiles, int items) {
    __shared__ __attribute__((aligned(16))) Rows8Shared<DT, ND> shared;
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
        [&](int id) { attention8_rows<DT, ND, true>(a, c, __builtin_amdgcn_readfirstlane(id), row_tiles, shared); });
}

// ----------------------------------------------------------------- few rows

// At most 32 rows (single tokens), as attention_few: every wave takes 32-key
// tiles of its own.  A lane reads 16 bytes of one key, 16 elements, which are
// the operands of 16 / per16 steps in an order that the queries share.  Tiles
// are counted from the block of 32 of the first key that a row sees; values
// before that key, and past the last, are read as zeros.
template <int DT, int ND, bool SAFE>
__device__ __forceinline__ void attention8_few(const AttnArgs& a, const Cache8Args& c8, int id, FewShared<DT, ND>& shared) {
    using T = Tile<DT, ND>;
    using W = Wide<DT, ND>;
    constexpr int VT = FewShared<DT, ND>::VT;
    const int l = threadIdx.x & 63, wave = wave_id(), half = l >> 5;

    const WorkItem w = work_item(id, a.B * a.Hkv, a.nsplit, false);
    const int split = w.item, b = w.head / a.Hkv, hk = w.head % a.Hkv;
    const int Lq = valid_length(a.q_len, b, a.Sq), Lk = valid_length(a.kv_len, b, a.Sk), whole = whole_blocks(c8, Lk);
    const int rows = a.Sq * a.G;
    const int row = l & 31, pos = row / a.G, head = hk * a.G + row % a.G;
    const bool live = row < rows;
    KeyRange mine = key_range(a, live ? pos : Lq, Lq, Lk);
    if (mine.hi < mine.lo) mine.hi = mine.lo;
    const RowsRange br = rows_range(a, 0, rows, rows, Lq, Lk);
    const int first = br.begin & ~31, n = br.end > br.begin ? (br.end - first + 31) / 32 : 0;
    const int per = (n + a.nsplit - 1) / a.nsplit, p0 = split * per, p1 = p0 + per < n ? p0 + per : n;
    const int eight = whole > first ? (whole - first) / 32 : 0;  // tiles in 8 bits
    const int p8 = p1 < eight ? p1 : eight;

    const char* kbase = a.k.p + b * a.k.sb + hk * a.k.sh;
    const char* vbase = a.v.p + b * a.v.sb + hk * a.v.sh;
    // element of vector i of a row's operand
    auto element = [&](int i) { return (2 * (i / W::PER) + half) * 16 + (i % W::PER) * T::PE; };
    uint4 qf[T::NS];
    const char* q = a.q.p + b * a.q.sb + pos * a.q.ss + head * a.q.sh;
#pragma unroll
    for (int i = 0; i < T::NS; ++i) {
        const int e = element(i);
        qf[i] = make_uint4(0, 0, 0, 0);
        if (live && pos < Lq && e < a.D) qf[i] = *reinterpret_cast<const uint4*>(q + e * T::ES);
    }
    if (a.scale < 0.0f)
#pragma unroll
        for (int s = 0; s < T::NS; ++s) qf[s] = negate16<DT>(qf[s]);
    arrived(qf);
    const float c = score_factor(a.scale);
    f32x16 acc[ND];
#pragma unroll
    for (int db = 0; db < ND; ++db) acc[db] = f32x16{};
    Running st{-INFINITY, 0.0f};
    char* vt = shared.lds + wave * VT;

    auto consume = [&](f32x16& s, int key0, float ks, float vs) {
        const bool part = key0 < br.all_lo || key0 + 32 > br.all_hi;
        if (part) mask_block(s, key0, mine);
        softmax_update<ND>(s, c * ks, st, acc);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= vs;
        Packed<DT> p;
        p.set(s);
        trans_product<DT, ND, true, SAFE>(vt, 0, opaque(trans_base<DT, ND>()), p, part, key0, mine, acc);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };

    uint4 kr[ND], vr[ND];
    float ks = 0.0f, vs = 0.0f;
    auto fetch = [&](int key0) {
        const RowView kv(kbase + key0 * a.k.ss, (int)a.k.ss, 32, 32, a.D), vv(vbase + key0 * a.v.ss, (int)a.v.ss, 32, 32, a.D);
#pragma unroll
        for (int j = 0; j < ND; ++j) {
            const int g = 2 * j + half;
            kr[j] = kv.load(g * 16 < a.D ? row * (int)a.k.ss + g * 16 : kOutside);
        }
#pragma unroll
        for (int j = 0; j < ND; ++j) {
            const int at = l + 64 * j, r = at / W::GROUPS, g = at % W::GROUPS;
            vr[j] = vv.load(g * 16 < a.D && key0 + r >= br.begin ? r * (int)a.v.ss + g * 16 : kOutside);
        }
        ks = scale_of(c8.ks, b, key0 >> c8.block_log, hk);
        vs = scale_of(c8.vs, b, key0 >> c8.block_log, hk);
    };
    int t = p0 + wave;
    if (t < p8) fetch(first + t * 32);
    for (; t < p8; t += 4) {
        const int key0 = first + t * 32;
        f32x16 s{};
#pragma unroll
        for (int j = 0; j < ND; ++j) {
            uint4 kf[W::PER];
            widen16<DT>(kr[j], kf);
#pragma unroll
            for (int i = 0; i < W::PER; ++i) s = mma_step<DT>(kf[i], qf[W::PER * j + i], s);
        }
        settle<DT>(s);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < ND; ++j) {
            const int at = l + 64 * j;
            W::put(vt, at / W::GROUPS, at % W::GROUPS, vr[j]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const float k_now = ks, v_now = vs;
        if (t + 4 < p8) fetch(key0 + 128);
        consume(s, key0, k_now, v_now);
    }
    for (; t < p1; t += 4) {  // the tail: at most one tile a wave
        const int key0 = first + t * 32, at = key0 - whole;
        const RowView kv(c8.kt.p + b * c8.kt.sb + hk * c8.kt.sh + at * c8.kt.ss, (int)c8.kt.ss, Lk - key0, 32, a.D * T::ES);
        const char* vtail = c8.vt.p + b * c8.vt.sb + hk * c8.vt.sh + at * c8.vt.ss;
        const RowView vv(vtail, (int)c8.vt.ss, Lk - key0, 32, a.D * T::ES);
        f32x16 s{};
        uint4 kf[T::NS];
#pragma unroll
        for (int i = 0; i < T::NS; ++i) {
            const int e = element(i);
            kf[i] = kv.load(e < a.D ? row * (int)c8.kt.ss + e * T::ES : kOutside);
        }
#pragma unroll
        for (int i = 0; i < T::NS; ++i) s = mma_step<DT>(kf[i], qf[i], s);
        settle<DT>(s);
        __builtin_amdgcn_wave_barrier();
#pragma unroll 4
        for (int i = 0; i < 32 * T::CPR / 64; ++i) {
            const int id2 = l + 64 * i, r = id2 / T::CPR, g = id2 % T::CPR;
            const uint4 v = vv.load(g * T::PE < a.D && key0 + r >= br.begin ? r * (int)c8.vt.ss + g * 16 : kOutside);
            *reinterpret_cast<uint4*>(vt + T::offset(r, g)) = v;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        consume(s, key0, 1.0f, 1.0f);
    }

#pragma unroll
    for (int db = 0; db < ND; ++db) settle<DT>(acc[db]);
    const bool marked = !SAFE && a.hides && !sums_finite<ND>(acc);
    join_waves<DT, ND>(a, shared, acc, st, marked, b, hk, split);
}

template <int DT, int ND>
__global__ __launch_bounds__(256, DT == DT_BF16 ? 2 : 1) void attention8_few_kernel(AttnArgs a, Cache8Args c) {
    __shared__ __attribute__((aligned(16))) FewShared<DT, ND> shared;
    attention8_few<DT, ND, false>(a, c, blockIdx.x, shared);
}

template <int DT, int ND>
__global__ __launch_bounds__(256, 1) void attention8_few_again_kernel(AttnArgs a, Cache8Args c, int items) {
    __shared__ __attribute__((aligned(16))) FewShared<DT, ND> shared;
    each_marked(
        items,
        [&](int id) {
            const WorkItem w = work_item(id, a.B * a.Hkv, a.nsplit, false);
            return is_marked(a, w, 0, w.item);
        },
        [&](int id) { attention8_few<DT, ND, true>(a, c, __builtin_amdgcn_readfirstlane(id), shared); });
}

int attention8_splits(int64_t B, int64_t Sq, int64_t Sk, int64_t Hkv, int64_t G, bool lengths, int num_cus) {
    return attention_splits(B, Sq, Sk, Hkv, G, lengths, num_cus);
}

template <int DT, int ND>
static void launch_attention8(const AttnArgs& a, const Cache8Args& c, hipStream_t st) {
    const int64_t rows = (int64_t)a.Sq * a.G, tiles = rows <= kFewRows ? 1 : (rows + 127) / 128;
    const int items = (int)((int64_t)a.B * a.Hkv * tiles * a.nsplit);
    const dim3 grid((unsigned)items), again((unsigned)std::min(items, a.num_cus));
    if (rows <= kFewRows) {
        hipLaunchKernelGGL((attention8_few_kernel<DT, ND>), grid, dim3(256), 0, st, a, c);
        if (a.hides) hipLaunchKernelGGL((attention8_few_again_kernel<DT, ND>), again, dim3(256), 0, st, a, c, items);
    } else {
        hipLaunchKernelGGL((attention8_kernel<DT, ND>), grid, dim3(256), 0, st, a, c, (int)tiles);
        if (a.hides) hipLaunchKernelGGL((attention8_again_kernel<DT, ND>), again, dim3(256), 0, st, a, c, (int)tiles, items);
    }
    if (a.nsplit > 1) launch_attention_join(a, DT, st);
}

hipError_t run_attention8(const AttnArgs& a, const Cache8Args& c, int dtype, hipStream_t st) {
    const int nd = (a.D + 31) / 32;
#define PAMM_CASE(DT, ND) \
    if (dtype == DT && nd == ND) launch_attention8<DT, ND>(a, c, st)
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
