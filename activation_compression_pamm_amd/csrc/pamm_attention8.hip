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
#include <type_traits>

#include "pamm_attention_forward.hpp"
#include "pamm_cache_kernels.hpp"

namespace pamm {

// 16 8-bit floats as 16 / per16 vectors of the type, bf16 times a power of two; exact.
template <int DT>
__device__ __forceinline__ void widen16(const uint4& r, uint4* out, float power = 1.0f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (DT == DT_BF16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                u[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * i + j], power, false));
                u[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * i + j], power, true));
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
    __device__ static __forceinline__ void put(char* tile, int r, int c, const uint4& raw, float power = 1.0f) {
        uint4 v[PER];
        widen16<DT>(raw, v, power);
#pragma unroll
        for (int i = 0; i < PER; ++i) *reinterpret_cast<uint4*>(tile + T::offset(r, PER * c + i)) = v[i];
    }
};

// The scales of 64 tiles to come, one a lane, from which each tile's are read
// into scalar registers.  Loaded tile by tile, a scale on its way is copied to
// where the current one was at the loop's end, and that copy waits for all loads.
struct TileScales {
    float v;
    __device__ __forceinline__ void load(const ScalesArg& s, int b, int h, int block, bool ok) {
        v = ok ? s.p[b * s.sb + h * s.sh + (int64_t)block * s.ss] : 1.0f;  // the tail's
    }
    // waits for them here and not, with all loads since, where they are used
    __device__ __forceinline__ void arrived() { asm volatile("" : "+v"(v)); }
    __device__ __forceinline__ float at(int i) const {
        return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), i));
    }
};

// What a tile's scores are multiplied by: never 0, with which a masked score would be a NaN.
__device__ __forceinline__ float tile_factor(float c, float kscale) { return fmaxf(c * kscale, 0x1p-126f); }

// The values' scales of 64 tiles as many rows take them in bf16: 2^k m, with 1 <= m < 2.  2^k goes
// to the values as they are widened, exactly; the logarithm of m to the exponent of the
// probabilities (one addition a tile instead of 16 multiplications, 4% of the time), whose sum is
// turned back by 1 / m.  So bf16 rounds in relation to each probability, however small it
// is beside the largest (a key that draws nearly all of the weight may have values of 0).
struct TileExponents {
    TileScales power, exponent, inverse;
    __device__ __forceinline__ void load(const ScalesArg& s, int b, int h, int block, bool ok) {
        power.load(s, b, h, block, ok);
    }
    __device__ __forceinline__ void arrived() {
        power.arrived();
        const uint32_t v = __float_as_uint(power.v);
        const float m = __uint_as_float((v & 0x7fffffu) | 0x3f800000u);
        power.v = __uint_as_float(v & 0x7f800000u);
        exponent.v = __builtin_amdgcn_logf(m);
        inverse.v = __builtin_amdgcn_rcpf(m);
    }
};

// The start of the tail.
__device__ __forceinline__ int whole_blocks(const Cache8Args& c, int Lk) { return Lk >> c.block_log << c.block_log; }

// ---------------------------------------------------------------- many rows

// As attention_rows: four waves of 32 rows share tiles of 32 keys in two LDS
// buffers, the next tile under way in registers.  Widening takes 16 conversions a
// thread and tile.
//
// In bf16 each probability is rounded once, as in attention.  2 x 512 queries over
// 8192 keys, 32/8 heads of 128: 165 to 170 us a call, box to box.  Beside 170: two bf16
// parts a probability, as few rows have them, 227; probabilities in fp16 178, and no bound
// to what they lose once they are below fp16's range.
//
// The softmax of a tile and its probabilities times the values' scale, in the
// exponent, from which the sum is turned back; otherwise as softmax_update.
template <int ND>
__device__ __forceinline__ void softmax_update8(f32x16& s, float f, float exponent, float inverse, Running& st, f32x16* acc) {
    const float top = largest(s) * f;
    if (__any(top > st.m + kSlack)) {
        const float m = fmaxf(st.m, top), g = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
        st.l *= g;
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[db][i] *= g;
        st.m = m;
    }
    const float from = exponent - (st.m == -INFINITY ? 0.0f : st.m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], f, from));
        sum += s[i];
    }
    st.l = fmaf(sum, inverse, st.l);
}

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

    const char* kbase = a.k.p + b * a.k.sb + hk * a.k.sh;
    const char* vbase = a.v.p + b * a.v.sb + hk * a.v.sh;
    TileScales ks, vs;     // fp32
    TileExponents ve;      // bf16
    int base = t0;         // the tile of the first lane's scales
    auto scales = [&](int t) {
        const int at = (t + l) * 32;
        ks.load(c8.ks, b, hk, at >> c8.block_log, at < whole);
        if constexpr (DT == DT_BF16)
            ve.load(c8.vs, b, hk, at >> c8.block_log, at < whole);
        else
            vs.load(c8.vs, b, hk, at >> c8.block_log, at < whole);
        base = t;
    };
    auto scales_arrived = [&] {
        ks.arrived();
        if constexpr (DT == DT_BF16)
            ve.arrived();
        else
            vs.arrived();
    };
    // the softmax of a tile, its probabilities times the values' scale (in bf16 but for the power of two)
    auto softmax = [&](f32x16& s, int t) {
        const float f = tile_factor(c, ks.at(t - base));
        if constexpr (DT == DT_BF16) {
            softmax_update8<ND>(s, f, ve.exponent.at(t - base), ve.inverse.at(t - base), st, acc);
        } else {  // whose precision the exponent's rounding would reach
            softmax_update<ND>(s, f, st, acc);
            const float vscale = vs.at(t - base);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] *= vscale;
        }
    };
    auto scores = [&](const char* keys, int key0, bool part) {
        const int rb = opaque(row_base<DT, ND>());
        f32x16 s{};
#pragma unroll
        for (int i = 0; i < T::NS; ++i) s = mma_step<DT>(row_operand<DT, ND>(keys, 0, rb, i), qf[i], s);
        settle<DT>(s);
        if (part) mask_block(s, key0, mine);
        return s;
    };

    // the tiles in 8 bits
    const int group_row = tid / W::GROUPS, group = tid % W::GROUPS;
    const bool takes = (W::N >= 256 || tid < W::N) && group * 16 < a.D;
    const int kat = takes ? group_row * (int)a.k.ss + group * 16 : kOutside;
    const int vat = takes ? group_row * (int)a.v.ss + group * 16 : kOutside;
    const int te = SAFE ? t0 : whole / 32 < t0 ? t0 : whole / 32 < t1 ? whole / 32 : t1;
    uint4 kr, vr;
    auto fetch = [&](int t) {
        const int key0 = t * 32, some = t < te ? 32 : 0;
        kr = RowView(kbase + key0 * a.k.ss, (int)a.k.ss, some, 32, a.D).load(kat);
        vr = RowView(vbase + key0 * a.v.ss, (int)a.v.ss, some, 32, a.D).load(vat);
    };
    auto put = [&](int to, int t) {
        if (W::N < 256 && tid >= W::N) return;
        W::put(lds[to][0], group_row, group, kr);
        W::put(lds[to][1], group_row, group, vr, DT == DT_BF16 ? ve.power.at(t - base) : 1.0f);
    };
    if (t0 < te) {
        scales(t0);
        fetch(t0);
        scales_arrived();
        put(0, t0);
        __syncthreads();
    }
    int cur = 0;
    for (int t = t0; t < te; ++t, cur ^= 1) {
        fetch(t + 1);
        const int key0 = t * 32;
        if (key0 < wr.end && key0 + 32 > wr.begin) {
            const bool part = key0 < wr.all_lo || key0 + 32 > wr.all_hi;
            f32x16 s = scores(lds[cur][0], key0, part);
            softmax(s, t);
            const int tb = opaque(trans_base<DT, ND>());
            Packed<DT> p;
            p.set(s);
            trans_product<DT, ND, true, false>(lds[cur][1], 0, tb, p, part, key0, mine, acc);
        }
        if (t + 1 < te) {
            if (t + 1 - base > 63) {
                scales(t + 1);
                scales_arrived();
            }
            put(cur ^ 1, t + 1);
        }
        __syncthreads();
    }

    // the tail, with SAFE all of it: one tile at a time
    for (int t = te, first = 1; t < t1; ++t, first = 0) {
        const int in = (t - t0) & 63, key0 = t * 32;
        if (first || in == 0) {
            scales(t - in);
            scales_arrived();
        }
        const bool eight = SAFE && key0 < whole;
        __syncthreads();
        if (eight) {
            if (W::N >= 256 || tid < W::N) {
                const uint4 k = RowView(kbase + key0 * a.k.ss, (int)a.k.ss, 32, 32, a.D).load(kat);
                const uint4 v = RowView(vbase + key0 * a.v.ss, (int)a.v.ss, 32, 32, a.D).load(vat);
                W::put(lds[0][0], group_row, group, k);
                W::put(lds[0][1], group_row, group, v, DT == DT_BF16 ? ve.power.at(t - base) : 1.0f);
            }
        } else {
            const int at = key0 - whole;
            TileCopy<DT, ND, 32, 256> copy;
            copy.fetch(c8.kt.p + b * c8.kt.sb + hk * c8.kt.sh + at * c8.kt.ss, (int)c8.kt.ss, Lk - key0, a.D, tid);
            copy.put(lds[0][0], tid);
            copy.fetch(c8.vt.p + b * c8.vt.sb + hk * c8.vt.sh + at * c8.vt.ss, (int)c8.vt.ss, Lk - key0, a.D, tid);
            copy.put(lds[0][1], tid);
        }
        __syncthreads();
        if (key0 >= wr.end || key0 + 32 <= wr.begin) continue;
        const bool part = key0 < wr.all_lo || key0 + 32 > wr.all_hi;
        f32x16 s = scores(lds[0][0], key0, part);
        softmax(s, t);
        Packed<DT> p;
        p.set(s);
        trans_product<DT, ND, true, SAFE>(lds[0][1], 0, opaque(trans_base<DT, ND>()), p, part, key0, mine, acc);
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
__global__ __launch_bounds__(256, DT == DT_BF16 ? (ND <= 2 ? 4 : 3) : 1) void attention8_kernel(AttnArgs a, Cache8Args c, int row_tiles) {
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

    // `tail`: the values are not in 8 bits
    auto consume = [&](f32x16& s, int key0, float ks, float vs, auto tail) {
        const bool part = key0 < br.all_lo || key0 + 32 > br.all_hi;
        if (part) mask_block(s, key0, mine);
        softmax_update<ND>(s, tile_factor(c, ks), st, acc);
        Packed<DT> p;
        f32x16 rest;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= vs;
        p.set(s);
        trans_product<DT, ND, true, SAFE>(vt, 0, opaque(trans_base<DT, ND>()), p, part, key0, mine, acc);
        if constexpr (DT == DT_BF16) {  // what bf16 left of them: the matrix unit is idle otherwise
#pragma unroll
            for (int i = 0; i < 16; ++i) rest[i] = s[i] - (float)p.v[i >> 3][i & 7];
            p.set(rest);
            // 8 bits have no infinities, a tail may; times what may be 0 they would be NaNs
            if constexpr (decltype(tail)::value)
                finite_product<DT, ND>(vt, 0, trans_base<DT, ND>(), p, acc);
            else
                trans_product<DT, ND, true, SAFE>(vt, 0, opaque(trans_base<DT, ND>()), p, part, key0, mine, acc);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };

    uint4 kr[ND], vr[ND];
    TileScales ks, vs;
    auto fetch = [&](int t) {
        const int key0 = first + t * 32, some = t < p8 ? 32 : 0;
        const RowView kv(kbase + key0 * a.k.ss, (int)a.k.ss, some, 32, a.D);
        const RowView vv(vbase + key0 * a.v.ss, (int)a.v.ss, some, 32, a.D);
#pragma unroll
        for (int j = 0; j < ND; ++j) {
            const int g = 2 * j + half;
            kr[j] = kv.load_once(g * 16 < a.D ? row * (int)a.k.ss + g * 16 : kOutside);
        }
#pragma unroll
        for (int j = 0; j < ND; ++j) {
            const int at = l + 64 * j, r = at / W::GROUPS, g = at % W::GROUPS;
            vr[j] = vv.load_once(g * 16 < a.D && key0 + r >= br.begin ? r * (int)a.v.ss + g * 16 : kOutside);
        }
    };
    // those of this wave's next 64 tiles
    auto scales = [&](int t) {
        const int mine = t + 4 * l, block = (first + mine * 32) >> c8.block_log;
        ks.load(c8.ks, b, hk, block, mine < p8);
        vs.load(c8.vs, b, hk, block, mine < p8);
    };
    int t = p0 + wave;
    scales(t);
    fetch(t);
    ks.arrived(), vs.arrived();
    for (int nth = 0; t < p8; t += 4, ++nth) {
        const int key0 = first + t * 32;
        if (nth == 64) {
            scales(t);
            ks.arrived(), vs.arrived();
            nth = 0;
        }
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
        fetch(t + 4);
        consume(s, key0, ks.at(nth), vs.at(nth), std::false_type{});
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
        consume(s, key0, 1.0f, 1.0f, std::true_type{});
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

// ------------------------------------------------------------ at most 16 rows

// Single tokens whose key/value heads are shared by up to 16 query heads: 16 x 16
// products, which take half the registers, exponentials and matrix cycles of the
// 32 x 32 ones.
//
// Bound by reading the cache.  64 sequences of 64 to 8192 keys, 8 heads of 128, 0.56
// GB: 101 us a call, the join included (5.5 TB/s); all of 8192, 1.07 GB: 160 us in one part (6.7
// TB/s), in fp32 (ragged) 209.  bf16 with three waves a SIMD; four spill, and a reload in the loop waits for
// all loads (124 and 205 us).  Without the hint that lines are read once the loads alone take 16% more
// (193 us for 167).  With the 32 x 32 products and two waves a SIMD 125 us.
//
// A lane holds row (A) or column (B) l % 16 of a product and the 16-byte vector
// of quarter l / 16 of each step; result element i is D[4 (l / 16) + i][l % 16].
template <int DT>
__device__ __forceinline__ f32x4 mma16_step(const uint4& a, const uint4& b, f32x4 c) {
    if constexpr (DT == DT_BF16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    } else {
        const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[j], y[j], c, 0, 0, 0);
        return c;
    }
}

// 8 8-bit floats as an operand of products over keys.
typedef float Eight __attribute__((ext_vector_type(8)));
template <int DT>
__device__ __forceinline__ auto widen8(uint32_t a, uint32_t b) {
    if constexpr (DT == DT_BF16) {
        const uint4 v = make_uint4(
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true)));
        return __builtin_bit_cast(bf16x8, v);
    } else {
        Eight x;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(i ? b : a, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(i ? b : a, true);
            x[4 * i] = lo[0], x[4 * i + 1] = lo[1], x[4 * i + 2] = hi[0], x[4 * i + 3] = hi[1];
        }
        return x;
    }
}

// As settle(): results are waited for before any branch (7 wait states after the
// bf16 product, 11 after the fp32 one).
__device__ __forceinline__ void settle16(f32x4& d) { asm volatile("s_nop 11" : "+v"(d)); }

// v of the four lanes that hold a column, in each.
template <typename F>
__device__ __forceinline__ float quarters(float v, F&& f) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return f(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// A tile of 32 keys or values as it lies in memory, rows PITCH bytes apart: group
// g of row r at slot g ^ key(r).  Sixteen rows read at one group (keys), and the
// eight rows of a transposing read (values), fall into different banks as far as
// their bytes fill a line of 256.
template <int ND>
struct Raw {
    static constexpr int GROUPS = ND == 1 ? 2 : ND == 2 ? 4 : 8, PITCH = 16 * GROUPS, SIZE = 32 * PITCH;
    static constexpr int LOADS = GROUPS / 2;  // 16 bytes a lane
    __device__ static __forceinline__ int offset(int r, int g) {
        return r * PITCH + ((g ^ (r / (256 / PITCH) % GROUPS)) << 4);
    }
};

template <int DT, int ND>
struct OneShared {
    static constexpr int OP = ND * 32 + 4;  // floats between rows of a wave's result
    static constexpr int most(int a, int b) { return a > b ? a : b; }
    // of each wave: keys and values in 8 bits, a tile of the tail's values, the result
    static constexpr int SLOT = most(most(2 * Raw<ND>::SIZE, 32 * Tile<DT, ND>::PITCH), 16 * OP * 4);
    char lds[4 * SLOT];
    float stat[4][2][16];
};

template <int DT, int ND>
__device__ __forceinline__ void attention8_one(const AttnArgs& a, const Cache8Args& c8, int id, OneShared<DT, ND>& shared) {
    using T = Tile<DT, ND>;
    using W = Wide<DT, ND>;
    using R = Raw<ND>;
    constexpr int NJ = (ND + 1) / 2, NB = 2 * ND;  // groups of a key's row in a lane, blocks of 16 elements
    const int tid = threadIdx.x, l = tid & 63, wave = wave_id(), quarter = l >> 4;

    const WorkItem w = work_item(id, a.B * a.Hkv, a.nsplit, false);
    const int split = w.item, b = w.head / a.Hkv, hk = w.head % a.Hkv;
    const int Lq = valid_length(a.q_len, b, a.Sq), Lk = valid_length(a.kv_len, b, a.Sk), whole = whole_blocks(c8, Lk);
    const int rows = a.Sq * a.G;
    const int row = l & 15, pos = row / a.G, head = hk * a.G + row % a.G;
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
    auto element = [&](int i) { return (4 * (i / W::PER) + quarter) * 16 + (i % W::PER) * T::PE; };
    char* vt = shared.lds + wave * OneShared<DT, ND>::SLOT;

    // Whole lines of a tile a load, which go through LDS: an operand's own 16 bytes of each key would take
    // half a line a load, and with the hint for what is read once be fetched twice (127 us instead of 114 in
    // the case above, both with spills).
    // Loads are issued in any case, past the last tile out of bounds: where a branch may leave
    // them out, the next wait is for every load instead of the oldest ones.
    uint4 kr[R::LOADS], vr[R::LOADS];
    TileScales ks, vs;
    auto fetch = [&](int t) {
        const int key0 = first + t * 32, some = t < p8 ? 32 : 0;
        const RowView kv(kbase + key0 * a.k.ss, (int)a.k.ss, some, 32, a.D);
        const RowView vv(vbase + key0 * a.v.ss, (int)a.v.ss, some, 32, a.D);
#pragma unroll
        for (int j = 0; j < R::LOADS; ++j) {
            const int at = l + 64 * j, r = at / R::GROUPS, g = at % R::GROUPS;
            kr[j] = kv.load_once(g * 16 < a.D ? r * (int)a.k.ss + g * 16 : kOutside);
        }
#pragma unroll
        for (int j = 0; j < R::LOADS; ++j) {
            const int at = l + 64 * j, r = at / R::GROUPS, g = at % R::GROUPS;
            vr[j] = vv.load_once(g * 16 < a.D && key0 + r >= br.begin ? r * (int)a.v.ss + g * 16 : kOutside);
        }
    };
    auto put = [&] {
#pragma unroll
        for (int j = 0; j < R::LOADS; ++j) {
            const int at = l + 64 * j, to = R::offset(at / R::GROUPS, at % R::GROUPS);
            *reinterpret_cast<uint4*>(vt + to) = kr[j];
            *reinterpret_cast<uint4*>(vt + R::SIZE + to) = vr[j];
        }
    };
    // those of this wave's next 64 tiles
    auto scales = [&](int t) {
        const int mine = t + 4 * l, block = (first + mine * 32) >> c8.block_log;
        ks.load(c8.ks, b, hk, block, mine < p8);
        vs.load(c8.vs, b, hk, block, mine < p8);
    };
    int t = p0 + wave;
    scales(t);
    fetch(t);
    uint4 qf[NJ * W::PER];
    const char* q = a.q.p + b * a.q.sb + pos * a.q.ss + head * a.q.sh;
#pragma unroll
    for (int i = 0; i < NJ * W::PER; ++i) {
        const int e = element(i);
        qf[i] = make_uint4(0, 0, 0, 0);
        if (live && pos < Lq && e < a.D) qf[i] = *reinterpret_cast<const uint4*>(q + e * T::ES);
    }
    if (a.scale < 0.0f)
#pragma unroll
        for (int i = 0; i < NJ * W::PER; ++i) qf[i] = negate16<DT>(qf[i]);
    ks.arrived(), vs.arrived();
    const float c = score_factor(a.scale);
    f32x4 acc[NB];
#pragma unroll
    for (int db = 0; db < NB; ++db) acc[db] = f32x4{};
    Running st{-INFINITY, 0.0f};

    // the softmax of a tile's scores: probabilities times the values' scale
    auto softmax = [&](f32x4 (&s)[2], float (&p)[8], int key0, float kscale, float vscale) {
        if (key0 < br.all_lo || key0 + 32 > br.all_hi)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t k = (uint32_t)(key0 + 16 * kb + 4 * quarter + i - mine.lo);
                    if (k >= (uint32_t)(mine.hi - mine.lo)) s[kb][i] = -INFINITY;
                }
        const float f = tile_factor(c, kscale);
        float top = s[0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, s[i >> 2][i & 3]);
        top = quarters(top, [](float x, float y) { return fmaxf(x, y); }) * f;
        if (__any(top > st.m + kSlack)) {
            const float m = fmaxf(st.m, top), g = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
            st.l *= g;
#pragma unroll
            for (int db = 0; db < NB; ++db) acc[db] *= g;
            st.m = m;
        }
        const float ref = st.m == -INFINITY ? 0.0f : st.m;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(fmaf(s[i >> 2][i & 3], f, -ref));
            sum += p[i];
            p[i] *= vscale;
        }
        st.l += sum;
    };
    // acc[db] += 16 columns of the values x p.  Contraction place 8 (l / 16) + i is key
    // 4 (l / 16) + i, 16 more for i >= 4, for both operands.  `tail`: the values are not in 8 bits.
    auto product = [&](int db, const auto& x, const float (&p)[8], auto tail) {
        if constexpr (DT == DT_BF16) {
            bf16x8 pk, rest;  // what bf16 leaves of the probabilities, too: the matrix unit is idle otherwise
#pragma unroll
            for (int i = 0; i < 8; ++i) pk[i] = (__bf16)p[i], rest[i] = (__bf16)(p[i] - (float)pk[i]);
            acc[db] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, pk, acc[db], 0, 0, 0);
            bf16x8 y = x;  // 8 bits have no infinities, a tail may; times what may be 0 they would be NaNs
            if constexpr (decltype(tail)::value)
                y = Columns<DT_BF16, ND>::each(x, [](float e) { return isfinite(e) ? e : 0.0f; });
            acc[db] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y, rest, acc[db], 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[db] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], p[i], acc[db], 0, 0, 0);
        }
    };
    // where this lane's part of the transposing reads lies
    const int vrow = 4 * quarter + ((l & 15) >> 1 & 3) + 16 * ((l & 15) >> 3);
    const int vbase8 = R::SIZE + R::offset(vrow, 0) + (l & 1) * 8, kbase8 = R::offset(row, 0);

    for (int nth = 0; t < p8; t += 4, ++nth) {
        const int key0 = first + t * 32;
        if (nth == 64) {
            scales(t);
            ks.arrived(), vs.arrived();
            nth = 0;
        }
        __builtin_amdgcn_wave_barrier();
        put();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        fetch(t + 4);
        const int kat = opaque(kbase8), vat = opaque(vbase8);
        f32x4 s[2] = {f32x4{}, f32x4{}};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                // rows 16 apart share a key; a quarter's group is 4 j + quarter
                const int slot = 4 * j + quarter;
                uint4 raw = *reinterpret_cast<const uint4*>(vt + 16 * kb * R::PITCH + (kat ^ (slot << 4)));
                if (ND == 1 && quarter > 1) raw = make_uint4(0, 0, 0, 0);  // past the row
                uint4 kf[W::PER];
                widen16<DT>(raw, kf);
#pragma unroll
                for (int i = 0; i < W::PER; ++i) s[kb] = mma16_step<DT>(kf[i], qf[W::PER * j + i], s[kb]);
            }
        settle16(s[0]);
        settle16(s[1]);
        float p[8];
        softmax(s, p, key0, ks.at(nth), vs.at(nth));
#pragma unroll
        for (int db = 0; db < NB; ++db) {
            typedef int i32x2 __attribute__((ext_vector_type(2)));
            typedef __attribute__((address_space(3))) i32x2* lds_i2;
            const i32x2 raw = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i2)(vt + (vat ^ (db << 4))));
            product(db, widen8<DT>(raw[0], raw[1]), p, std::false_type{});
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    for (; t < p1; t += 4) {  // the tail: at most one tile a wave
        const int key0 = first + t * 32, at = key0 - whole;
        const RowView kv(c8.kt.p + b * c8.kt.sb + hk * c8.kt.sh + at * c8.kt.ss, (int)c8.kt.ss, Lk - key0, 32, a.D * T::ES);
        const RowView vv(c8.vt.p + b * c8.vt.sb + hk * c8.vt.sh + at * c8.vt.ss, (int)c8.vt.ss, Lk - key0, 32, a.D * T::ES);
        f32x4 s[2] = {f32x4{}, f32x4{}};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint4 kf[NJ * W::PER];
#pragma unroll
            for (int i = 0; i < NJ * W::PER; ++i) {
                const int e = element(i);
                kf[i] = kv.load(e < a.D ? (16 * kb + row) * (int)c8.kt.ss + e * T::ES : kOutside);
            }
#pragma unroll
            for (int i = 0; i < NJ * W::PER; ++i) s[kb] = mma16_step<DT>(kf[i], qf[i], s[kb]);
        }
        settle16(s[0]);
        settle16(s[1]);
        __builtin_amdgcn_wave_barrier();
#pragma unroll 4
        for (int i = 0; i < 32 * T::CPR / 64; ++i) {
            const int at2 = l + 64 * i, r = at2 / T::CPR, g = at2 % T::CPR;
            const uint4 v = vv.load(g * T::PE < a.D && key0 + r >= br.begin ? r * (int)c8.vt.ss + g * 16 : kOutside);
            *reinterpret_cast<uint4*>(vt + T::offset(r, g)) = v;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        float p[8];
        softmax(s, p, key0, 1.0f, 1.0f);
        const int base = T::offset(4 * quarter + ((l & 15) >> 2), (l & 3) >> 1) + (l & 1) * 8;
#pragma unroll
        for (int db = 0; db < NB; ++db) {
            if constexpr (DT == DT_BF16) {
                typedef __attribute__((address_space(3))) s16x4* lds_s4;
                typedef short s16x8 __attribute__((ext_vector_type(8)));
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(vt + (base ^ (db << 5))));
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(vt + 16 * T::PITCH + (base ^ (db << 5))));
                const s16x8 x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                product(db, __builtin_bit_cast(bf16x8, x), p, std::true_type{});
            } else {
                Eight x;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int key = 16 * (i >> 2) + 4 * quarter + (i & 3), e = 16 * db + row;
                    x[i] = *reinterpret_cast<const float*>(vt + T::offset(key, e >> 2) + (e & 3) * 4);
                }
                product(db, x, p, std::true_type{});
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }

    uint32_t big = 0;
#pragma unroll
    for (int db = 0; db < NB; ++db) {
        settle16(acc[db]);
#pragma unroll
        for (int i = 0; i < 4; ++i) big = max(big, __float_as_uint(acc[db][i]) & 0x7fffffffu);
    }
    const bool marked = a.hides && !__all(big < 0x7f800000u);

    // join the four waves: the common reference first, then the sums in order
    constexpr int OP = OneShared<DT, ND>::OP, SLOT = OneShared<DT, ND>::SLOT;
    const float sum = marked ? NAN : quarters(st.l, [](float x, float y) { return x + y; });
    if (l < 16) {
        shared.stat[wave][0][l] = sum == 0.0f ? -INFINITY : st.m;
        shared.stat[wave][1][l] = sum;
    }
    __syncthreads();
    float m = -INFINITY, total = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, shared.stat[i][0][row]);
    const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < 4; ++i) total += shared.stat[i][1][row] * __builtin_amdgcn_exp2f(shared.stat[i][0][row] - ref);
    const float f = sum == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(st.m - ref) / total;
    if (live)
#pragma unroll
        for (int db = 0; db < NB; ++db) {
            float4 x = make_float4(acc[db][0] * f, acc[db][1] * f, acc[db][2] * f, acc[db][3] * f);
            if (sum == 0.0f) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            *reinterpret_cast<float4*>(vt + (row * OP + 16 * db + 4 * quarter) * 4) = x;
        }
    const float lse2 = total == 0.0f ? -INFINITY : m + __builtin_amdgcn_logf(total);
    const int64_t at = ((int64_t)b * a.H + head) * a.Sq + pos;
    if (tid < 16 && live) {
        if (a.nsplit > 1)
            a.part_lse[at * a.nsplit + split] = lse2;
        else
            a.lse[at] = lse2 * kLn2;
    }
    __syncthreads();
    const int per_row = a.D / 4;
    for (int e = tid; e < rows * per_row; e += 256) {
        const int r = e / per_row, x = (e - r * per_row) * 4, p = r / a.G, h = hk * a.G + r % a.G;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 u = *reinterpret_cast<const float4*>(shared.lds + i * SLOT + (r * OP + x) * 4);
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        if (a.nsplit > 1) {
            *reinterpret_cast<float4*>(a.part_o + ((((int64_t)b * a.H + h) * a.Sq + p) * a.nsplit + split) * a.D + x) = v;
            continue;
        }
        char* o = a.o.p + b * a.o.sb + p * a.o.ss + h * a.o.sh + x * T::ES;
        if constexpr (DT == DT_BF16) {
            bf16x2 y, z;
            y[0] = (__bf16)v.x, y[1] = (__bf16)v.y, z[0] = (__bf16)v.z, z[1] = (__bf16)v.w;
            *reinterpret_cast<uint2*>(o) = make_uint2(__builtin_bit_cast(uint32_t, y), __builtin_bit_cast(uint32_t, z));
        } else {
            *reinterpret_cast<float4*>(o) = v;
        }
    }
}

template <int DT, int ND>
__global__ __launch_bounds__(256, DT == DT_BF16 ? 3 : 2) void attention8_one_kernel(AttnArgs a, Cache8Args c) {
    __shared__ __attribute__((aligned(16))) OneShared<DT, ND> shared;
    attention8_one<DT, ND>(a, c, blockIdx.x, shared);
}

// Few rows: two workgroups a unit, in at most a part for each 1024 keys begun (of the room,
// whatever a window shows of it).  A second launch and the parts' memory cost a call 7 us
// (1 x 1024 keys, 12 heads of 64: 16.9 us whole, 22 to 24 in parts; 8192, 8 heads of 128: 63
// whole, 27 in 4, 25 in 8).  Where lengths are given, which then differ as a rule, eight a unit
// even them out, as long as parts have 2048 keys (64 sequences of up to 8192, 8 heads of 128, side by
// side: 104 us whole, 100 and 98 in 2 and 4, 105 in 8; of up to 2048: 30 whole, 37 in 2; where all have 8192
// after all: 160 whole, 170 in 4).  Many rows are cut as over a cache that is not in 8 bits.
int attention8_splits(int64_t B, int64_t Sq, int64_t Sk, int64_t Hkv, int64_t G, bool lengths, int num_cus) {
    if (Sq * G > kFewRows) return attention_splits(B, Sq, Sk, Hkv, G, lengths, num_cus);
    const int64_t blocks = B * Hkv, units = num_cus;
    if (blocks == 0) return 1;
    int64_t n = std::min((2 * units + blocks - 1) / blocks, (Sk + 1023) / 1024);
    if (lengths) n = std::max(n, std::min((8 * units + blocks - 1) / blocks, Sk / 2048));
    return (int)std::max<int64_t>(1, std::min<int64_t>(n, kMaxSplits));
}

template <int DT, int ND>
static void launch_attention8(const AttnArgs& a, const Cache8Args& c, hipStream_t st) {
    const int64_t rows = (int64_t)a.Sq * a.G, tiles = rows <= kFewRows ? 1 : (rows + 127) / 128;
    const int items = (int)((int64_t)a.B * a.Hkv * tiles * a.nsplit);
    const dim3 grid((unsigned)items), again((unsigned)std::min(items, a.num_cus));
    if (rows <= kFewRows) {
        if (rows <= 16)
            hipLaunchKernelGGL((attention8_one_kernel<DT, ND>), grid, dim3(256), 0, st, a, c);
        else
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
