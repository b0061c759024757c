// pamm_attention_bwd.hip -- attention's backward pass on gfx950.
//
//   P_ij = exp(s_ij - lse_i)          delta_i = <do_i, o_i>
//   dS_ij = P_ij (<do_i, v_j> - delta_i)
//   dv_j = sum_i P_ij do_i,  dk_j = scale sum_i dS_ij q_i,
//   dq_i = scale sum_j dS_ij k_j
//
// The products that form s and <do, v> start from -lse / scale (bf16) and -delta,
// so what comes out needs one multiplication and an exponential to be P, and one
// more multiplication to be dS.  In fp32 s starts from 0 and lse is taken off in
// the exponent: on top of lse / scale each of a score's D / 2 steps is rounded at
// that size, which bf16's own rounding of P hides but fp32's does not (gradients of
// 215 tokens, heads of 96: 1.2e-6 off, from 0 0.5e-6 to 0.6e-6).
//
// Two kinds of workgroup, each with its sums in registers and in a fixed order:
// one owns queries and runs over keys (dq, and delta on the way), one owns keys
// and runs over the queries of every head that shares them (dk, dv).  Forming P
// and dS in both costs 7 products instead of 5, and buys sums without atomics:
// the results are bitwise repeatable and no fp32 copy of dq is kept.
#include <algorithm>

#include "pamm_attention_device.hpp"

namespace pamm {

__device__ __forceinline__ float score_factor(float scale) { return fmaxf(fabsf(scale) * kLog2e, 1e-36f); }

// What takes a row's lse off its scores: bf16 -lse in units of the raw products,
// from which a score starts, so that 2^(c (start + <q, k>)) is the probability;
// fp32 -lse in log2 units, 2^(c <q, k> + start).  A row that saw nothing (lse =
// -infinity) has what makes its probabilities 2^(-infinity) = 0.
template <int DT>
__device__ __forceinline__ float start_of(float lse, float c) {
    if constexpr (DT == DT_BF16)
        return lse == -INFINITY ? (c < 0.0f ? INFINITY : -INFINITY) : -lse * kLog2e / c;
    else
        return lse == -INFINITY ? -INFINITY : -lse * kLog2e;
}
template <int DT>
__device__ __forceinline__ float probability(float s, float c, float start) {
    return __builtin_amdgcn_exp2f(DT == DT_BF16 ? s * c : fmaf(s, c, start));
}

template <int DT>
__device__ __forceinline__ float dot16(const uint4& x, const uint4& y) {
    float u[8], v[8], sum = 0.0f;
    unpack16<DT>(x, u);
    unpack16<DT>(y, v);
#pragma unroll
    for (int i = 0; i < Elem<DT>::per16; ++i) sum = fmaf(u[i], v[i], sum);
    return sum;
}

// delta = <do, o> with o rounded to bf16 is off by 2^-8 |do||o| at random, and
// dS = P (<do, v> - delta) with it; rows that see few keys feel it most.  It is
// also sum_j P_ij <do_i, v_j>: where the first 32 keys of a workgroup are all that
// a wave's rows see, that sum corrects delta (dk of 300 tokens, 8 heads of 64,
// causal: relative error 0.0025 -> 0.0024, of 20 tokens 0.0028 -> 0.0024, where
// the rounding of an exact result is 0.0017 and that of dS as much).  The dq side
// does it before its loop; inside, it cost a tenth.  With a window of up to 32
// keys every row sees few, and the dq side goes over the keys twice (window 8: dq
// and dk 0.0027 -> 0.0024).  So it does without a causal mask where all keys are two
// or three tiles (35 keys, 16/4 heads of 32: 1.52 -> 1.45 times the error of an exact
// result's rounding; 8 x 64 tokens, 12 heads of 64, 17.6 -> 20.2 us for the second
// launch); from 80 keys on the error is below 1.5 times anyway, and causal rows
// start with the first 32 keys, where it counts most.
__device__ __host__ inline bool short_window(const AttnArgs& a) { return a.window > 0 && a.window <= 32; }
constexpr int kFewKeys = 96;
inline bool few_keys(const AttnArgs& a) { return !a.causal && a.Sk > 32 && a.Sk <= kFewKeys; }

// dq.  Laid out as the forward pass: transposed scores, a lane owns a query.
// Tiles of 32 keys, not 64: three waves a SIMD at D = 64 (8 x 1024, 12 heads: 1.7 us
// less) and fewer registers above.  Three products for each pair; bound as the
// forward pass (matrix unit busy 41% of the cycles, vector instructions 35%, waits 35%).
// 4 x 2048 tokens, 32 heads of 128: 248 us, 832 TFLOP/s; 8192, 32/8 of 64: 406 us, 1015.
template <int DT, int ND>
struct DqShared {
    static constexpr int BK = 32;
    char tile[2][2][BK * Tile<DT, ND>::PITCH];
};

template <int DT, int ND, bool ONE, bool SAFE>
__device__ __forceinline__ void attention_dq(const AttnArgs& a, int id, int row_tiles, DqShared<DT, ND>& shared) {
    using T = Tile<DT, ND>;
    constexpr int BK = DqShared<DT, ND>::BK;
    auto& lds = shared.tile;
    const int tid = threadIdx.x, l = tid & 63, wave = wave_id();

    const WorkItem w = work_item(id, a.B * a.Hkv, row_tiles, a.causal);
    const int tile = row_tiles - 1 - w.item, b = w.head / a.Hkv, hk = w.head % a.Hkv;
    const int Lq = valid_length(a.q_len, b, a.Sq), Lk = valid_length(a.kv_len, b, a.Sk);
    const int rows = a.Sq * a.G;
    const int r0 = tile * 128, w0 = r0 + wave * 32, row = w0 + (l & 31);
    const int pos = row / a.G, head = hk * a.G + row % a.G;
    const bool live = row < rows;
    KeyRange mine = key_range(a, live ? pos : Lq, Lq, Lk);
    if (mine.hi < mine.lo) mine.hi = mine.lo;
    const RowsRange wr = rows_range(a, w0, 32, rows, Lq, Lk), br = rows_range(a, r0, 128, rows, Lq, Lk);
    const int t0 = br.begin / BK, t1 = (br.end + BK - 1) / BK;

    const char* kbase = a.k.p + b * a.k.sb + hk * a.k.sh;
    const char* vbase = a.v.p + b * a.v.sb + hk * a.v.sh;
    const bool seen = live && pos < Lq;
    uint4 qf[T::NS], dof[T::NS];
    load_row_operand<DT, ND>(qf, a.o.p + b * a.o.sb + pos * a.o.ss + head * a.o.sh, seen, a.D);
    load_row_operand<DT, ND>(dof, a.dout.p + b * a.dout.sb + pos * a.dout.ss + head * a.dout.sh, seen, a.D);
    float delta = 0.0f;
#pragma unroll
    for (int s = 0; s < T::NS; ++s) delta += dot16<DT>(qf[s], dof[s]);
    delta = half_sum(delta);
    const int64_t at = ((int64_t)b * a.H + head) * a.Sq + pos;
    load_row_operand<DT, ND>(qf, a.q.p + b * a.q.sb + pos * a.q.ss + head * a.q.sh, seen, a.D);
    if (a.scale < 0.0f)
#pragma unroll
        for (int s = 0; s < T::NS; ++s) qf[s] = negate16<DT>(qf[s]);
    arrived(qf);
    arrived(dof);
    const float c = score_factor(a.scale);
    float start = start_of<DT>(live ? a.lse[at] : 0.0f, c);
    asm volatile("" : "+v"(start));  // as for the operands

    TileCopy<DT, ND, BK, 256> kc, vc;
    if (t0 < t1) {
        kc.fetch(kbase + t0 * BK * a.k.ss, (int)a.k.ss, Lk - t0 * BK, a.D, tid);
        vc.fetch(vbase + t0 * BK * a.v.ss, (int)a.v.ss, Lk - t0 * BK, a.D, tid);
        kc.put(lds[0][0], tid);
        vc.put(lds[0][1], tid);
    }
    __syncthreads();
    // delta corrected (see above): all tiles first where a window is short, then the first again
    int cur = 0;
    if constexpr (DT == DT_BF16) {
        const bool whole = !ONE && t1 - t0 > 1 && (short_window(a) || (!a.causal && t1 - t0 <= kFewKeys / BK));
        const int rb = row_base<DT, ND>(), tp = whole ? t1 : t0 + 1;
        float off = 0.0f;
        for (int t = t0; t < tp; ++t) {
            const int next = t + 1 < tp ? t + 1 : t0, key0 = t * BK;
            if (whole) {
                kc.fetch(kbase + next * BK * a.k.ss, (int)a.k.ss, Lk - next * BK, a.D, tid);
                vc.fetch(vbase + next * BK * a.v.ss, (int)a.v.ss, Lk - next * BK, a.D, tid);
            }
            if (wr.begin < wr.end &&
                (whole ? key0 < wr.end && key0 + BK > wr.begin : wr.begin >= key0 && wr.end <= key0 + BK)) {
                f32x16 s = splat(start), dp = splat(-delta);  // bf16
#pragma unroll
                for (int i = 0; i < T::NS; ++i) {
                    s = mma_step<DT>(row_operand<DT, ND>(lds[cur][0], 0, rb, i), qf[i], s);
                    dp = mma_step<DT>(row_operand<DT, ND>(lds[cur][1], 0, rb, i), dof[i], dp);
                }
                settle<DT>(s);
                settle<DT>(dp);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (sees(key0, i, mine)) off += __builtin_amdgcn_exp2f(s[i] * c) * dp[i];
            }
            if (whole) {
                cur ^= 1;
                kc.put(lds[cur][0], tid);
                vc.put(lds[cur][1], tid);
                __syncthreads();
            }
        }
        delta += half_sum(off);
    }
    if (!SAFE && !ONE && live && l < 32) a.delta[at] = delta;
    f32x16 acc[ND];
#pragma unroll
    for (int db = 0; db < ND; ++db) acc[db] = f32x16{};
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
            f32x16 s = splat(DT == DT_BF16 ? start : 0.0f), dp = splat(-delta);
#pragma unroll
            for (int i = 0; i < T::NS; ++i) {
                s = mma_step<DT>(row_operand<DT, ND>(lds[cur][0], kb * 32, rb, i), qf[i], s);
                dp = mma_step<DT>(row_operand<DT, ND>(lds[cur][1], kb * 32, rb, i), dof[i], dp);
            }
            settle<DT>(s);
            settle<DT>(dp);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = probability<DT>(s[i], c, start) * dp[i];
            const bool part = key0 < wr.all_lo || key0 + 32 > wr.all_hi;
            if (part) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!sees(key0, i, mine)) s[i] = 0.0f;
            }
            Packed<DT> ds;
            ds.set(s);
            trans_product<DT, ND, false, SAFE>(lds[cur][0], kb * 32, tb, ds, part, key0, mine, acc);
        }
        if (more) {
            kc.put(lds[cur ^ 1][0], tid);
            vc.put(lds[cur ^ 1][1], tid);
        }
        __syncthreads();
    }
#pragma unroll
    for (int db = 0; db < ND; ++db) settle<DT>(acc[db]);
    if (!SAFE && a.hides) {
        const bool ok = sums_finite<ND>(acc);
        if (l == 0) a.marks[id * 4 + wave] = !ok;
    }
    if (live) store_rows<DT, ND>(a.dq.p + b * a.dq.sb + pos * a.dq.ss + head * a.dq.sh, acc, a.scale, mine.hi == mine.lo, a.D);
}

template <int DT, int ND>
__global__ __launch_bounds__(256, DT == DT_BF16 ? 2 : 1) void attention_dq_kernel(AttnArgs a, int row_tiles) {
    __shared__ __attribute__((aligned(16))) DqShared<DT, ND> shared;
    attention_dq<DT, ND, false, false>(a, blockIdx.x, row_tiles, shared);
}

// dk and dv.  Scores as S = Q K^T: a lane owns a key.  Four waves of 32 keys
// share tiles of 32 queries of one head, head after head.  V stays in
// registers as an operand, K in LDS: both in registers beside 128 sums a lane
// would leave one wave a SIMD, and where registers still do not suffice V's last
// 32-byte steps are kept in LDS (spilled, their reload waited for the next
// tile's loads every time round).  Where there are few key tiles and many queries,
// the queries of a tile are cut into parts whose sums a second kernel joins.
// Four products for each pair; with two waves a SIMD waves wait 42% of their
// cycles and the matrix unit is busy 38%.  4 x 2048 tokens, 32 heads of 128: 339 us,
// 812 TFLOP/s; 8192, 32/8 of 64: 611 us, 900.
template <int DT, int ND>
struct DkvShared {
    static constexpr int BQ = 32;
    static constexpr int VL = DT != DT_BF16 ? 0 : ND == 4 ? 3 : ND == 2 ? 1 : 0;  // steps of V in LDS
    char tile[2][2][BQ * Tile<DT, ND>::PITCH];
    char k[128 * Tile<DT, ND>::PITCH];
    char v[VL ? VL * 128 * 32 : 16];
    float rowstat[2][2][BQ];
};

template <int DT, int ND, bool ONE, bool SAFE>
__device__ __forceinline__ void attention_dkv(const AttnArgs& a, int id, int key_tiles, DkvShared<DT, ND>& shared) {
    using T = Tile<DT, ND>;
    constexpr int BQ = DkvShared<DT, ND>::BQ, VR = T::NS - DkvShared<DT, ND>::VL;
    auto& lds = shared.tile;
    auto& rowstat = shared.rowstat;
    char *ldk = shared.k, *ldv = shared.v;
    const int tid = threadIdx.x, l = tid & 63, wave = wave_id();

    const WorkItem w = work_item(id, a.B * a.Hkv, key_tiles * a.nsplit_kv, a.causal);
    const int tile = w.item / a.nsplit_kv, part_id = w.item % a.nsplit_kv;  // the first keys are seen by the most queries
    const int b = w.head / a.Hkv, hk = w.head % a.Hkv;
    const int Lq = valid_length(a.q_len, b, a.Sq), Lk = valid_length(a.kv_len, b, a.Sk);
    const int off = Lk - Lq;
    const int b0 = tile * 128, w0 = b0 + wave * 32, key = w0 + (l & 31);
    const bool live = key < a.Sk;

    // positions that see some key of the workgroup (of the wave): [p0, p1) ([wp0, wp1))
    int p0 = 0, p1 = b0 < Lk ? Lq : 0, wp0 = 0, wp1 = w0 < Lk ? Lq : 0;
    if (a.causal) {
        if (b0 - off > p0) p0 = b0 - off;
        if (w0 - off > wp0) wp0 = w0 - off;
        if (a.window) {
            const int e = b0 + 127 - off + a.window, we = w0 + 31 - off + a.window;
            if (e < p1) p1 = e;
            if (we < wp1) wp1 = we;
        }
    }
    const int n0 = p0 / BQ;
    int n1 = (p1 + BQ - 1) / BQ;
    if (n1 < n0) n1 = n0;
    const int per_head = n1 - n0;  // heads x tiles fit 32 bits as rows do
    const int per = (per_head * a.G + a.nsplit_kv - 1) / a.nsplit_kv, i0 = part_id * per;
    const int i1 = i0 + per < per_head * a.G ? i0 + per : per_head * a.G;
    // tiles of which this wave holds all keys: as in the dq kernel, delta is corrected
    int one_block = 0;
    if (w0 == 0) {
        // positions that see none but the first 32
        const int end = Lk <= 32 ? Lq : !a.causal ? 0 : 32 - off < Lq ? 32 - off : Lq;
        one_block = end >= Lq ? (Lq + BQ - 1) / BQ : end / BQ;
    }
    // positions that see a key: [lo, hi)
    auto positions = [&](int k) {
        KeyRange r{0, k < Lk ? Lq : 0};
        if (a.causal) {
            if (k - off > 0) r.lo = k - off;
            if (a.window && k - off + a.window < r.hi) r.hi = k - off + a.window;
        }
        if (r.hi < r.lo) r.hi = r.lo;
        return r;
    };

    uint4 vf[T::NS];
    load_row_operand<DT, ND>(vf, a.v.p + b * a.v.sb + key * a.v.ss + hk * a.v.sh, key < Lk, a.D);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        TileCopy<DT, ND, 64, 256> kc;
        kc.fetch(a.k.p + b * a.k.sb + (b0 + 64 * i) * a.k.ss + hk * a.k.sh, (int)a.k.ss, Lk - b0 - 64 * i, a.D, tid);
        kc.put(ldk + 64 * i * T::PITCH, tid);
    }
    arrived(vf);
    char* vl = ldv + (wave * 32 + (l & 31)) * 32 + (l >> 5) * 16;
#pragma unroll
    for (int x = VR; x < T::NS; ++x) *reinterpret_cast<uint4*>(vl + (x - VR) * 128 * 32) = vf[x];
    const float c = score_factor(a.scale) * (a.scale < 0.0f ? -1.0f : 1.0f);

    f32x16 dk[ND], dv[ND];
#pragma unroll
    for (int db = 0; db < ND; ++db) dk[db] = dv[db] = f32x16{};

    using Copy = TileCopy<DT, ND, BQ, 256>;
    Copy qc, oc, rc;  // q, do and, for delta, o
    // Where a row's vectors are no power of two, its sum's come again, LPR threads a row.
    constexpr bool NEIGHBOURS = (T::CPR & (T::CPR - 1)) == 0;
    constexpr int LPR = T::CPR <= 16 ? 16 : 32, RPP = 256 / LPR, PASSES = BQ / RPP;
    uint4 xo[PASSES], xr[PASSES];
    float stat = 0.0f;
    auto fetch = [&](int g, int t) {
        const int head = hk * a.G + g, q0 = t * BQ;
        qc.fetch(a.q.p + b * a.q.sb + head * a.q.sh + q0 * a.q.ss, (int)a.q.ss, Lq - q0, a.D, tid);
        oc.fetch(a.dout.p + b * a.dout.sb + head * a.dout.sh + q0 * a.dout.ss, (int)a.dout.ss, Lq - q0, a.D, tid);
        if constexpr (ONE && NEIGHBOURS) {
            rc.fetch(a.o.p + b * a.o.sb + head * a.o.sh + q0 * a.o.ss, (int)a.o.ss, Lq - q0, a.D, tid);
        } else if constexpr (ONE) {
            const RowView o(a.o.p + b * a.o.sb + head * a.o.sh + q0 * a.o.ss, (int)a.o.ss, Lq - q0, BQ, a.D * T::ES);
            const RowView d(a.dout.p + b * a.dout.sb + head * a.dout.sh + q0 * a.dout.ss, (int)a.dout.ss, Lq - q0, BQ,
                            a.D * T::ES);
            const int row = tid / LPR, x = tid % LPR;
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const int at = row + i * RPP;
                const bool in = x * T::PE < a.D && q0 + at < Lq;
                xr[i] = o.load(in ? at * (int)a.o.ss + x * 16 : kOutside);
                xo[i] = d.load(in ? at * (int)a.dout.ss + x * 16 : kOutside);
            }
        }
        const int r = tid % BQ;
        const int64_t at = ((int64_t)b * a.H + head) * a.Sq + q0 + r;
        stat = 0.0f;
        if (tid < (ONE ? BQ : 2 * BQ) && q0 + r < Lq) stat = tid < BQ ? a.lse[at] : a.delta[at];
    };
    auto put = [&](int buf) {
        qc.put(lds[buf][0], tid);
        oc.put(lds[buf][1], tid);
        if constexpr (ONE && !NEIGHBOURS) {
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                float d = dot16<DT>(xo[i], xr[i]);
#pragma unroll
                for (int m = 1; m < LPR; m <<= 1) d += shfl_xor(d, m);
                if (tid % LPR == 0) rowstat[buf][1][tid / LPR + i * RPP] = -d;
            }
            if (tid < BQ) rowstat[buf][0][tid] = start_of<DT>(stat, c);
        } else if constexpr (ONE) {
            // the threads that copy a row are neighbours
#pragma unroll
            for (int i = 0; i < Copy::PER; ++i) {
                float d = dot16<DT>(oc.r[i], rc.r[i]);
#pragma unroll
                for (int m = 1; m < T::CPR; m <<= 1) d += shfl_xor(d, m);
                const int at = tid + i * 256;
                if (at < Copy::N && at % T::CPR == 0) rowstat[buf][1][at / T::CPR] = -d;
            }
            if (tid < BQ) rowstat[buf][0][tid] = start_of<DT>(stat, c);
        } else if (tid < 2 * BQ) {
            rowstat[buf][tid / BQ][tid % BQ] = tid < BQ ? start_of<DT>(stat, c) : -stat;
        }
    };
    int t = n0, g = 0;
    if (i0 < i1) {
        g = i0 / per_head;
        t = n0 + i0 % per_head;
        fetch(g, t);
        put(0);
    }
    __syncthreads();
    int cur = 0;
    for (int i = i0; i < i1; ++i, cur ^= 1) {
        int tn = t + 1, gn = g;
        if (tn == n1) tn = n0, ++gn;
        if (i + 1 < i1) fetch(gn, tn);
        const int q0 = t * BQ;
        if (q0 < wp1 && q0 + BQ > wp0) {
            const int rb = opaque(row_base<DT, ND>()), tb = opaque(trans_base<DT, ND>());
            const int quad = 4 * (l >> 5);
            // results' rows 8 y + quad + (0..3) of this tile's starts
            auto starts = [&](int which) {
                f32x16 d;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const f32x4 v = *reinterpret_cast<const f32x4*>(&rowstat[cur][which][8 * y + quad]);
#pragma unroll
                    for (int z = 0; z < 4; ++z) d[4 * y + z] = v[z];
                }
                return d;
            };
            auto probabilities = [&] {
                f32x16 s = starts(0);
#pragma unroll
                for (int x = 0; x < T::NS; ++x)
                    s = mma_step<DT>(row_operand<DT, ND>(lds[cur][0], 0, rb, x),
                                     row_operand<DT, ND>(ldk, wave * 32, rb, x), s);
                settle<DT>(s);
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = __builtin_amdgcn_exp2f(s[e] * c);
                return s;
            };
            auto dout_v = [&] {  // <do, v> - delta
                f32x16 dp = starts(1);
#pragma unroll
                for (int x = 0; x < T::NS; ++x) {
                    const uint4 v = x < VR ? vf[x] : *reinterpret_cast<const uint4*>(vl + (x - VR) * 128 * 32);
                    dp = mma_step<DT>(row_operand<DT, ND>(lds[cur][1], 0, rb, x), v, dp);
                }
                settle<DT>(dp);
                return dp;
            };
            if (ONE && DT == DT_BF16 && t < one_block) {
                f32x16 p = probabilities();
                const f32x16 dp = dout_v();
                const KeyRange seen = positions(opaque(key));
#pragma unroll
                for (int e = 0; e < 16; ++e) p[e] = sees(q0, e, seen) ? p[e] * dp[e] : 0.0f;
                // over the 32 lanes; each step halves the elements a lane is left with
#pragma unroll
                for (int n = 8, m = 1; n; n >>= 1, m <<= 1)
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        const float keep = l & m ? p[i + n] : p[i], give = l & m ? p[i] : p[i + n];
                        p[i] = keep + shfl_xor(give, m);
                    }
                const float off = p[0] + shfl_xor(p[0], 16);
                const int row = (l & 1) * 16 + (l & 2) * 4 + (l >> 2 & 1) * 2 + (l >> 3 & 1) + quad;
                if (!(l & 16)) rowstat[cur][1][row] -= off;
                // half of the lanes write what all of the wave read next
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
            f32x16 s = DT == DT_BF16 ? starts(0) : f32x16{}, dp = starts(1);
#pragma unroll
            for (int x = 0; x < T::NS; ++x)
                s = mma_step<DT>(row_operand<DT, ND>(lds[cur][0], 0, rb, x),
                                 row_operand<DT, ND>(ldk, wave * 32, rb, x), s);
#pragma unroll
            for (int x = 0; x < T::NS; ++x) {
                const uint4 v = x < VR ? vf[x] : *reinterpret_cast<const uint4*>(vl + (x - VR) * 128 * 32);
                dp = mma_step<DT>(row_operand<DT, ND>(lds[cur][1], 0, rb, x), v, dp);
            }
            if constexpr (DT == DT_BF16) {
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = __builtin_amdgcn_exp2f(s[e] * c);
            } else {
                const f32x16 lse2 = starts(0);
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = probability<DT>(s[e], c, lse2[e]);
            }
            settle<DT>(dp);
            // some pair of this block is masked?
            bool part = w0 + 32 > Lk || q0 + BQ > Lq;
            if (a.causal) {
                part = part || w0 + 31 > q0 + off;
                if (a.window) part = part || w0 <= q0 + BQ - 1 + off - a.window;
            }
            if (part) {
                const KeyRange seen = positions(opaque(key));
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (!sees(q0, e, seen)) s[e] = 0.0f;
            }
            Packed<DT> pk;
            pk.set(s);
            trans_product<DT, ND, false, SAFE>(lds[cur][1], 0, tb, pk, part, q0, positions(opaque(key)), dv);
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] *= dp[e];
            if (part) {  // P is 0 there; keep what is not finite out as well
                const KeyRange seen = positions(opaque(key));
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (!sees(q0, e, seen)) s[e] = 0.0f;
            }
            pk.set(s);
            trans_product<DT, ND, false, SAFE>(lds[cur][0], 0, tb, pk, part, q0, positions(opaque(key)), dk);
        }
        if (i + 1 < i1) put(cur ^ 1);
        __syncthreads();
        t = tn;
        g = gn;
    }
#pragma unroll
    for (int db = 0; db < ND; ++db) {
        settle<DT>(dk[db]);
        settle<DT>(dv[db]);
    }
    if (!SAFE && a.hides) {
        const bool ok = sums_finite<ND>(dk) && sums_finite<ND>(dv);
        if (l == 0) a.marks[(a.dq_items + id) * 4 + wave] = !ok;
    }
    if (!live) return;
    const KeyRange used = positions(key);
    const bool empty = used.lo == used.hi;
    if (a.nsplit_kv > 1) {
        const int64_t at = ((((int64_t)part_id * a.B + b) * a.Hkv + hk) * a.Sk + key) * a.D;
        store_rows<DT_F32, ND>(reinterpret_cast<char*>(a.part_dk + at), dk, a.scale, empty, a.D);
        store_rows<DT_F32, ND>(reinterpret_cast<char*>(a.part_dv + at), dv, 1.0f, empty, a.D);
    } else {
        store_rows<DT, ND>(a.dk.p + b * a.dk.sb + key * a.dk.ss + hk * a.dk.sh, dk, a.scale, empty, a.D);
        store_rows<DT, ND>(a.dv.p + b * a.dv.sb + key * a.dv.ss + hk * a.dv.sh, dv, 1.0f, empty, a.D);
    }
}

// Waves a SIMD: as many as registers and LDS can hold without spills (fp32 heads up
// to 64: 1 x 512, 12 heads of 64, 93 us with two, 103 with one).
template <int DT, int ND>
constexpr int kDkvWaves = ND > 2 ? (DT == DT_BF16 ? 2 : 1) : DT == DT_BF16 ? 3 : 2;

template <int DT, int ND>
__global__ __launch_bounds__(256, (kDkvWaves<DT, ND>)) void attention_dkv_kernel(AttnArgs a, int key_tiles) {
    __shared__ __attribute__((aligned(16))) DkvShared<DT, ND> shared;
    attention_dkv<DT, ND, false, false>(a, blockIdx.x, key_tiles, shared);
}

template <int DT, int ND>
struct BackwardShared {
    static constexpr int BYTES = sizeof(DqShared<DT, ND>) > sizeof(DkvShared<DT, ND>) ? sizeof(DqShared<DT, ND>)
                                                                                     : sizeof(DkvShared<DT, ND>);
    char bytes[BYTES];
    __device__ __forceinline__ DqShared<DT, ND>& dq() { return *reinterpret_cast<DqShared<DT, ND>*>(bytes); }
    __device__ __forceinline__ DkvShared<DT, ND>& dkv() { return *reinterpret_cast<DkvShared<DT, ND>*>(bytes); }
};

// Both in one launch, the dk/dv items, which take longer, first.  They form delta
// themselves (reading o too) instead of waiting for the dq items'.
template <int DT, int ND>
__global__ __launch_bounds__(256, (kDkvWaves<DT, ND>)) void attention_backward_kernel(AttnArgs a, int row_tiles,
                                                                                  int key_tiles, int dkv_items) {
    __shared__ __attribute__((aligned(16))) BackwardShared<DT, ND> shared;
    if ((int)blockIdx.x < dkv_items)
        attention_dkv<DT, ND, true, false>(a, blockIdx.x, key_tiles, shared.dkv());
    else
        attention_dq<DT, ND, true, false>(a, blockIdx.x - dkv_items, row_tiles, shared.dq());
}

// The marked items of both, with delta as the first pass formed it (ONE), so that
// what nothing hidden reaches keeps its bits.  With none marked, as ever but for a
// NaN or an infinity that a mask hides, a launch and a look at the marks: 4 to 5 us.
template <int DT, int ND, bool ONE>
__global__ __launch_bounds__(256, 1) void attention_backward_again_kernel(AttnArgs a, int row_tiles, int key_tiles,
                                                                          int items) {
    __shared__ __attribute__((aligned(16))) BackwardShared<DT, ND> shared;
    each_marked(
        items,
        [&](int i) {
            const int4 m = reinterpret_cast<const int4*>(a.marks)[i];
            return (m.x | m.y | m.z | m.w) != 0;
        },
        [&](int i) {
            i = __builtin_amdgcn_readfirstlane(i);
            if (i < a.dq_items)
                attention_dq<DT, ND, ONE, true>(a, i, row_tiles, shared.dq());
            else
                attention_dkv<DT, ND, ONE, true>(a, i - a.dq_items, key_tiles, shared.dkv());
        });
}

// Adds the parts of dk and dv in order, four elements a thread.  Bound by reading
// them: 8192 keys, 8 heads of 64, 4 parts, 143 MB with the result: 24 us, 5.9 TB/s.
template <int DT>
__global__ __launch_bounds__(256) void attention_dkv_join_kernel(AttnArgs a) {
    const int64_t quads = (int64_t)a.B * a.Hkv * a.Sk * (a.D / 4), i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= 2 * quads) return;
    const bool second = i >= quads;
    const int64_t at = second ? i - quads : i, row = at / (a.D / 4);
    const int e = (int)(at % (a.D / 4)) * 4;
    const float* from = (second ? a.part_dv : a.part_dk) + at * 4;
    float4 s = *reinterpret_cast<const float4*>(from);
    for (int p = 1; p < a.nsplit_kv; ++p) {
        const float4 x = *reinterpret_cast<const float4*>(from + p * quads * 4);
        s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    const int key = (int)(row % a.Sk);
    const int64_t bh = row / a.Sk;
    const HeadsArg& t = second ? a.dv : a.dk;
    char* to = t.p + (bh / a.Hkv) * t.sb + key * t.ss + (bh % a.Hkv) * t.sh;
    if constexpr (DT == DT_BF16) {
        bf16x2 u, v;
        u[0] = (__bf16)s.x, u[1] = (__bf16)s.y, v[0] = (__bf16)s.z, v[1] = (__bf16)s.w;
        *reinterpret_cast<uint2*>(to + 2 * e) =
            make_uint2(__builtin_bit_cast(uint32_t, u), __builtin_bit_cast(uint32_t, v));
    } else {
        *reinterpret_cast<float4*>(to + 4 * e) = s;
    }
}

// Two reasons to cut a key tile's queries into parts, up to 8.  Many queries
// share few keys: the workgroups of a causal mask are then few and uneven.  A
// part costs a write and a read of fp32 sums, 16 bytes an element of its keys,
// against 8 Sq G operations, so with 4096 rows or more a part it is lost in
// the rest (8192 tokens, 32/8 heads of 64: the backward pass takes 1404 us whole,
// 1033 in 4 parts; 4096: 658 and 305).  Or the device is not full: then parts run side by side, and the
// joining launch is paid for by a tile of 32 rows in fp32 (4 us) or 8 such
// tiles in bf16.
int attention_dkv_splits(int64_t B, int64_t Sq, int64_t Sk, int64_t Hkv, int64_t G, int dtype, int num_cus) {
    const int64_t blocks = B * Hkv * ((Sk + 127) / 128), rows = Sq * G, least = dtype == DT_BF16 ? 256 : 64;
    if (blocks == 0 || blocks >= 8 * (int64_t)num_cus) return 1;
    int64_t n = std::min<int64_t>((8 * (int64_t)num_cus + blocks - 1) / blocks, rows / 4096);
    if (blocks < num_cus) n = std::max<int64_t>(n, std::min<int64_t>((2 * num_cus + blocks - 1) / blocks, rows / least));
    return (int)std::max<int64_t>(1, std::min<int64_t>(n, 8));
}

// One launch or two?  One saves the wait between two kernels and fills the end
// of the first with the second; two form delta once only.  With all items on
// the device in two rounds of resident workgroups one launch is the faster
// (bf16, causal: 1 x 512 tokens, 16 heads of 128, 44 us against 61; 4 x 1024, 16 of
// 128, 112 / 121; 8 x 1024, 12 of 64, 73 / 83; 4 x 512, 8 of 80, 41 / 53; fp32: 4 x
// 128, 16 of 128, 57 / 88), with more it loses (4 x 2048, 16 of 128: 335 / 297; 8 x
// 4096, 12 of 64: 888 / 809).
// Without a causal mask workgroups end together, and rows above 64 gain in one
// round only (4 x 1024, 16 of 128: 158 / 144; 4 x 512: 55 / 62).
template <int DT, int ND>
static bool one_backward_kernel(const AttnArgs& a, int64_t items) {
    const int resident = DT != DT_BF16 ? 1 : ND <= 2 ? 3 : 2, rounds = ND <= 2 || a.causal ? 2 : 1;
    // delta of a short window or of few keys comes from the dq side
    if (DT == DT_BF16 && (short_window(a) || few_keys(a))) return false;
    return items <= (int64_t)a.num_cus * resident * rounds;
}

template <int DT, int ND>
static void launch_backward(const AttnArgs& a, hipStream_t st) {
    const int64_t tiles = ((int64_t)a.Sq * a.G + 127) / 128, key_tiles = ((int64_t)a.Sk + 127) / 128;
    const int64_t heads = (int64_t)a.B * a.Hkv;
    const int dq_items = (int)(heads * tiles), items = dq_items + (int)(heads * key_tiles * a.nsplit_kv);
    const bool one = one_backward_kernel<DT, ND>(a, items);
    if (one && items > 0)
        hipLaunchKernelGGL((attention_backward_kernel<DT, ND>), dim3((unsigned)items), dim3(256), 0, st, a, (int)tiles,
                           (int)key_tiles, items - dq_items);
    if (!one) {
        if (tiles > 0)
            hipLaunchKernelGGL((attention_dq_kernel<DT, ND>), dim3((unsigned)dq_items), dim3(256), 0, st, a, (int)tiles);
        if (key_tiles > 0)
            hipLaunchKernelGGL((attention_dkv_kernel<DT, ND>), dim3((unsigned)(items - dq_items)), dim3(256), 0, st, a,
                               (int)key_tiles);
    }
    if (a.hides && items > 0) {
        const dim3 grid((unsigned)std::min(items, a.num_cus));
        if (one)
            hipLaunchKernelGGL((attention_backward_again_kernel<DT, ND, true>), grid, dim3(256), 0, st, a, (int)tiles,
                               (int)key_tiles, items);
        else
            hipLaunchKernelGGL((attention_backward_again_kernel<DT, ND, false>), grid, dim3(256), 0, st, a, (int)tiles,
                               (int)key_tiles, items);
    }
    if (a.nsplit_kv > 1) {
        const int64_t quads = heads * a.Sk * (a.D / 4);
        hipLaunchKernelGGL((attention_dkv_join_kernel<DT>), dim3((unsigned)((2 * quads + 255) / 256)), dim3(256), 0, st,
                           a);
    }
}

hipError_t run_attention_backward(const AttnArgs& a, int dtype, hipStream_t st) {
    const int nd = (a.D + 31) / 32;
#define PAMM_CASE(DT, ND) \
    if (dtype == DT && nd == ND) launch_backward<DT, ND>(a, st)
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
