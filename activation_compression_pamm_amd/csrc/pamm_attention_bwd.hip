// pamm_attention_bwd.hip -- attention's backward pass on gfx950.
//
//   P_ij = exp(s_ij - lse_i)          delta_i = <do_i, o_i>
//   dS_ij = P_ij (<do_i, v_j> - delta_i)
//   dv_j = sum_i P_ij do_i,  dk_j = scale sum_i dS_ij q_i,
//   dq_i = scale sum_j dS_ij k_j
//
// Two kernels, each with its sums in registers and in a fixed order: one owns
// queries and runs over keys (dq, and delta on the way), one owns keys and
// runs over the queries of every head that shares them (dk, dv).  Forming P
// and dS in both costs 7 products instead of 5, and buys sums without atomics:
// the results are bitwise repeatable and no fp32 copy of dq is kept.
#include "pamm_attention_device.hpp"

namespace pamm {

__device__ __forceinline__ float score_factor(float scale) { return fmaxf(fabsf(scale) * kLog2e, 1e-36f); }

template <int DT>
__device__ __forceinline__ float dot16(const uint4& x, const uint4& y) {
    float u[8], v[8], sum = 0.0f;
    unpack16<DT>(x, u);
    unpack16<DT>(y, v);
#pragma unroll
    for (int i = 0; i < Elem<DT>::per16; ++i) sum = fmaf(u[i], v[i], sum);
    return sum;
}

// dq.  Laid out as the forward pass: transposed scores, a lane owns a query.
template <int DT, int ND>
__global__ __launch_bounds__(256, DT == DT_BF16 ? 2 : 1) void attention_dq_kernel(AttnArgs a, int row_tiles) {
    using T = Tile<DT, ND>;
    constexpr int BK = DT == DT_BF16 ? 64 : 32;
    __shared__ __attribute__((aligned(16))) char lds[2][2][BK * T::PITCH];
    const int tid = threadIdx.x, l = tid & 63, wave = tid >> 6;

    const WorkItem w = work_item(blockIdx.x, a.B * a.Hkv, row_tiles, a.causal);
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
    if (live && l < 32) a.delta[at] = delta;
    load_row_operand<DT, ND>(qf, a.q.p + b * a.q.sb + pos * a.q.ss + head * a.q.sh, seen, a.D);
    if (a.scale < 0.0f)
#pragma unroll
        for (int s = 0; s < T::NS; ++s) qf[s] = negate16<DT>(qf[s]);
    arrived(qf);
    arrived(dof);
    const float c = score_factor(a.scale);
    // a row that saw nothing (lse = -infinity) has probabilities 2^(-infinity) = 0
    float lse2 = live ? a.lse[at] * kLog2e : 0.0f;
    if (lse2 == -INFINITY) lse2 = INFINITY;
    asm volatile("" : "+v"(lse2));

    f32x16 acc[ND];
#pragma unroll
    for (int db = 0; db < ND; ++db) acc[db] = f32x16{};
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
            f32x16 s{}, dp{};
#pragma unroll
            for (int i = 0; i < T::NS; ++i) {
                s = mma_step<DT>(row_operand<DT, ND>(lds[cur][0], kb * 32, rb, i), qf[i], s);
                dp = mma_step<DT>(row_operand<DT, ND>(lds[cur][1], kb * 32, rb, i), dof[i], dp);
            }
            settle<DT>(s);
            settle<DT>(dp);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -lse2)) * (dp[i] - delta);
            if (key0 < wr.all_lo || key0 + 32 > wr.all_hi) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!sees(key0, i, mine)) s[i] = 0.0f;
            }
            Packed<DT> ds;
            ds.set(s);
            trans_product<DT, ND>(lds[cur][0], kb * 32, tb, ds, acc);
        }
        if (more) {
            kc.put(lds[cur ^ 1][0], tid);
            vc.put(lds[cur ^ 1][1], tid);
        }
        __syncthreads();
    }
#pragma unroll
    for (int db = 0; db < ND; ++db) settle<DT>(acc[db]);
    if (live) store_rows<DT, ND>(a.dq.p + b * a.dq.sb + pos * a.dq.ss + head * a.dq.sh, acc, a.scale, a.D);
}

// dk and dv.  Scores as S = Q K^T: a lane owns a key.  Four waves of 32 keys
// share tiles of 32 queries of one head, head after head.  V stays in
// registers as an operand, K in LDS: both in registers beside 128 sums a lane
// would leave one wave a SIMD.
template <int DT, int ND>
__global__ __launch_bounds__(256, DT == DT_BF16 ? 2 : 1) void attention_dkv_kernel(AttnArgs a, int key_tiles) {
    using T = Tile<DT, ND>;
    constexpr int BQ = 32;
    __shared__ __attribute__((aligned(16))) char lds[2][2][BQ * T::PITCH];
    __shared__ __attribute__((aligned(16))) char ldk[128 * T::PITCH];
    __shared__ __attribute__((aligned(16))) float rowstat[2][2][BQ];
    const int tid = threadIdx.x, l = tid & 63, wave = tid >> 6;

    const WorkItem w = work_item(blockIdx.x, a.B * a.Hkv, key_tiles, a.causal);
    const int tile = w.item, b = w.head / a.Hkv, hk = w.head % a.Hkv;  // the first keys are seen by the most queries
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
    const int64_t n = (int64_t)(n1 - n0) * a.G;
    // positions that see this lane's key: [first, last)
    int first = 0, last = key < Lk ? Lq : 0;
    if (a.causal) {
        if (key - off > first) first = key - off;
        if (a.window && key - off + a.window < last) last = key - off + a.window;
    }
    if (last < first) last = first;

    uint4 vf[T::NS];
    load_row_operand<DT, ND>(vf, a.v.p + b * a.v.sb + key * a.v.ss + hk * a.v.sh, key < Lk, a.D);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        TileCopy<DT, ND, 64, 256> kc;
        kc.fetch(a.k.p + b * a.k.sb + (b0 + 64 * i) * a.k.ss + hk * a.k.sh, (int)a.k.ss, Lk - b0 - 64 * i, a.D, tid);
        kc.put(ldk + 64 * i * T::PITCH, tid);
    }
    arrived(vf);
    const float c = score_factor(a.scale) * (a.scale < 0.0f ? -1.0f : 1.0f);

    f32x16 dk[ND], dv[ND];
#pragma unroll
    for (int db = 0; db < ND; ++db) dk[db] = dv[db] = f32x16{};

    TileCopy<DT, ND, BQ, 256> qc, oc;
    float stat = 0.0f;
    auto fetch = [&](int g, int t) {
        const int head = hk * a.G + g, q0 = t * BQ;
        qc.fetch(a.q.p + b * a.q.sb + head * a.q.sh + q0 * a.q.ss, (int)a.q.ss, Lq - q0, a.D, tid);
        oc.fetch(a.dout.p + b * a.dout.sb + head * a.dout.sh + q0 * a.dout.ss, (int)a.dout.ss, Lq - q0, a.D, tid);
        const int r = tid % BQ;
        const int64_t at = ((int64_t)b * a.H + head) * a.Sq + q0 + r;
        stat = 0.0f;
        if (tid < 2 * BQ && q0 + r < Lq) stat = tid < BQ ? a.lse[at] : a.delta[at];
    };
    auto put = [&](int buf) {
        qc.put(lds[buf][0], tid);
        oc.put(lds[buf][1], tid);
        // lse in log2 units; a row that saw nothing has probabilities 2^(-infinity) = 0
        if (tid < BQ) stat = stat == -INFINITY ? INFINITY : stat * kLog2e;
        if (tid < 2 * BQ) rowstat[buf][tid / BQ][tid % BQ] = stat;
    };
    int t = n0, g = 0;
    if (n > 0) {
        fetch(0, n0);
        put(0);
    }
    __syncthreads();
    int cur = 0;
    for (int64_t i = 0; i < n; ++i, cur ^= 1) {
        int tn = t + 1, gn = g;
        if (tn == n1) tn = n0, ++gn;
        if (i + 1 < n) fetch(gn, tn);
        const int q0 = t * BQ;
        if (q0 < wp1 && q0 + BQ > wp0) {
            const int rb = opaque(row_base<DT, ND>()), tb = opaque(trans_base<DT, ND>());
            f32x16 s{};
#pragma unroll
            for (int x = 0; x < T::NS; ++x)
                s = mma_step<DT>(row_operand<DT, ND>(lds[cur][0], 0, rb, x),
                                 row_operand<DT, ND>(ldk, wave * 32, rb, x), s);
            settle<DT>(s);
            const int quad = 4 * (l >> 5);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float4 ls = *reinterpret_cast<const float4*>(&rowstat[cur][0][8 * y + quad]);
                const float lv[4] = {ls.x, ls.y, ls.z, ls.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) s[4 * y + z] = __builtin_amdgcn_exp2f(fmaf(s[4 * y + z], c, -lv[z]));
            }
            // some pair of this block is masked?
            bool part = w0 + 32 > Lk || q0 + BQ > Lq;
            if (a.causal) {
                part = part || w0 + 31 > q0 + off;
                if (a.window) part = part || w0 <= q0 + BQ - 1 + off - a.window;
            }
            const KeyRange seen{first, last};
            if (part) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (!sees(q0, e, seen)) s[e] = 0.0f;
            }
            Packed<DT> pk;
            pk.set(s);
            trans_product<DT, ND>(lds[cur][1], 0, tb, pk, dv);
            f32x16 dp{};
#pragma unroll
            for (int x = 0; x < T::NS; ++x) dp = mma_step<DT>(row_operand<DT, ND>(lds[cur][1], 0, rb, x), vf[x], dp);
            settle<DT>(dp);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float4 de = *reinterpret_cast<const float4*>(&rowstat[cur][1][8 * y + quad]);
                const float ev[4] = {de.x, de.y, de.z, de.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) s[4 * y + z] *= dp[4 * y + z] - ev[z];
            }
            if (part) {  // P is 0 there; keep what is not finite out as well
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (!sees(q0, e, seen)) s[e] = 0.0f;
            }
            pk.set(s);
            trans_product<DT, ND>(lds[cur][0], 0, tb, pk, dk);
        }
        if (i + 1 < n) put(cur ^ 1);
        __syncthreads();
        t = tn;
        g = gn;
    }
#pragma unroll
    for (int db = 0; db < ND; ++db) {
        settle<DT>(dk[db]);
        settle<DT>(dv[db]);
    }
    if (live) {
        store_rows<DT, ND>(a.dk.p + b * a.dk.sb + key * a.dk.ss + hk * a.dk.sh, dk, a.scale, a.D);
        store_rows<DT, ND>(a.dv.p + b * a.dv.sb + key * a.dv.ss + hk * a.dv.sh, dv, 1.0f, a.D);
    }
}

template <int DT, int ND>
static void launch_backward(const AttnArgs& a, hipStream_t st) {
    const int64_t tiles = ((int64_t)a.Sq * a.G + 127) / 128, key_tiles = ((int64_t)a.Sk + 127) / 128;
    const int64_t heads = (int64_t)a.B * a.Hkv;
    if (tiles > 0)
        hipLaunchKernelGGL((attention_dq_kernel<DT, ND>), dim3((unsigned)(heads * tiles)), dim3(256), 0, st, a, (int)tiles);
    if (key_tiles > 0)
        hipLaunchKernelGGL((attention_dkv_kernel<DT, ND>), dim3((unsigned)(heads * key_tiles)), dim3(256), 0, st, a,
                           (int)key_tiles);
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
