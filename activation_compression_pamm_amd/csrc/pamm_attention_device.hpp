// pamm_attention_device.hpp -- tiles and matrix products shared by the
// attention kernels (gfx950).
//
// Everything is built from one 32 x 32 product whose operands are 16 bytes a
// lane: bf16 takes one v_mfma_f32_32x32x16_bf16 (a contraction of 16), fp32
// four v_mfma_f32_32x32x2f32 (a contraction of 8).  A lane holds row (A) or
// column (B) l % 32, elements of the 16-byte group 2 s + l / 32 of step s.
//
// Result element i of lane l is D[8 (i / 4) + 4 (l / 32) + i % 4][l % 32].
// That is also a valid B operand of the next product when its contraction
// runs over D's rows in that same order: a contraction's order is free as long
// as both operands agree, so probabilities go from one product to the next in
// the registers they were born in, and only the A operand is fetched in
// matching order (trans_product below).
#pragma once
#include "pamm_block_kernels.hpp"
#include "pamm_device.hpp"

namespace pamm {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A tile of rows in LDS, ND x 32 elements a row, rows PITCH bytes apart.  The
// 16-byte group c of row r lies at slot c ^ key(r): sixteen rows read at one
// group (row operand) fall into sixteen different slots of the 256-byte bank
// line, and the eight 64-byte pieces that half a wave reads for a transposed
// operand (four rows and four more) do not share banks either.
template <int DT, int ND>
struct Tile {
    static constexpr int ES = Elem<DT>::size;
    static constexpr int PE = Elem<DT>::per16;
    static constexpr int PITCH = (ND <= 2 ? 64 : 128) * ES;
    static constexpr int NS = ND * ES;        // 32-byte contraction steps of a row
    static constexpr int CPR = 2 * NS;        // 16-byte groups of a row that are used
    __host__ __device__ static constexpr int key(int r) {
        if constexpr (PITCH == 128) {
            const int r2 = r >> 1;
            return ((r2 & 1) << 2) | ((r2 >> 1) & 3);
        } else {
            return ((r & 3) << 2) | ((r >> 2) & 3);
        }
    }
    __device__ static __forceinline__ int offset(int r, int c) { return r * PITCH + ((c ^ key(r)) << 4); }
};

// The wave's number as a value the compiler knows to be the same in all lanes:
// what follows from it stays in scalar registers and branches.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Lane-dependent parts of LDS addresses.  The group index only ever meets the
// key by exclusive or, so the address of group c + 2 s is base ^ (s << 5).
// Hidden from the compiler once an iteration, the base stays one register and
// each address costs one instruction; left alone, all of them are kept in
// registers over the loop, and what does not fit is spilled.
__device__ __forceinline__ int opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}
// Row operand: row l % 32, group l / 32.
template <int DT, int ND>
__device__ __forceinline__ int row_base() {
    const int l = lane_id();
    return Tile<DT, ND>::offset(l & 31, l >> 5);
}
// Transposed bf16 operand: rows 4 (l / 32) + (l % 16) / 4, and 8 more (the key
// of row + 8 is the key of row with one bit flipped).
template <int DT, int ND>
__device__ __forceinline__ int trans_base() {
    const int l = lane_id();
    if constexpr (DT == DT_BF16)
        return Tile<DT, ND>::offset(4 * (l >> 5) + ((l & 15) >> 2), ((l >> 4) & 1) * 2 + ((l & 3) >> 1)) + (l & 1) * 8;
    else
        return l;  // the fp32 operand's address is formed from the lane
}

// One 32 x 32 product step; a and b are 16 bytes of A and B.
template <int DT>
__device__ __forceinline__ f32x16 mma_step(const uint4& a, const uint4& b, f32x16 c) {
    if constexpr (DT == DT_BF16) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    } else {
        const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[j], y[j], c, 0, 0, 0);
        return c;
    }
}

// A result may be read by ordinary instructions only some wait states after its
// last product (11 after the bf16 product's 8 passes, 18 after the fp32 one's
// 16), which the compiler counts and fills.  Where a branch that may be skipped
// lies between the two, ROCm 7.2's compiler was seen to count along the longer
// way round only and to read results too early.  So each result is waited for
// in the block that computed it, before any branch.
template <int DT>
__device__ __forceinline__ void settle(f32x16& d) {
    if constexpr (DT == DT_BF16)
        asm volatile("s_nop 10" : "+v"(d));
    else
        asm volatile("s_nop 15\n\ts_nop 1" : "+v"(d));
}

// 32 x 32 results as the B operand of a product that contracts over D's rows:
// bf16 rounds each value once (nearest even) and packs, fp32 keeps them.
template <int DT> struct Packed;
template <> struct Packed<DT_BF16> {
    bf16x8 v[2];
    __device__ __forceinline__ void set(const f32x16& d) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i >> 3][i & 7] = (__bf16)d[i];
    }
};
template <> struct Packed<DT_F32> {
    f32x16 v;
    __device__ __forceinline__ void set(const f32x16& d) { v = d; }
};

// The operands of one block of 32 tile rows, all of them: rows (for products
// that contract over a row's elements) and transposed (for products that
// contract over the rows).  A load from LDS takes several products' time, so
// a block's operands are all requested before the first is used; `fence` keeps
// the compiler from moving them back to their uses.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Row operand of step s: 16 bytes of row r0 + l % 32 (r0 a multiple of 32).
template <int DT, int ND>
__device__ __forceinline__ uint4 row_operand(const char* tile, int r0, int base, int s) {
    return *reinterpret_cast<const uint4*>(tile + r0 * Tile<DT, ND>::PITCH + (base ^ (s << 5)));
}

template <int DT, int ND>
struct Rows {
    static constexpr int NS = Tile<DT, ND>::NS;
    uint4 v[NS];
    __device__ __forceinline__ void load(const char* tile, int r0, int base) {
#pragma unroll
        for (int s = 0; s < NS; ++s) v[s] = row_operand<DT, ND>(tile, r0, base, s);
    }
    // c + rows x b
    __device__ __forceinline__ f32x16 product(const uint4* b, f32x16 c) const {
#pragma unroll
        for (int s = 0; s < NS; ++s) c = mma_step<DT>(v[s], b[s], c);
        return c;
    }
};

// acc[db] += (the 32 rows of `tile` from row r0, transposed) x b, for the ND
// 32-element column blocks db: acc[db][e][col] += sum_r tile[r][32 db + e] b[r][col].
// bf16 reads its operand with the transposing LDS load: the 16 lanes of a
// group point at four rows of 32 bytes and each gets one column of the four.
template <int DT, int ND> struct Columns;
template <int ND>
struct Columns<DT_BF16, ND> {
    using T = Tile<DT_BF16, ND>;
    static constexpr int STEPS = 2;
    bf16x8 v[STEPS][ND];
    __device__ static __forceinline__ bf16x8 one(const char* tile, int r0, int base, int t, int db) {
        constexpr int flip = (T::key(8) ^ T::key(0)) << 4;
        typedef __attribute__((address_space(3))) s16x4* lds_s4;
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const char* at = tile + (r0 + 16 * t) * T::PITCH;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(at + (base ^ (db << 6))));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(at + 8 * T::PITCH + (base ^ (db << 6) ^ flip)));
        const s16x8 x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8, x);
    }
    __device__ __forceinline__ void load(const char* tile, int r0, int base) {
#pragma unroll
        for (int t = 0; t < STEPS; ++t)
#pragma unroll
            for (int db = 0; db < ND; ++db) v[t][db] = one(tile, r0, base, t, db);
    }
    __device__ static __forceinline__ f32x16 step(const bf16x8& x, const Packed<DT_BF16>& b, int t, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, b.v[t], c, 0, 0, 0);
    }
    __device__ __forceinline__ void product(const Packed<DT_BF16>& b, f32x16* acc) const {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int db = 0; db < ND; ++db)
                acc[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[t][db], b.v[t], acc[db], 0, 0, 0);
    }
    template <typename F>
    __device__ static __forceinline__ bf16x8 each(const bf16x8& x, F&& f) {
        bf16x8 y;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (__bf16)f((float)x[i]);
        return y;
    }
    __device__ static __forceinline__ bool finite(const bf16x8& x) {
        const uint4 w = __builtin_bit_cast(uint4, x);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        bool ok = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) ok &= ((u[i] & 0x7f80u) != 0x7f80u) & ((u[i] & 0x7f800000u) != 0x7f800000u);
        return ok;
    }
};
template <int ND>
struct Columns<DT_F32, ND> {
    using T = Tile<DT_F32, ND>;
    static constexpr int STEPS = 16;
    float v[STEPS][ND];
    __device__ static __forceinline__ float one(const char* tile, int r0, int base, int t, int db) {
        const int l = base, row = r0 + 8 * (t >> 2) + 4 * (l >> 5) + (t & 3), e = 32 * db + (l & 31);
        return *reinterpret_cast<const float*>(tile + T::offset(row, e >> 2) + (e & 3) * 4);
    }
    __device__ __forceinline__ void load(const char* tile, int r0, int base) {
#pragma unroll
        for (int t = 0; t < STEPS; ++t)
#pragma unroll
            for (int db = 0; db < ND; ++db) v[t][db] = one(tile, r0, base, t, db);
    }
    __device__ static __forceinline__ f32x16 step(float x, const Packed<DT_F32>& b, int t, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x2f32(x, b.v[t], c, 0, 0, 0);
    }
    __device__ __forceinline__ void product(const Packed<DT_F32>& b, f32x16* acc) const {
#pragma unroll
        for (int t = 0; t < STEPS; ++t)
#pragma unroll
            for (int db = 0; db < ND; ++db) acc[db] = step(v[t][db], b, t, acc[db]);
    }
    template <typename F>
    __device__ static __forceinline__ float each(float x, F&& f) {
        return f(x);
    }
    __device__ static __forceinline__ bool finite(float x) { return isfinite(x); }
};

// Whether all 32 rows' elements are finite.  One operand at a time: only
// blocks with masked pairs are looked through, and what they need in registers
// must not be more than the plain product's.
template <int DT, int ND>
__device__ __forceinline__ bool rows_finite(const char* tile, int r0, int base) {
    using C = Columns<DT, ND>;
    const int at = opaque(base);  // loads of its own: shared ones would be held for the product
    bool ok = true;
#pragma unroll
    for (int t = 0; t < C::STEPS; ++t)
#pragma unroll
        for (int db = 0; db < ND; ++db) {
            ok &= C::finite(C::one(tile, r0, at, t, db));  // no branch: all lanes take part in each load
            fence();
        }
    return __all(ok);
}

// The clean part of a product with a block that holds something not finite:
// those elements count as 0.
template <int DT, int ND>
__device__ __forceinline__ void finite_product(const char* tile, int r0, int base, const Packed<DT>& b, f32x16* acc) {
    using C = Columns<DT, ND>;
    const int at = opaque(base);
#pragma unroll
    for (int db = 0; db < ND; ++db)
#pragma unroll
        for (int t = 0; t < C::STEPS; ++t) {
            acc[db] = C::step(C::each(C::one(tile, r0, at, t, db), [](float x) { return isfinite(x) ? x : 0.0f; }), b, t,
                              acc[db]);
            fence();
        }
#pragma unroll
    for (int db = 0; db < ND; ++db) settle<DT>(acc[db]);
}

// This lane's 16-byte groups of one global row (zero where !ok or past D).
template <int DT, int ND>
__device__ __forceinline__ void load_row_operand(uint4* f, const char* row, bool ok, int D) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int s = 0; s < Tile<DT, ND>::NS; ++s) {
        const int c = 2 * s + h;
        f[s] = make_uint4(0, 0, 0, 0);
        if (ok && c * Elem<DT>::per16 < D) f[s] = *reinterpret_cast<const uint4*>(row + c * 16);
    }
}

// A result that starts from v instead of 0.
__device__ __forceinline__ f32x16 splat(float v) {
    f32x16 d;
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i] = v;
    return d;
}

// Waits for operands loaded before a loop.  Left to the compiler, the wait
// stands at their first use inside the loop, where it also waits for the next
// tile's loads, every time round.
template <int N>
__device__ __forceinline__ void arrived(uint4 (&f)[N]) {
#pragma unroll
    for (int s = 0; s < N; ++s) asm volatile("" : "+v"(f[s].x), "+v"(f[s].y), "+v"(f[s].z), "+v"(f[s].w));
}

// Flip the sign of every element (exact).
template <int DT>
__device__ __forceinline__ uint4 negate16(uint4 v) {
    const uint32_t m = DT == DT_BF16 ? 0x80008000u : 0x80000000u;
    return make_uint4(v.x ^ m, v.y ^ m, v.z ^ m, v.w ^ m);
}

// The two halves of a wave hold the other half of a column: v of lane l % 32
// and of lane l % 32 + 32, in every lane.
__device__ __forceinline__ float half_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A bounded view of `rows` rows of D elements, `stride` bytes apart: what is
// read through it past the last row's end is zero.  64 rows span less than
// 2 GiB, so offsets into it are 32 bits; tiles move the base.
struct RowView {
    __amdgpu_buffer_rsrc_t rsrc;
    __device__ __forceinline__ RowView(const char* base, int stride, int rows, int most, int row_bytes) {
        const int n = rows < most ? rows : most;
        const int bytes = n > 0 ? (n - 1) * stride + row_bytes : 0;
        rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, bytes, 0x00020000);
    }
    __device__ __forceinline__ uint4 load(int offset) const {
        return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, offset, 0, 0));
    }
    // the same for what is read once: it does not push other lines out of the caches
    __device__ __forceinline__ uint4 load_once(int offset) const {
        return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, offset, 0, 2));
    }
};
constexpr int kOutside = (int)0x80000000u;  // an offset past every view's end

// Copies rows [0, ROWS) of a tile through registers: fetch() issues the
// global loads, put() writes them to LDS.  NT threads take part.  Rows at or
// past `rows` and elements past D become zero.
template <int DT, int ND, int ROWS, int NT>
struct TileCopy {
    using T = Tile<DT, ND>;
    static constexpr int N = ROWS * T::CPR;
    static constexpr int PER = (N + NT - 1) / NT;
    // rows between a thread's vectors, where that is a whole number: one offset
    // then serves all of them, in memory from a base of their own, in LDS with
    // an immediate (the key repeats every 16 rows)
    static constexpr bool EVEN = NT % T::CPR == 0 && (NT / T::CPR) % 16 == 0 && N % NT == 0;
    static constexpr int RPI = NT / T::CPR;
    uint4 r[PER];
    __device__ __forceinline__ void fetch(const char* base, int stride, int rows, int D, int tid) {
        if constexpr (EVEN) {
            const int row = tid / T::CPR, c = tid % T::CPR, at = c * T::PE < D ? row * stride + c * 16 : kOutside;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                r[i] = RowView(base + (int64_t)i * RPI * stride, stride, rows - i * RPI, RPI, D * T::ES).load(at);
        } else {
            const RowView v(base, stride, rows, ROWS, D * T::ES);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int id = tid + i * NT, row = id / T::CPR, c = id % T::CPR;
                r[i] = v.load((N % NT == 0 || id < N) && c * T::PE < D ? row * stride + c * 16 : kOutside);
            }
        }
    }
    __device__ __forceinline__ void put(char* tile, int tid) const {
        if constexpr (EVEN) {
            const int at = T::offset(tid / T::CPR, tid % T::CPR);
#pragma unroll
            for (int i = 0; i < PER; ++i) *reinterpret_cast<uint4*>(tile + at + i * RPI * T::PITCH) = r[i];
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int id = tid + i * NT, row = id / T::CPR, c = id % T::CPR;
                if (N % NT == 0 || id < N) *reinterpret_cast<uint4*>(tile + T::offset(row, c)) = r[i];
            }
        }
    }
};

// Keys [lo, hi) that query position p sees, given the sequence's lengths.
// Sequences hold fewer than 2^30 rows, so positions and their sums fit 32 bits.
struct KeyRange {
    int lo, hi;
};
__device__ __forceinline__ KeyRange key_range(const AttnArgs& a, int p, int Lq, int Lk) {
    KeyRange r{0, Lk};
    if (p >= Lq) {
        r.hi = 0;
    } else if (a.causal) {
        const int last = p + (Lk - Lq);  // < Lk
        r.hi = last + 1;
        if (a.window) r.lo = last + 1 - a.window;
        if (r.hi < 0) r.hi = 0;
        if (r.lo < 0) r.lo = 0;
    }
    return r;
}

__device__ __forceinline__ int valid_length(const int32_t* len, int b, int most) {
    if (!len) return most;
    const int v = len[b];
    return v < 0 ? 0 : v > most ? most : v;
}

// The keys that the rows [first, first + n) of one key/value head see between
// them, [begin, end), and those that all of them see, [all_lo, all_hi).
struct RowsRange {
    int begin, end, all_lo, all_hi;
};
__device__ __forceinline__ RowsRange rows_range(const AttnArgs& a, int first, int n, int rows, int Lq, int Lk) {
    const int p0 = first / a.G, p1 = (first + n <= rows ? first + n - 1 : rows - 1) / a.G;
    RowsRange r;
    r.begin = key_range(a, p0, Lq, Lk).lo;
    r.end = p0 < Lq ? key_range(a, p1 < Lq ? p1 : Lq - 1, Lq, Lk).hi : 0;
    r.all_lo = key_range(a, p1, Lq, Lk).lo;
    r.all_hi = first + n <= rows && p1 < Lq ? key_range(a, p0, Lq, Lk).hi : 0;
    return r;
}

// Is key0 + (the key of result element i) one of [lo, hi)?  One subtraction
// and one unsigned comparison an element.
__device__ __forceinline__ bool sees(int key0, int i, const KeyRange& r) {
    const uint32_t k = (uint32_t)(key0 + 4 * (lane_id() >> 5) - r.lo) + (uint32_t)(8 * (i >> 2) + (i & 3));
    return k < (uint32_t)(r.hi - r.lo);
}

// acc += (32 rows of `tile` from r0, transposed) x b.  Where `part`, some pairs
// are masked (the edge of a causal mask or a window): tile row k is seen by
// this lane's column if row0 + k lies in [r.lo, r.hi).
//
// What a mask hides must not come through, but 0 x infinity is NaN.  A wave
// whose sums are not all finite therefore marks its rows, and a second kernel
// goes over the items with a mark, with SAFE: blocks with a masked pair are then
// looked through, and one that holds something not finite is multiplied without
// it, after which the results that do see such an element take it up (its
// infinity if SIGNED, where b is not negative, else NaN).  In one kernel the two
// share registers: the forward pass of 4 x 2048 tokens, 32 heads of 128, took 14%
// more time (a function of its own) or 28% (inline); the second kernel's look
// at the marks takes 4 to 5 us.
template <int DT, int ND, bool SIGNED, bool SAFE>
__device__ __forceinline__ void trans_product(const char* tile, int r0, int base, const Packed<DT>& b, bool part,
                                              int row0, const KeyRange& r, f32x16* acc) {
    if (SAFE && part && !rows_finite<DT, ND>(tile, r0, base)) {
        finite_product<DT, ND>(tile, r0, base, b, acc);
        const int h = opaque(lane_id() >> 5);  // nothing of this is worth registers over the kernel's loop
        const uint32_t from = (uint32_t)opaque(row0 - r.lo), many = (uint32_t)(r.hi - r.lo);
#pragma unroll 1
        for (int k = 0; k < 32; ++k) {
            const float take = from + (uint32_t)k < many ? 1.0f : 0.0f;
#pragma unroll
            for (int db = 0; db < ND; ++db)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float x[4];
                    if constexpr (DT == DT_BF16) {
                        const uint2 w =
                            *reinterpret_cast<const uint2*>(tile + Tile<DT, ND>::offset(r0 + k, 4 * db + g) + 8 * h);
                        x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xffff0000u);
                        x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xffff0000u);
                    } else {
                        const float4 w =
                            *reinterpret_cast<const float4*>(tile + Tile<DT, ND>::offset(r0 + k, 8 * db + 2 * g + h));
                        x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool hit = !isfinite(x[i]) & (take != 0.0f);
                        acc[db][4 * g + i] += hit ? (SIGNED ? x[i] : NAN) : 0.0f;
                    }
                    fence();
                }
        }
    } else {
        Columns<DT, ND> c;
        c.load(tile, r0, base);
        c.product(b, acc);
    }
}

// Whether the wave's sums are finite, which nothing hidden can have touched then.
template <int ND>
__device__ __forceinline__ bool sums_finite(const f32x16* acc) {
    uint32_t top = 0;
#pragma unroll
    for (int db = 0; db < ND; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(acc[db][i]) & 0x7fffffffu);
    return __all(top < 0x7f800000u);
}

// Runs f(item) for the items of [0, items) that marked(item) picks, the same for
// the whole workgroup, item by item.  The picks of 256 items of this workgroup
// are looked at together, so where there is none the kernel ends after one load.
template <typename M, typename F>
__device__ __forceinline__ void each_marked(int items, M&& marked, F&& f) {
    __shared__ uint64_t picks[4];
    for (int64_t first = blockIdx.x; first < items; first += (int64_t)gridDim.x * 256) {
        const int64_t mine = first + (int64_t)threadIdx.x * gridDim.x;
        const uint64_t found = __ballot(mine < items && marked((int)mine));
        if (!__syncthreads_or(found != 0)) continue;
        if ((threadIdx.x & 63) == 0) picks[threadIdx.x >> 6] = found;
        __syncthreads();
        for (int w = 0; w < 4; ++w) {
            uint64_t left = picks[w];
            while (left) {
                const int lane = __builtin_ctzll(left);
                left &= left - 1;
                f((int)(first + (int64_t)(w * 64 + lane) * gridDim.x));
                __syncthreads();  // the next item uses the same LDS
            }
        }
        __syncthreads();
    }
}

// Workgroup id -> (head of the batch, item of the head).  Workgroups are dealt
// to the 8 XCDs in turn, each with an L2 of its own: a head's items stay on one
// XCD where the heads divide evenly.  Items of falling cost (causal masks) are
// started in that order over all heads of the XCD, so that the longest do not
// start last; items of equal cost head after head, which shares the L2 best.
struct WorkItem {
    int head, item;
};
__device__ __forceinline__ WorkItem work_item(uint32_t id, uint32_t heads, uint32_t items, bool falling) {
    WorkItem w;
    if (heads % 8 == 0) {
        const uint32_t x = id % 8, s = id / 8, n = heads / 8, d = falling ? n : items;
        const uint32_t hi = s / d, lo = s - hi * d;
        w.item = (int)(falling ? hi : lo);
        w.head = (int)(x + 8 * (falling ? lo : hi));
    } else {
        uint32_t at = id, d = heads;
        if (!falling) {
            const uint32_t total = heads * items, x = id % 8, q = total / 8, r = total % 8;
            at = x * q + (x < r ? x : r) + id / 8;
            d = items;
        }
        const uint32_t hi = at / d, lo = at - hi * d;
        w.item = (int)(falling ? hi : lo);
        w.head = (int)(falling ? lo : hi);
    }
    return w;
}

// Writes ND blocks of 32 x 32 results that are transposed rows: this lane's
// row `row` gets elements 32 db + 8 (i / 4) + 4 h + i % 4, scaled by f.  A row
// that nothing was added to is 0, whatever its unused products made of it.
template <int DT, int ND>
__device__ __forceinline__ void store_rows(char* row, const f32x16* acc, float f, bool empty, int D) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int db = 0; db < ND; ++db) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int e = 32 * db + 8 * g + 4 * h;
            if (e >= D) continue;
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = empty ? 0.0f : acc[db][4 * g + i] * f;
            if constexpr (DT == DT_BF16) {
                bf16x2 u, v;
                u[0] = (__bf16)x[0], u[1] = (__bf16)x[1], v[0] = (__bf16)x[2], v[1] = (__bf16)x[3];
                uint2 w;
                w.x = __builtin_bit_cast(uint32_t, u), w.y = __builtin_bit_cast(uint32_t, v);
                *reinterpret_cast<uint2*>(row + 2 * e) = w;
            } else {
                *reinterpret_cast<float4*>(row + 4 * e) = make_float4(x[0], x[1], x[2], x[3]);
            }
        }
    }
}

}  // namespace pamm
