// scaled_tile.hpp -- 8-bit block-scaled products on BM x BN tiles.
//
// A k-tile is 128 bytes: one k-block of the scales.  Both operands are
// K-contiguous and come straight to LDS, double buffered.  The factors of the
// k-tile, sA[row] * sB[column block] for every row and 128-column block of the
// tile, are formed once by the workgroup and put beside the operands, so a wave
// reads four of them with one LDS read for each 16 x 16 block of rows.  Every
// 16 x 16 block's sum over the k-block starts from zero and enters the
// accumulator by four fused multiply-adds.  So the accumulators are in the
// ordinary registers (vector instructions cannot write the accumulation
// registers), which limits a wave to a 128 x 64 part of the tile: two waves to
// a SIMD, one's multiply-adds running beside the other's matrix instructions.
//
// The next k-tile's copies are spread over the first half of the row blocks (all of
// them at once: 63.8 us instead of 62 for 4096^3).
//
// Measured: 4096^3 e4m3 with bf16 results 63 us, 2.2 PFLOP/s; with fp32 results 16
// groups, 8011 rows, 2064 x 4096: 171 us, 0.79 PFLOP/s; with bf16 ones 8000 rows there,
// equal groups 93 to 99 us, uneven ones 130: 17 k-tiles between a prologue and an epilogue, two
// rounds of tiles.  The matrix units are
// busy for about half of the time; the multiply-adds run beside them (two waves to a
// SIMD: 34 cycles for an instruction and four multiply-adds, 33 without), the rest
// is the LDS (192 KB read and 64 KB written for a k-tile of 256 x 256) and the
// barrier of each k-tile.
//
// Two ways to the k-block's sum:
//  * the 8-bit matrix instruction on 128 k.  Within every 8 consecutive k it
//    aligns the products to the largest and drops what lies 13 bits below
//    (found by feeding it pairs of powers of two), an error of about 1.5e-5 of
//    a sum of random terms.  It is used where D has 16 bits, whose own rounding
//    is 2e-3 (bf16) or 2.4e-4 (fp16) of each value.
//  * EXACT, where D is fp32: the bytes are widened to bf16, which holds every
//    e4m3 and e5m2 value, and the bf16 instruction (half the rate) sums exact
//    products in fp32.
#pragma once
#include "ragged_tile.hpp"

namespace dmp {

// Bytes 8 h + 2 w and the next of a granule as two bf16 values (exact).
template <int FMT>
__device__ static inline int widen2(const intx4 &v, int h, int w) {
    const uint32_t x = (uint32_t)v[2 * h + w / 2];
    if constexpr (FMT == 0)
        return __builtin_bit_cast(int, w % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, false));
    else
        return __builtin_bit_cast(int, w % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(x, 1.0f, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(x, 1.0f, false));
}
// Bytes 8 h .. 8 h + 7 as eight.
template <int FMT>
__device__ static inline intx4 widen8(const intx4 &v, int h) {
    return intx4{widen2<FMT>(v, h, 0), widen2<FMT>(v, h, 1), widen2<FMT>(v, h, 2), widen2<FMT>(v, h, 3)};
}

// A k-block's factor sA * sB as s * 2^e.  Almost always e = 0.  Where the product of
// two finite factors leaves the normal numbers (factors of 2^-76 each, or of 2^70),
// though the scaled sum may well lie within them, s is the product of their
// significands and e the sum of their exponents.
struct Factor {
    float s;
    int e;
};
__device__ static inline bool factor_leaves(float a, float b, float product) {
    constexpr int FINITE_NONZERO = 0x198, ZERO_SUBNORMAL_INF = 0x2f4;  // v_cmp_class masks
    return __builtin_amdgcn_classf(product, ZERO_SUBNORMAL_INF) && __builtin_amdgcn_classf(a, FINITE_NONZERO) &&
           __builtin_amdgcn_classf(b, FINITE_NONZERO);
}
__device__ static inline Factor split_factor(float a, float b) {
    const float p = a * b;
    if (!factor_leaves(a, b, p)) return {p, 0};
    return {__builtin_amdgcn_frexp_mantf(a) * __builtin_amdgcn_frexp_mantf(b),
            __builtin_amdgcn_frexp_expf(a) + __builtin_amdgcn_frexp_expf(b)};
}
// acc + s 2^e part; for e = 0 the same fused multiply-add as everywhere.
__device__ static inline float add_scaled(float s, int e, float part, float acc) {
    const float rare = acc + __builtin_amdgcn_ldexpf(s * part, e);
    return e == 0 ? __builtin_fmaf(s, part, acc) : rare;
}

template <int FA, int FB, int BM, int BN, int WM, int WN, bool EXACT>
__global__ __launch_bounds__(WM *WN * 64, 2) void scaled_tile(const RaggedArgs p) {
    using DT = F8<FA, FB>;
    constexpr int NW = WM * WN, WTM = BM / WM, WTN = BN / WN;
    constexpr int TM = WTM / 16, TN = WTN / 16, KT = 128;
    static_assert(128 % WTN == 0, "a wave's columns lie in one block of B's scales");
    using OpA = Operand<DT, BM, NW, true>;
    using OpB = Operand<DT, BN, NW, true>;
    constexpr int NB = BN / 128, ITEMS = BM * NB;
    static_assert(ITEMS <= NW * 64, "a factor to a thread");
    __shared__ __attribute__((aligned(1024))) char lds_a0[OpA::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b0[OpB::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_a1[OpA::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b1[OpB::BYTES];
    __shared__ __attribute__((aligned(16))) float sc0[ITEMS], sc1[ITEMS];
    __shared__ __attribute__((aligned(16))) int se0[ITEMS], se1[ITEMS];
    __shared__ int again;
    DMP_LDS char *LA[2] = {(DMP_LDS char *)lds_a0, (DMP_LDS char *)lds_a1};
    DMP_LDS char *LB[2] = {(DMP_LDS char *)lds_b0, (DMP_LDS char *)lds_b1};
    DMP_LDS float *SC[2] = {(DMP_LDS float *)sc0, (DMP_LDS float *)sc1};
    DMP_LDS int *SE[2] = {(DMP_LDS int *)se0, (DMP_LDS int *)se1};

    int lane = lane_id(), tid = threadIdx.x;
    const int wave = wave_id();
    const int wm = wave / WN, wn = wave % WN;
    TileAt at;
    if (!my_tile<DT, true, true, RAGGED_SCALED, BM, BN>(p, lane, at)) return;

    const int kspan = at.k, nkt = kspan / KT + (kspan % KT != 0);
    OpA opa;
    OpB opb;
    // copy c (A's chunks, then B's) of k-tile kt; past the end: zeros, no memory is touched
    constexpr int NC = OpA::CPW + OpB::CPW;
    auto copy = [&](int kt, int buf, int c) {
        const int64_t k0 = (int64_t)kt * KT;
        const int kleft = min(kspan - kt * KT, KT);
        if (c < OpA::CPW) opa.issue(make_rsrc(OpA::tile_base(at.A, p.lda, 0, k0)), LA[buf], wave, c, kleft, at.rows);
        else opb.issue(make_rsrc(OpB::tile_base(at.B, p.ldb, 0, k0)), LB[buf], wave, c - OpA::CPW, kleft, at.cols);
    };
    // this thread's factor: row srow of the tile, column block snb
    int srow, snb;
    bool has;
    const float *sa, *sb;
    auto place = [&]() {
        opa.init(wave, lane, p.lda, 0, at.rows);
        opb.init(wave, lane, p.ldb, 0, at.cols);
        srow = tid % BM;
        snb = tid / BM;
        has = tid < ITEMS && srow < at.rows && 128 * snb < at.cols;
        sa = p.sa + (at.row0 + srow) * p.sa_row;
        sb = p.sb + at.group * p.sb_group + ((at.col0 >> 7) + snb) * p.sb_col;
    };
    float va = 0.0f, vb = 0.0f;
    auto fetch = [&](int kt) {
        if (has && kt < nkt) {
            va = sa[kt * p.sa_k];
            vb = sb[kt * p.sb_k];
        }
    };
    bool leaves = false;
    auto put = [&](auto split, int buf) {
        if (tid >= ITEMS) return;
        if constexpr (decltype(split)::value) {
            const Factor f = split_factor(va, vb);
            SC[buf][snb * BM + srow] = f.s;
            SE[buf][snb * BM + srow] = f.e;
        } else {
            const float f = va * vb;
            leaves |= factor_leaves(va, vb, f);
            SC[buf][snb * BM + srow] = f;
        }
    };

    floatx4 acc[TM][TN];
    const int nb = (wn * WTN) >> 7;
    // One k-tile, kt in LDS buffer buf: row blocks i in turn, and in the first half of
    // them the next k-tile's copies.  While the matrix instructions of row
    // block i run, the sums of row block i - 1 enter the accumulators and the
    // fragment and factors of i + 1 are read.  The scheduling barriers keep this
    // order; without them the compiler draws all row blocks' reads together and
    // spills.
    auto compute = [&](auto split, int kt, int buf) {
        constexpr bool SPLIT = decltype(split)::value;
        // frag16's place for rows that begin at a multiple of 16: the swizzle then
        // depends on the lane alone, and a row block is an immediate offset
        const int own = (lane & 15) * 128, sw = swz(lane & 15), gr = 2 * (lane >> 4);
        const int off[2] = {own + ((gr ^ sw) << 4), own + (((gr + 1) ^ sw) << 4)};
        const DMP_LDS char *la[2], *lb[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            la[h] = LA[buf] + wm * WTM * 128 + off[h];
            lb[h] = LB[buf] + wn * WTN * 128 + off[h];
        }
        auto frag = [&](const DMP_LDS char *l, int blk) { return *(const DMP_LDS intx4 *)(l + blk * 2048); };
        const int sc_at = nb * BM + wm * WTM + 4 * (lane >> 4);
        const DMP_LDS float *sc = SC[buf] + sc_at;
        const DMP_LDS int *se = SE[buf] + sc_at;
        intx4 b[TN][EXACT ? 4 : 2];
        intx4 lo[2], hi[2];
        floatx4 s[4], part[2][TN];
        intx4 a[EXACT ? 2 : 1][4];  // EXACT: A's row blocks, widened one ahead
        auto read = [&](int i) {
            lo[i & 1] = frag(la[0], i);
            hi[i & 1] = frag(la[1], i);
            if constexpr (!SPLIT) s[i % 4] = *(const DMP_LDS floatx4 *)(sc + i * 16);
        };
        auto add = [&](int i, int j) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if constexpr (SPLIT) acc[i][j][q] = add_scaled(sc[i * 16 + q], se[i * 16 + q], part[i & 1][j][q], acc[i][j][q]);
                else acc[i][j][q] = __builtin_fmaf(s[i % 4][q], part[i & 1][j][q], acc[i][j][q]);
            asm volatile("" : "+v"(acc[i][j]));  // here, not sunk to where the sum is next used
        };
        read(0);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const intx4 l = frag(lb[0], j), h = frag(lb[1], j);
            if constexpr (EXACT) {
                b[j][0] = widen8<FB>(l, 0); b[j][1] = widen8<FB>(l, 1);
                b[j][2] = widen8<FB>(h, 0); b[j][3] = widen8<FB>(h, 1);
            } else {
                b[j][0] = l; b[j][1] = h;
            }
        }
        if constexpr (EXACT) {
#pragma unroll
            for (int q = 0; q < 4; ++q) a[0][q] = widen8<FA>(q < 2 ? lo[0] : hi[0], q & 1);
            read(1);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            if (i + 1 + EXACT < TM) read(i + 1 + EXACT);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (c * (TM / 2) / NC == i) copy(kt + 1, buf ^ 1, c);
            step_sync();
            if constexpr (EXACT) {
                // four instructions to a sum, those of the TN sums in turn: each waits for
                // the one before it of its own sum
                static_assert(TN == 4, "a pair of bytes of the next row block to each instruction");
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        part[i & 1][j] = mma16<BF16>(a[i & 1][q], b[j][q], q == 0 ? floatx4{0, 0, 0, 0} : part[i & 1][j]);
                        if (i + 1 < TM) a[(i + 1) & 1][q][j] = widen2<FA>(q < 2 ? lo[(i + 1) & 1] : hi[(i + 1) & 1], q & 1, j);
                        if (i > 0 && q == 3) add(i - 1, j);
                        __builtin_amdgcn_sched_barrier(0);
                    }
            } else {
                const intx8 a8 = __builtin_shufflevector(lo[i & 1], hi[i & 1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const intx8 b8 = __builtin_shufflevector(b[j][0], b[j][1], 0, 1, 2, 3, 4, 5, 6, 7);
                    part[i & 1][j] = DT::mma(a8, b8, floatx4{0, 0, 0, 0});
                    if (i > 0) add(i - 1, j);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) add(TM - 1, j);
    };
    auto walk = [&](auto split) {
        place();
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = floatx4{0, 0, 0, 0};
        if (nkt > 0) {
#pragma unroll
            for (int c = 0; c < NC; ++c) copy(0, 0, c);
            fetch(0);
            put(split, 0);
            wait_vmcnt<0>();
        }
        __syncthreads();
        auto ktile = [&](int kt, int cur) {
            fetch(kt + 1);
            compute(split, kt, cur);
            put(split, cur ^ 1);
            wait_vmcnt<0>();
            __syncthreads();
        };
        for (int kt = 0; kt < nkt; kt += 2) {
            ktile(kt, 0);
            if (kt + 1 < nkt) ktile(kt + 1, 1);
        }
    };
    // The factors' products are watched on the way; where one left the normal numbers
    // the tile is computed once more with split factors.  (Splitting every factor would
    // take three vector instructions for each multiply-add of the loop.)
    if (tid == 0) again = 0;
    walk(std::false_type{});
    if (leaves) again = 1;
    __syncthreads();
    if (__builtin_expect(again, 0)) {
        asm volatile("" : "+v"(lane), "+v"(tid));  // places are found anew, not kept in registers meanwhile
        walk(std::true_type{});
    }
    // each wave's slab in one of the operand buffers, as many as fit each
    constexpr int SLAB = 32 * (WTN + 4) * 4, INA = OpA::BYTES / SLAB, INB = OpB::BYTES / SLAB;
    static_assert(2 * (INA + INB) >= NW, "slabs must fit");
    const int w2 = wave % (INA + INB), half = wave / (INA + INB);
    DMP_LDS char *slab = w2 < INA ? (half ? LA[1] : LA[0]) + w2 * SLAB
                                  : (half ? LB[1] : LB[0]) + (w2 - INA) * SLAB;
    const int64_t first = at.row0 * p.ldc + at.col0;
    store_wave_tile<WTM, WTN>((DMP_LDS float *)slab, p.ep, (const char *)p.C + first * out_size(p.ep.c_type),
                              (char *)p.D + first * out_size(p.ep.d_type), p.ldc, at.rows, at.cols, wm * WTM,
                              wn * WTN, lane_id(), [&](int i, int j) { return acc[i][j]; });
}

}  // namespace dmp
