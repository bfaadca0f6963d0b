// ragged_tile.hpp -- 16-bit products over ragged groups on large tiles.
//
// The K loop is tile16_gemm's (tile16_gemm.hpp): four waves on a BM x BN tile,
// 16x16x32 matrix instructions with the accumulators tied in place, 128-byte
// k-tiles copied straight to LDS into the buffer that is not read, the next
// step's fragments read between the instructions of this one.  What differs:
//  * the tile's place.  ROWS: a workgroup finds its tile's group by a scan of
//    the offsets.  WGRAD: the outputs are common to all groups, so the grid is
//    known; only the number of k-tiles differs from group to group.
//  * edges.  A group's last row tile is usually partial, so rows are bounded by
//    predicates on whole vectors instead of a slow path for the whole slab.
#pragma once
#include "ragged.hpp"

namespace dmp {

// Which of the tiles [base, base + count) a workgroup takes: XCD-aware.
// Workgroup i runs on XCD i % 8; consecutive tiles go to one XCD and its L2.
__device__ static inline int xcd_remap(int i, int count) {
    const int per = count / 8;
    return i < per * 8 ? (i % 8) * per + i / 8 : i;
}

// Tile t of a tiles_m x tiles_n grid in groups of four tile rows (walked column
// by column), so that neighbouring tiles share the panels of A and of B.
__device__ static inline void grouped_order(int t, int tiles_m, int tiles_n, int &tm, int &tn) {
    constexpr int GM = 4;
    const int group = t / (GM * tiles_n);
    const int first = group * GM, gm = min(tiles_m - first, GM);
    t -= group * GM * tiles_n;
    tm = first + t % gm;
    tn = t / gm;
}

// Output stage of one wave's WTM x WTN part of a tile, whose first element is
// at row r0, column c0 of a tile with `rows` x `cols` valid elements; C and D
// point at the tile's first element.  Accumulators (`get(i, j)`: instruction
// block i, j; lane L, register G: row 4 (L / 16) + G, column L % 16) pass
// through the wave's LDS slab, 32 rows at a time, so that C and D move as
// vectors of four.
template <int WTM, int WTN, class Get>
__device__ static inline void store_wave_tile(DMP_LDS float *slab, const EpiParams &ep, const char *Cb,
                                              char *Db, int64_t ldc, int64_t rows, int64_t cols, int r0,
                                              int c0, int lane, Get get) {
    constexpr int TN = WTN / 16, SP = WTN + 4;
    constexpr int LPR = WTN / 4, RPP = 64 / LPR, PASSES = 32 / RPP;
    const bool c_f16 = ep.c_type == OUT_F16, d_f16 = ep.d_type == OUT_F16;
    auto to_slab = [&](int q) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const floatx4 v = get(2 * q + h, j);
#pragma unroll
                for (int G = 0; G < 4; ++G)
                    slab[(16 * h + 4 * (lane >> 4) + G) * SP + j * 16 + (lane & 15)] = v[G];
            }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    };
    auto run = [&](auto cs_c, auto ds_c) {
        constexpr int CS = decltype(cs_c)::value, DS = decltype(ds_c)::value;
        const bool vec = ldc % 4 == 0 && (CS == 0 || (uintptr_t)Cb % (4 * (CS ? CS : 1)) == 0) &&
                         (uintptr_t)Db % (4 * DS) == 0;
        const int rl = lane / LPR, cl = (lane % LPR) * 4;
        const int64_t at = (int64_t)(r0 + rl) * ldc + c0 + cl;
        if (vec && c0 + WTN <= cols) {
            // C of the next 32 rows is loaded before these are transposed and stored
            floatx4 cv[2][PASSES];
            auto load_c = [&](int q, floatx4 (&dst)[PASSES]) {
#pragma unroll
                for (int u = 0; u < PASSES; ++u) {
                    dst[u] = floatx4{0, 0, 0, 0};
                    if constexpr (CS != 0) {
                        const int r = q * 32 + u * RPP;
                        if (r0 + r + rl < rows)
                            dst[u] = load4s<float, CS>(Cb, at + r * ldc, c_f16, true, 4);
                    }
                }
            };
            load_c(0, cv[0]);
#pragma unroll
            for (int q = 0; q < WTM / 32; ++q) {
                if (r0 + q * 32 >= rows) break;
                if (q + 1 < WTM / 32) load_c(q + 1, cv[(q + 1) & 1]);
                to_slab(q);
#pragma unroll
                for (int u = 0; u < PASSES; ++u) {
                    const floatx4 v = *(const DMP_LDS floatx4 *)(slab + (u * RPP + rl) * SP + cl);
                    const int r = q * 32 + u * RPP;
                    if (r0 + r + rl < rows)
                        store4s<float, DS>(Db, at + r * ldc, finish4(v, cv[q & 1][u], ep), d_f16, true, 4);
                }
                __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
            }
            return;
        }
#pragma unroll
        for (int q = 0; q < WTM / 32; ++q) {
            to_slab(q);
#pragma unroll 1
            for (int u = 0; u < PASSES; ++u) {
                const int r = q * 32 + u * RPP;
                const int n = r0 + r + rl < rows ? cols_in(cols, c0 + cl) : 0;
                floatx4 c = {0, 0, 0, 0};
                if constexpr (CS != 0) c = load4s<float, CS>(Cb, at + r * ldc, c_f16, vec, n);
                const floatx4 v = *(const DMP_LDS floatx4 *)(slab + (u * RPP + rl) * SP + cl);
                store4s<float, DS>(Db, at + r * ldc, finish4(v, c, ep), d_f16, vec, n);
            }
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        }
    };
    using S0 = std::integral_constant<int, 0>;
    using S2 = std::integral_constant<int, 2>;
    using S4 = std::integral_constant<int, 4>;
    const bool c16 = out_size(ep.c_type) == 2, d16 = out_size(ep.d_type) == 2;
    if (!ep.use_c) {
        if (d16) run(S0{}, S2{});
        else run(S0{}, S4{});
    } else if (c16) {
        if (d16) run(S2{}, S2{});
        else run(S2{}, S4{});
    } else {
        if (d16) run(S4{}, S2{});
        else run(S4{}, S4{});
    }
}

// NS slots (matrix instructions), N things spread evenly behind them: does slot
// s have thing s * N / NS behind it?
__device__ static constexpr bool slot_has(int s, int N, int NS) { return (s + 1) * N / NS != s * N / NS; }

template <class DT, int BM, int BN, bool AK, bool BKC, int MODE>
__global__ __launch_bounds__(256) void ragged_tile(const RaggedArgs p) {
    constexpr int WM = 2, WN = 2, NW = 4;
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int TM = WTM / 16, TN = WTN / 16, NI = TM * TN;
    constexpr int KT = 128 / DT::ESZ;
    // padding of the MN-contiguous panels: see tile16_gemm
    using OpA = Operand<DT, BM, NW, AK, AK ? 0 : 32>;
    using OpB = Operand<DT, BN, NW, BKC, BKC ? 0 : 32>;
    constexpr int NC = OpA::CPW + OpB::CPW;

    __shared__ __attribute__((aligned(1024))) char lds_a0[OpA::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b0[OpB::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_a1[OpA::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b1[OpB::BYTES];
    DMP_LDS char *LA[2] = {(DMP_LDS char *)lds_a0, (DMP_LDS char *)lds_a1};
    DMP_LDS char *LB[2] = {(DMP_LDS char *)lds_b0, (DMP_LDS char *)lds_b1};

    const int lane = lane_id(), wave = wave_id();
    const int wm = wave / WN, wn = wave % WN;
    const int total = (int)(MODE == RAGGED_WGRAD ? p.K : p.M);

    auto tile = [&](const TileAt &at) {
        const int kspan = (int)at.k, nkt = (kspan + KT - 1) / KT;
        OpA opa;
        OpB opb;
        opa.init(wave, lane, p.lda, 0, at.rows);
        opb.init(wave, lane, p.ldb, 0, at.cols);
        floatx4 acc[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = floatx4{0, 0, 0, 0};
        auto pin_acc = [&]() {  // see tile16_gemm
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) asm volatile("" : "+a"(acc[i][j]));
        };
        auto copy = [&](int kt, int buf, int c) {
            const int64_t k0 = (int64_t)kt * KT;
            int kleft = kspan - kt * KT;
            kleft = kleft > KT ? KT : (kleft < 0 ? 0 : kleft);
            if (c < OpA::CPW) {
                const __amdgpu_buffer_rsrc_t ra = make_rsrc(OpA::tile_base(at.A, p.lda, 0, k0));
                opa.issue(ra, LA[buf], wave, c, kleft, at.rows);
            } else {
                const __amdgpu_buffer_rsrc_t rb = make_rsrc(OpB::tile_base(at.B, p.ldb, 0, k0));
                opb.issue(rb, LB[buf], wave, c - OpA::CPW, kleft, at.cols);
            }
        };
        auto fragA = [&](int buf, int i, int s) {
            return frag16<DT, OpA, BM, AK>(LA[buf], wm * WTM + i * 16, s, lane);
        };
        auto fragB = [&](int buf, int j, int s) {
            return frag16<DT, OpB, BN, BKC>(LB[buf], wn * WTN + j * 16, s, lane);
        };
        // fragment sets: as in tile16_gemm
        constexpr int NSA = AK ? 2 : 4, NSB = BKC ? 2 : 4;
        intx4 fa[NSA][TM], fb[NSB][TN];
        auto seta = [](int buf, int s) { return AK ? s : 2 * buf + s; };
        auto setb = [](int buf, int s) { return BKC ? s : 2 * buf + s; };
        auto read_mn = [&](int buf) {
            if constexpr (!AK) {
#pragma unroll
                for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
                    for (int i = 0; i < TM; ++i) fa[seta(buf, s2)][i] = fragA(buf, i, s2);
            }
            if constexpr (!BKC) {
#pragma unroll
                for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
                    for (int j = 0; j < TN; ++j) fb[setb(buf, s2)][j] = fragB(buf, j, s2);
            }
        };
        // fragment r (A's, then B's) of step s of the k-tile in buf, where it is read between instructions
        auto read_one = [&](int buf, int s, int r) {
            if (r < TM) {
                if constexpr (AK) fa[seta(buf, s)][r] = fragA(buf, r, s);
            } else {
                if constexpr (BKC) fb[setb(buf, s)][r - TM] = fragB(buf, r - TM, s);
            }
        };
        auto ktile = [&](int kt, int cur) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    Mma16<DT>::run(acc[i][j], fa[seta(cur, 0)][i], fb[setb(cur, 0)][j]);
                    const int s = i * TN + j;
                    if (slot_has(s, TM + TN, NI)) read_one(cur, 1, s * (TM + TN) / NI);
                }
            wait_vmcnt<0>();
            __syncthreads();
            read_mn(cur ^ 1);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    Mma16<DT>::run(acc[i][j], fa[seta(cur, 1)][i], fb[setb(cur, 1)][j]);
                    const int s = i * TN + j;
                    if (slot_has(s, NC, NI)) copy(kt + 2, cur, s * NC / NI);
                    if (slot_has(s, TM + TN, NI)) read_one(cur ^ 1, 0, s * (TM + TN) / NI);
                }
            step_sync();
        };
        if (nkt > 0) {
#pragma unroll
            for (int c = 0; c < NC; ++c) copy(0, 0, c);
            wait_vmcnt<0>();
            __syncthreads();
            read_mn(0);
#pragma unroll
            for (int r = 0; r < TM + TN; ++r) read_one(0, 0, r);
#pragma unroll
            for (int c = 0; c < NC; ++c) copy(1, 1, c);
            pin_acc();
            asm volatile("s_nop 7" ::);
            for (int kt = 0; kt < nkt; kt += 2) {
                ktile(kt, 0);
                ktile(kt + 1, 1);
            }
            mma_drain();
            pin_acc();
        }
        wait_vmcnt<0>();  // the zero-fill copies past the last k-tile have landed
        __syncthreads();  // every wave is done with the operand buffers
        DMP_LDS char *slab = wave == 0 ? LA[0] : wave == 1 ? LB[0] : wave == 2 ? LA[1] : LB[1];
        static_assert(32 * (WTN + 4) * 4 <= OpA::BYTES && 32 * (WTN + 4) * 4 <= OpB::BYTES, "slab must fit");
        const int64_t first = (MODE == RAGGED_WGRAD ? at.group * p.sC : 0) + at.row0 * p.ldc + at.col0;
        store_wave_tile<WTM, WTN>((DMP_LDS float *)slab, p.ep,
                                  (const char *)p.C + first * out_size(p.ep.c_type),
                                  (char *)p.D + first * out_size(p.ep.d_type), p.ldc, at.rows, at.cols,
                                  wm * WTM, wn * WTN, lane, [&](int i, int j) { return acc[i][j]; });
    };

    if constexpr (MODE == RAGGED_WGRAD) {
        const int tiles = p.tiles_m * p.tiles_n;
        const int wg = xcd_remap(blockIdx.x, gridDim.x);
        const int g = wg / tiles;
        const int r0 = load_offset(p, g, total), r1 = max(r0, load_offset(p, g + 1, total));
        int tm, tn;
        grouped_order(wg - g * tiles, p.tiles_m, p.tiles_n, tm, tn);
        tile(tile_at<DT, AK, BKC, MODE, BM, BN>(p, g, r0, r1, tm, tn));
    } else {
        // the grid is the most row tiles there can be; the ones past the last leave
        GroupWalk<BM> count, walk;
        count.load(p, total, lane);
        walk = count;
        const int64_t tiles = (int64_t)count.all(p, total, lane) * p.tiles_n;
        if ((int64_t)blockIdx.x >= tiles) return;
        const int t = xcd_remap(blockIdx.x, (int)tiles);
        int g, r0, r1, tile0;
        if (!walk.find(p, total, lane, t / p.tiles_n, g, r0, r1, tile0)) return;
        int tm, tn;
        grouped_order(t - tile0 * p.tiles_n, (r1 - r0 - 1) / BM + 1, p.tiles_n, tm, tn);
        tile(tile_at<DT, AK, BKC, MODE, BM, BN>(p, g, r0, r1, tm, tn));
    }
}

}  // namespace dmp
