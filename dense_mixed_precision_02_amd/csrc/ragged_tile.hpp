// ragged_tile.hpp -- 16-bit products over ragged groups on large tiles.
//
// As in tile16_gemm (tile16_gemm.hpp): four waves on a tile, 16x16x32 matrix
// instructions with the accumulators tied in place, 128-byte k-tiles copied
// straight to LDS, double buffered, fragments read between the instructions.
//
// The K loop and the reading of MN-contiguous operands (B row-major, and both of
// the weight gradients') are tile16_gemm's.  Two other ways for the latter were
// built: turning 8 x 8 blocks in registers between the load and LDS (872 TFLOP/s on
// 8 groups of 2048 rows by 4096 x 4096 row-major, where this takes 1172: the loads of
// eight rows to an instruction take longer than the transposing reads), and copies
// written as assembly so that the compiler would not hold the transposing reads
// back (not kept).
//
// Which tile.  ROWS: a workgroup finds its tile's group by a scan of the
// offsets.  The tiles past the last full round of the device's workgroups are
// cut into four, so that they spread over four times as many; a tile that one
// workgroup works on while the others idle costs the whole launch its time.
// WGRAD: the outputs are common to all groups, so the grid is known, but a
// tile's time is its group's rows: groups are taken longest first, and each
// group's tiles are spread over the XCDs in runs (2048 x 4096 gradients of 16384
// rows, unevenly over 8 groups: 366 us with each group on one XCD, 286 so; equal
// groups: 265 and 269).
//
// Measured (bf16): 8 groups of 2048 rows by 4096 x 4096, column-major B: 442 us, 1244
// TFLOP/s, row-major 1172; tile16_gemm on 8 such products 1297 and 1213.  Bound by the
// power limit there and, with uneven groups, by their partial row tiles and the last
// round of tiles (16384 rows unevenly over 8 groups: 488 us, 1.13 PFLOP/s, row-major 519
// us).  Gradients of 2048 x 4096 from 8 groups of 2048 rows: 269 us, 1022 TFLOP/s, where
// tile16_gemm has 1189 on the same layouts; from 16384 uneven rows 287 us.  The matrix
// units are busy for 41 % there, at 2.0 GHz, so the power limit does not bound them;
// both operands' transposing reads all follow the barrier of the k-tile.
//
// Edges: a group's last row tile is usually partial, so rows are bounded by
// predicates on whole vectors instead of a slow path for the whole slab.
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
                                              char *Db, int64_t ldc, int rows, int cols, int r0,
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

// One tile of BM x BN on four waves; the LDS arrays hold at least its panels.
template <class DT, int BM, int BN, bool AK, bool BKC>
struct Tile16 {
    static constexpr int WM = 2, WN = 2, NW = 4;
    static constexpr int WTM = BM / WM, WTN = BN / WN;
    static constexpr int TM = WTM / 16, TN = WTN / 16, NI = TM * TN;
    static constexpr int KT = 128 / DT::ESZ;
    // padding of the MN-contiguous panels: see tile16_gemm
    using OpA = Operand<DT, BM, NW, AK, AK ? 0 : 32>;
    using OpB = Operand<DT, BN, NW, BKC, BKC ? 0 : 32>;
    static constexpr int NC = OpA::CPW + OpB::CPW;

    __device__ static inline void run(const RaggedArgs &p, const TileAt &at, int64_t first, DMP_LDS char *a0,
                                      DMP_LDS char *b0, DMP_LDS char *a1, DMP_LDS char *b1) {
        DMP_LDS char *LA[2] = {a0, a1};
        DMP_LDS char *LB[2] = {b0, b1};
        const int lane = lane_id(), wave = wave_id();
        const int wm = wave / WN, wn = wave % WN;
        const int kspan = at.k, nkt = kspan / KT + (kspan % KT != 0);
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
        // copy c (A's chunks, then B's) of k-tile kt; k-tiles past the end are zeros and touch no memory
        auto copy = [&](int kt, int buf, int c) {
            const int kleft = min(kspan - kt * KT, KT);
            if (c < OpA::CPW)
                opa.issue(make_rsrc(OpA::tile_base(at.A, p.lda, 0, (int64_t)kt * KT)), LA[buf], wave, c, kleft, at.rows);
            else
                opb.issue(make_rsrc(OpB::tile_base(at.B, p.ldb, 0, (int64_t)kt * KT)), LB[buf], wave, c - OpA::CPW,
                          kleft, at.cols);
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
                    const int q = i * TN + j;
                    if (slot_has(q, TM + TN, NI)) read_one(cur, 1, q * (TM + TN) / NI);
                }
            wait_vmcnt<0>();
            __syncthreads();
            read_mn(cur ^ 1);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    Mma16<DT>::run(acc[i][j], fa[seta(cur, 1)][i], fb[setb(cur, 1)][j]);
                    const int q = i * TN + j;
                    if (slot_has(q, NC, NI)) copy(kt + 2, cur, q * NC / NI);
                    if (slot_has(q, TM + TN, NI)) read_one(cur ^ 1, 0, q * (TM + TN) / NI);
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
            // two k-tiles to a trip so that each buffer is named statically; an
            // odd count runs one zero-filled k-tile more
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
        store_wave_tile<WTM, WTN>((DMP_LDS float *)slab, p.ep, (const char *)p.C + first * out_size(p.ep.c_type),
                                  (char *)p.D + first * out_size(p.ep.d_type), p.ldc, at.rows, at.cols,
                                  wm * WTM, wn * WTN, lane, [&](int i, int j) { return acc[i][j]; });
    }
};

// The group with the q-th most rows (ties: the lower group first), of at most 64.
__device__ static inline int longest_first(const RaggedArgs &p, int q, int total, int lane) {
    const int rows = lane < p.groups ? max(0, load_offset(p, lane + 1, total) - load_offset(p, lane, total)) : -1;
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
        const int o = __builtin_amdgcn_readlane(rows, g);
        rank += o > rows || (o == rows && g < lane);
    }
    return __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(lane < p.groups && rank == q)) - 1);
}

// This workgroup's tile (false: it has none).  One tile to a workgroup; the grid
// is the most tiles there can be.
template <class DT, bool AK, bool BKC, int MODE, int BM, int BN>
__device__ static inline bool my_tile(const RaggedArgs &p, int lane, TileAt &at) {
    const int total = (int)(MODE == RAGGED_WGRAD ? p.K : p.M), id = workgroup_id();
    if constexpr (MODE == RAGGED_WGRAD) {
        // Workgroup i runs on XCD i % 8 and is the (i / 8)-th there.  Every group's
        // tiles are cut into runs of p.run, as many as one XCD works on at a time (they
        // share panels through its L2); the runs, longest groups first, are dealt out
        // to the XCDs to and fro, so that no XCD gets a long group alone.
        const int tiles = p.tiles_m * p.tiles_n, runs = (tiles + p.run - 1) / p.run;
        const int seq = id / 8, s = seq / p.run, xcd = id % 8;
        const int r = 8 * s + (s % 2 ? 7 - xcd : xcd), q = r / runs;
        const int t = (r - q * runs) * p.run + seq - s * p.run;
        if (q >= p.groups || t >= tiles) return false;
        const int g = p.groups <= 64 ? longest_first(p, q, total, lane) : q;
        int tm, tn;
        grouped_order(t, p.tiles_m, p.tiles_n, tm, tn);
        const int r0 = __builtin_amdgcn_readfirstlane(load_offset(p, g, total));
        const int r1 = max(r0, __builtin_amdgcn_readfirstlane(load_offset(p, g + 1, total)));
        at = tile_at<DT, AK, BKC, MODE, BM, BN>(p, g, r0, r1, tm, tn);
    } else {
        GroupWalk<BM> count, walk;
        count.load(p, total, lane);
        walk = count;
        const int64_t tiles = (int64_t)count.all(p, total, lane) * p.tiles_n;
        if (id >= tiles) return false;
        const int t = xcd_remap(id, (int)tiles);
        int g, r0, r1, tile0, tm, tn;
        if (!walk.find(p, total, lane, t / p.tiles_n, g, r0, r1, tile0)) return false;
        grouped_order(t - tile0 * p.tiles_n, (r1 - r0 - 1) / BM + 1, p.tiles_n, tm, tn);
        at = tile_at<DT, AK, BKC, MODE, BM, BN>(p, g, r0, r1, tm, tn);
    }
    return true;
}

template <class DT, int BM, int BN, bool AK, bool BKC, int MODE>
__global__ __launch_bounds__(256) void ragged_tile(const RaggedArgs p) {
    using T = Tile16<DT, BM, BN, AK, BKC>;
    __shared__ __attribute__((aligned(1024))) char lds_a0[T::OpA::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b0[T::OpB::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_a1[T::OpA::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b1[T::OpB::BYTES];
    const int lane = lane_id();
    if constexpr (MODE == RAGGED_WGRAD) {
        TileAt at;
        if (!my_tile<DT, AK, BKC, MODE, BM, BN>(p, lane, at)) return;
        T::run(p, at, at.group * p.sC + at.row0 * p.ldc + at.col0, (DMP_LDS char *)lds_a0, (DMP_LDS char *)lds_b0,
               (DMP_LDS char *)lds_a1, (DMP_LDS char *)lds_b1);
    } else {
        const int total = (int)p.M, id = workgroup_id();
        GroupWalk<BM> count, walk;
        count.load(p, total, lane);
        walk = count;
        const int64_t tiles = (int64_t)count.all(p, total, lane) * p.tiles_n;
        // p.cut: workgroups that fit the device at once, where the last round may be cut
        int whole = (int)tiles;
        if (BM == 256 && p.cut > 0) {
            const int last = whole % p.cut;
            if (2 * last <= p.cut) whole -= last;
        }
        const int parts = whole + 4 * ((int)tiles - whole);
        if (id >= parts) return;
        const bool cut = id >= whole;
        const int i = cut ? whole + (id - whole) / 4 : xcd_remap(id, whole);
        int g, r0, r1, tile0;
        if (!walk.find(p, total, lane, i / p.tiles_n, g, r0, r1, tile0)) return;
        int tm, tn;
        grouped_order(i - tile0 * p.tiles_n, (r1 - r0 - 1) / BM + 1, p.tiles_n, tm, tn);
        if constexpr (BM == 256) {
            if (cut) {
                const int part = (id - whole) % 4;
                const TileAt at = tile_at<DT, AK, BKC, MODE, BM / 2, BN / 2>(p, g, r0, r1, 2 * tm + part / 2, 2 * tn + part % 2);
                if (at.rows <= 0 || at.cols <= 0) return;
                Tile16<DT, BM / 2, BN / 2, AK, BKC>::run(p, at, at.row0 * p.ldc + at.col0, (DMP_LDS char *)lds_a0,
                                                         (DMP_LDS char *)lds_b0, (DMP_LDS char *)lds_a1,
                                                         (DMP_LDS char *)lds_b1);
                return;
            }
        }
        const TileAt at = tile_at<DT, AK, BKC, MODE, BM, BN>(p, g, r0, r1, tm, tn);
        T::run(p, at, at.row0 * p.ldc + at.col0, (DMP_LDS char *)lds_a0, (DMP_LDS char *)lds_b0,
               (DMP_LDS char *)lds_a1, (DMP_LDS char *)lds_b1);
    }
}

}  // namespace dmp
