// ragged_tile.hpp -- 16-bit products over ragged groups on large tiles.
//
// As in tile16_gemm (tile16_gemm.hpp): four waves on a tile, 16x16x32 matrix
// instructions with the accumulators tied in place, 128-byte k-tiles copied
// straight to LDS, double buffered, fragments read between the instructions.
//
// K-contiguous operands are copied straight to LDS.  An MN-contiguous one (B
// row-major, and both of the weight gradients') is turned on its way: a thread
// loads 8 k of 8 rows as eight vectors, packs the pairs of neighbouring k with
// byte permutes and writes K-contiguous granules, so that LDS and the K loop are
// the same for every layout.  tile16_gemm reads such an operand with transposing
// LDS reads instead, in one piece behind the barrier, with no matrix instruction
// beside them (the compiler makes each wait for every copy in flight).
//
// Which tile.  ROWS: a workgroup finds its tile's group by a scan of the
// offsets.  The tiles past the last full round of the device's workgroups are
// cut into four, so that they spread over four times as many; a tile that one
// workgroup works on while the others idle costs the whole launch its time.
// WGRAD: the outputs are common to all groups, so the grid is known, but a
// tile's time is its group's rows: groups are taken longest first, and each
// group's tiles are spread over all XCDs.
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

// A K-contiguous operand's copies to LDS: Operand::issue's places and bounds.
template <class DT, int R>
struct Copied {
    using Op = Operand<DT, R, 4, true>;
    static constexpr int FETCHES = Op::CPW, PUTS = 0;
    Op op;
    const char *base;
    int wave, rows, kleft;
    __amdgpu_buffer_rsrc_t rs;
    __device__ void init(const char *X, int wave_, int lane, int64_t ld, int rows_) {
        op.init(wave_, lane, ld, 0, rows_);
        base = X;
        wave = wave_;
        rows = rows_;
    }
    // For k-tile kt, of which kleft values remain (none: not positive).
    __device__ void aim(int64_t, int kt, int kleft_) {
        rs = make_rsrc(base + (int64_t)kt * 128);
        kleft = kleft_;
    }
    __device__ void fetch(DMP_LDS char *lds, int c) const { op.issue(rs, lds, wave, c, kleft, rows); }
    __device__ void put(DMP_LDS char *, int) const {}
};

// An MN-contiguous 16-bit operand, turned.  Thread: k 8 kb .. 8 kb + 7 of rows
// PER rb .. PER rb + PER - 1; kb = lane % 8, so that eight lanes write the eight
// granules of a row (no bank conflicts), and rb = lane / 8 counts on, so that a
// load takes runs of 8 PER neighbouring elements (128 bytes for R = 256).  The
// loads (fetch) stay in registers from step 1 of a k-tile to step 0 of the next,
// where they are turned and written (put), one granule at a time.
template <class DT, int R>
struct Turned {
    using Op = Operand<DT, R, 4, true>;  // the LDS layout
    static_assert(DT::ESZ == 2 && (R == 256 || R == 128), "8 k of 8 or 4 rows to a thread");
    static constexpr int PER = R / 32, W = PER / 2, FETCHES = 8, PUTS = PER;
    const char *base;
    int off, kb8, pitch, kleft;  // off: this thread's first element, or out of range; pitch: bytes from k to k
    uint32_t at;                 // its first granule in LDS
    int in[8][W];
    __amdgpu_buffer_rsrc_t rs;
    __device__ void init(const char *X, int wave, int lane, int64_t ld, int rows) {
        const int rb = wave * 8 + (lane >> 3), row = rb * PER;
        base = X;
        kb8 = (lane & 7) * 8;
        pitch = (int)ld * 2;
        off = row < rows ? kb8 * pitch + row * 2 : OOB_OFFSET;
        at = row * 128 + (((lane & 7) ^ swz(row)) << 4);
    }
    __device__ void aim(int64_t ld, int kt, int kleft_) {
        rs = make_rsrc(base + (int64_t)kt * Op::KT * ld * 2);
        kleft = kleft_;
    }
    __device__ void fetch(DMP_LDS char *, int e) {
        const int v = kb8 < kleft - e ? off : OOB_OFFSET;
        if constexpr (W == 4) {
            const intx4 x = __builtin_bit_cast(intx4, __builtin_amdgcn_raw_buffer_load_b128(rs, v, e * pitch, 0));
#pragma unroll
            for (int w = 0; w < 4; ++w) in[e][w] = x[w];
        } else {
            const intx2 x = __builtin_bit_cast(intx2, __builtin_amdgcn_raw_buffer_load_b64(rs, v, e * pitch, 0));
            in[e][0] = x[0];
            in[e][1] = x[1];
        }
    }
    // Row r of the block: swz xors the low three bits of the row, which count r,
    // into the granule's place.
    __device__ void put(DMP_LDS char *lds, int r) const {
        intx4 v;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            v[c] = __builtin_amdgcn_perm(in[2 * c + 1][r / 2], in[2 * c][r / 2], r % 2 ? 0x07060302u : 0x05040100u);
        *(DMP_LDS intx4 *)(lds + (at ^ (r << 4)) + r * 128) = v;
    }
};

// frag16 (tile16_gemm.hpp) of row block r of a wave, l being the wave's first: the
// lane's place once, the row block and the step as constants beside it.
__device__ static inline intx4 frag_at(const DMP_LDS char *l, int r, int s, int lane) {
    const int row = lane & 15, grp = lane >> 4;
    return *(const DMP_LDS intx4 *)(l + row * 128 + (((2 * grp + s) ^ swz(row)) << 4) + r * 2048);
}

// One tile of BM x BN on four waves; the LDS arrays hold at least its panels.
template <class DT, int BM, int BN, bool AK, bool BKC>
struct Tile16 {
    static constexpr int WM = 2, WN = 2, NW = 4;
    static constexpr int WTM = BM / WM, WTN = BN / WN;
    static constexpr int TM = WTM / 16, TN = WTN / 16, NI = TM * TN;
    static constexpr int KT = 128 / DT::ESZ;
    using SrcA = std::conditional_t<AK, Copied<DT, BM>, Turned<DT, BM>>;
    using SrcB = std::conditional_t<BKC, Copied<DT, BN>, Turned<DT, BN>>;
    using OpA = typename SrcA::Op;
    using OpB = typename SrcB::Op;
    static constexpr int NC = SrcA::FETCHES + SrcB::FETCHES, NP = SrcA::PUTS + SrcB::PUTS;

    __device__ static inline void run(const RaggedArgs &p, const TileAt &at, int64_t first, DMP_LDS char *a0,
                                      DMP_LDS char *b0, DMP_LDS char *a1, DMP_LDS char *b1) {
        DMP_LDS char *LA[2] = {a0, a1};
        DMP_LDS char *LB[2] = {b0, b1};
        const int lane = lane_id(), wave = wave_id();
        const int wm = wave / WN, wn = wave % WN;
        const int kspan = at.k, nkt = kspan / KT + (kspan % KT != 0);
        SrcA ca;
        SrcB cb;
        ca.init(at.A, wave, lane, p.lda, at.rows);
        cb.init(at.B, wave, lane, p.ldb, at.cols);
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
        // fetch c (A's, then B's) of the k-tile that `aim` named; k-tiles past the end
        // are zeros and touch no memory
        auto aim = [&](int kt) {
            ca.aim(p.lda, kt, min(kspan - kt * KT, KT));
            cb.aim(p.ldb, kt, min(kspan - kt * KT, KT));
        };
        auto fetch = [&](int buf, int c) {
            if (c < SrcA::FETCHES) ca.fetch(LA[buf], c);
            else cb.fetch(LB[buf], c - SrcA::FETCHES);
        };
        auto put = [&](int buf, int c) {
            if (c < SrcA::PUTS) ca.put(LA[buf], c);
            else cb.put(LB[buf], c - SrcA::PUTS);
        };
        // fragments: the next step's are read while this one's are multiplied
        intx4 fa[2][TM], fb[2][TN];
        // fragment r (A's, then B's) of step s of the k-tile in buf
        auto read = [&](int buf, int s, int r) {
            if (r < TM) fa[s][r] = frag_at(LA[buf] + wm * WTM * 128, r, s, lane);
            else fb[s][r - TM] = frag_at(LB[buf] + wn * WTN * 128, r - TM, s, lane);
        };
        // Per k-tile kt in buffer cur, step 0: the step-1 fragments are read, and in the
        // second half k-tile kt + 1, on its way in registers where an operand is turned,
        // is written to the other buffer.  Then every copy has landed and the waves meet.
        // Step 1: the next k-tile's step-0 fragments are read, and k-tile kt + 2 is
        // fetched (to buffer cur, or to registers).
        auto ktile = [&](int kt, int cur) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    Mma16<DT>::run(acc[i][j], fa[0][i], fb[0][j]);
                    const int q = i * TN + j, h = q - NI / 2;
                    if (slot_has(q, TM + TN, NI)) read(cur, 1, q * (TM + TN) / NI);
                    if constexpr (NP > 0) {
                        if (h >= 0 && slot_has(h, NP, NI / 2)) put(cur ^ 1, h * NP / (NI / 2));
                    }
                }
            wait_vmcnt<0>();
            __syncthreads();
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    Mma16<DT>::run(acc[i][j], fa[1][i], fb[1][j]);
                    const int q = i * TN + j;
                    if (q == 0) aim(kt + 2);
                    if (slot_has(q, NC, NI)) fetch(cur, q * NC / NI);
                    if (slot_has(q, TM + TN, NI)) read(cur ^ 1, 0, q * (TM + TN) / NI);
                }
            step_sync();
        };
        if (nkt > 0) {
            aim(0);
#pragma unroll
            for (int c = 0; c < NC; ++c) fetch(0, c);
#pragma unroll
            for (int c = 0; c < NP; ++c) put(0, c);
            wait_vmcnt<0>();
            __syncthreads();
#pragma unroll
            for (int r = 0; r < TM + TN; ++r) read(0, 0, r);
            aim(1);
#pragma unroll
            for (int c = 0; c < NC; ++c) fetch(1, c);
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

template <class DT, int BM, int BN, bool AK, bool BKC, int MODE>
__global__ __launch_bounds__(256) void ragged_tile(const RaggedArgs p) {
    using T = Tile16<DT, BM, BN, AK, BKC>;
    __shared__ __attribute__((aligned(1024))) char lds_a0[T::OpA::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b0[T::OpB::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_a1[T::OpA::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b1[T::OpB::BYTES];
    const int lane = lane_id();
    const int total = (int)(MODE == RAGGED_WGRAD ? p.K : p.M);

    if constexpr (MODE == RAGGED_WGRAD) {
        // Workgroup i runs on XCD i % 8 and is the (i / 8)-th there.  Every group's
        // tiles (rounded up to a multiple of 8) are dealt out in eight runs, one to
        // each XCD, so that no XCD gets a long group alone.
        const int tiles = p.tiles_m * p.tiles_n, per = (tiles + 7) / 8;
        const int seq = blockIdx.x / 8, q = seq / per;
        const int t = (blockIdx.x % 8) * per + seq - q * per;
        if (t >= tiles) return;
        const int g = BM == 256 && p.groups <= 64 ? longest_first(p, q, total, lane) : q;
        const int r0 = __builtin_amdgcn_readfirstlane(load_offset(p, g, total));
        const int r1 = max(r0, __builtin_amdgcn_readfirstlane(load_offset(p, g + 1, total)));
        int tm, tn;
        grouped_order(t, p.tiles_m, p.tiles_n, tm, tn);
        const TileAt at = tile_at<DT, AK, BKC, MODE, BM, BN>(p, g, r0, r1, tm, tn);
        T::run(p, at, at.group * p.sC + at.row0 * p.ldc + at.col0, (DMP_LDS char *)lds_a0, (DMP_LDS char *)lds_b0,
               (DMP_LDS char *)lds_a1, (DMP_LDS char *)lds_b1);
    } else {
        // the grid is the most row tiles there can be; the ones past the last leave
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
        if ((int)blockIdx.x >= parts) return;
        const bool cut = (int)blockIdx.x >= whole;
        const int i = cut ? whole + ((int)blockIdx.x - whole) / 4 : xcd_remap(blockIdx.x, whole);
        int g, r0, r1, tile0;
        if (!walk.find(p, total, lane, i / p.tiles_n, g, r0, r1, tile0)) return;
        int tm, tn;
        grouped_order(i - tile0 * p.tiles_n, (r1 - r0 - 1) / BM + 1, p.tiles_n, tm, tn);
        if constexpr (BM == 256) {
            if (cut) {
                const int part = ((int)blockIdx.x - whole) % 4;
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
