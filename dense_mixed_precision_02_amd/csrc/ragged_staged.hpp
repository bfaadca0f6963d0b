// ragged_staged.hpp -- 16-bit products over ragged groups, operands staged
// through registers: for groups of middling size, and for every size, alignment
// and layout.
//
// A k-tile (128 bytes of K) comes from memory into registers, two k-tiles ahead,
// and goes to one of two LDS buffers just before its turn.  With groups of a
// hundred rows a k-tile's instructions take a few hundred cycles and its loads
// some thousands, so the time goes with the bytes in flight, and registers add to
// what LDS holds (ragged_tile.hpp's direct copies have one k-tile on its way).
// Four k-tiles ahead measured the same as two.  A loop that reads half a k-tile's
// fragments beside the other half's instructions was 2 to 7 % faster for ROWS and 8 %
// slower for WGRAD, whose groups have few k-tiles: not kept.
//
// Measured: 32 groups, 5003 rows in all, by 2056 x 1000 row-major, fp32 results added to:
// 76 us, 2.5 TB/s; 24 gradients of 520 x 1032 from 3001 rows, fp32 results added to: 34
// us, 3.3 TB/s.  What bounds it is what one CU can have on its way: with one tile on
// a CU a k-tile of 32 KB takes 0.7 us, in this kernel as in scaled_tile's: 4096 of K take
// 50 us whatever the rows and columns, as long as there are no more tiles than CUs.
//
// LDS layouts and fragment reads are tile_gemm.hpp's and frag16's; without direct
// copies in flight the compiler lets the transposing reads run freely.
//
// FAST: operands whose 16-byte granules are aligned and whole, read through
// descriptors that turn what is out of range into zeros.  Otherwise a lane loads
// its granule wherever it lies (unaligned 16-byte loads are allowed on global
// memory), element by element only where it crosses the operand's end.  (5003 rows over
// 32 groups by 2057 x 1001: column-major 102 us, row-major 174, where 2056 x 1000 takes 64;
// 24 gradients of 521 x 1033 from 3001 rows: 88 us against 34 for 520 x 1032; 8 groups of
// 2048 rows by 4097 x 4097 1.6 ms.)
#pragma once
#include "ragged_tile.hpp"

namespace dmp {

// This lane's granules of one k-tile of an operand: chunks j = 0 .. CPW - 1, in the
// places of Operand::issue.
template <class DT, int R, int NW, bool KCONTIG, bool FAST, int PAD = 0>
struct Staged {
    using Op = Operand<DT, R, NW, KCONTIG, PAD>;
    using elem = typename DT::elem;
    static constexpr int G = DT::G, CPW = Op::CPW, KT = Op::KT;
    Op op;
    const char *base;
    int64_t ld;
    int wave, rows;
    __device__ void init(const char *X, int wave_, int lane, int64_t ld_, int rows_) {
        op.init(wave_, lane, ld_, 0, rows_);
        base = X;
        ld = ld_;
        wave = wave_;
        rows = rows_;
    }
    // k-tile kt, of which kleft values remain (none: not positive)
    __device__ void fetch(int kt, int kleft, intx4 (&v)[CPW]) const {
        const char *q = Op::tile_base(base, ld, 0, (int64_t)kt * KT);
        if constexpr (FAST) {
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(q);
#pragma unroll
            for (int j = 0; j < CPW; ++j) {
                const bool ok = KCONTIG ? op.row_or_k + 8 * NW * j < rows && op.fixed < kleft
                                        : op.fixed < rows && op.row_or_k + Op::KSTEP * j < kleft;
                v[j] = __builtin_bit_cast(
                    intx4, __builtin_amdgcn_raw_buffer_load_b128(rs, ok ? op.off0 + j * op.step : OOB_OFFSET, 0, 0));
            }
        } else {
            constexpr int EPW = 4 / DT::ESZ;
#pragma unroll
            for (int j = 0; j < CPW; ++j) {
                const int r = KCONTIG ? op.row_or_k + 8 * NW * j : op.fixed;
                const int k = KCONTIG ? op.fixed : op.row_or_k + Op::KSTEP * j;
                const int n = KCONTIG ? (r < rows ? kleft - k : 0) : (k < kleft ? rows - r : 0);
                const elem *e = (const elem *)q + (KCONTIG ? r * ld + k : k * ld + r);
                v[j] = intx4{0, 0, 0, 0};
                if (n >= G) {
                    __builtin_memcpy(&v[j], e, 16);
                } else if (n > 0) {
#pragma unroll
                    for (int i = 0; i < G; ++i)
                        if (i < n) v[j][i / EPW] |= (int)((uint32_t)e[i] << (i % EPW * 8 * DT::ESZ));
                }
            }
        }
    }
    __device__ void put(DMP_LDS char *lds, int lane, const intx4 (&v)[CPW]) const {
#pragma unroll
        for (int j = 0; j < CPW; ++j) *(DMP_LDS intx4 *)(lds + Op::chunk_offset(j * NW + wave) + lane * 16) = v[j];
    }
};

template <class DT, int BM, int BN, int WM, int WN, bool AK, bool BKC, int MODE, bool FAST>
__global__ __launch_bounds__(WM *WN * 64, 2) void ragged_staged(const RaggedArgs p) {
    constexpr int NW = WM * WN, WTM = BM / WM, WTN = BN / WN, TM = WTM / 16, TN = WTN / 16, KT = 128 / DT::ESZ;
    constexpr int DEPTH = 2;
    using SA = Staged<DT, BM, NW, AK, FAST>;
    using SB = Staged<DT, BN, NW, BKC, FAST>;
    __shared__ __attribute__((aligned(1024))) char lds_a[2][SA::Op::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b[2][SB::Op::BYTES];
    const int lane = lane_id(), wave = wave_id();
    const int wm = wave / WN, wn = wave % WN;
    TileAt at;
    if (!my_tile<DT, AK, BKC, MODE, BM, BN>(p, lane, at)) return;
    const int nkt = at.k / KT + (at.k % KT != 0);
    SA a;
    SB b;
    a.init(at.A, wave, lane, p.lda, at.rows);
    b.init(at.B, wave, lane, p.ldb, at.cols);

    floatx4 acc[TM][TN] = {};
    intx4 ra[DEPTH][SA::CPW], rb[DEPTH][SB::CPW];
    auto fetch = [&](int kt, int slot) {
        a.fetch(kt, at.k - kt * KT, ra[slot]);
        b.fetch(kt, at.k - kt * KT, rb[slot]);
    };
    auto put = [&](int slot, int buf) {
        a.put((DMP_LDS char *)lds_a[buf], lane, ra[slot]);
        b.put((DMP_LDS char *)lds_b[buf], lane, rb[slot]);
    };
    auto multiply = [&](int buf) {
        const DMP_LDS char *la = (const DMP_LDS char *)lds_a[buf], *lb = (const DMP_LDS char *)lds_b[buf];
        // all of the k-tile's fragments first: the reads' latency is met once
        intx4 fa[2][TM], fb[2][TN];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[s][i] = frag16<DT, typename SA::Op, BM, AK>(la, wm * WTM + i * 16, s, lane);
#pragma unroll
            for (int j = 0; j < TN; ++j) fb[s][j] = frag16<DT, typename SB::Op, BN, BKC>(lb, wn * WTN + j * 16, s, lane);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mma16<DT>(fa[s][i], fb[s][j], acc[i][j]);
    };
    const int64_t first = (MODE == RAGGED_WGRAD ? at.group * p.sC : 0) + at.row0 * p.ldc + at.col0;
    if (nkt > 0) {
        // K-tiles past the end are fetched too (out of range: zeros, no memory is
        // touched), so that on every path the same number of loads is in flight: behind
        // a branch the compiler would wait for all of them at each turn.
#pragma unroll
        for (int s = 0; s < DEPTH; ++s) fetch(s, s);
        put(0, 0);
        barrier_vmcnt<63>();
        bool done = nkt == 1;
        for (int kt = 0; !done; kt += DEPTH) {
#pragma unroll
            for (int s = 0; s < DEPTH; ++s) {
                // k-tile kt + s is in LDS buffer s % 2, the next DEPTH - 1 are on their way
                fetch(kt + s + DEPTH, s);
                asm volatile("" ::: "memory");  // issued here, not sunk to where it is needed
                __builtin_amdgcn_sched_barrier(0);
                step_sync();
                multiply(s % 2);
                put((s + 1) % DEPTH, (s + 1) % 2);
                step_sync();
                barrier_vmcnt<63>();
                if (kt + s + 2 >= nkt) {
                    done = true;
                    break;
                }
            }
        }
        multiply((nkt - 1) % 2);
    }
    __syncthreads();
    // each wave's slab in one of the operands' buffers, as many as fit A's
    constexpr int SLAB = 32 * (WTN + 4) * 4, INA = 2 * SA::Op::BYTES / SLAB;
    static_assert((NW - INA) * SLAB <= 2 * SB::Op::BYTES, "slabs must fit");
    DMP_LDS char *slab = wave < INA ? (DMP_LDS char *)&lds_a[0][0] + wave * SLAB
                                    : (DMP_LDS char *)&lds_b[0][0] + (wave - INA) * SLAB;
    // (C is read here, not ahead of the last k-tiles: fetching it into registers early
    // made no case faster and 520 x 1032 gradients slower, 36 -> 43 us)
    store_wave_tile<WTM, WTN>((DMP_LDS float *)slab, p.ep, (const char *)p.C + first * out_size(p.ep.c_type),
                              (char *)p.D + first * out_size(p.ep.d_type), p.ldc, at.rows, at.cols, wm * WTM,
                              wn * WTN, lane, [&](int i, int j) { return acc[i][j]; });
}

}  // namespace dmp
