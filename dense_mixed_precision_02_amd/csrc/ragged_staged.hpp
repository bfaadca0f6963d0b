// ragged_staged.hpp -- 16-bit products over ragged groups, operands staged
// through registers: for groups of middling size, and for every size, alignment
// and layout.
//
// A k-tile (128 bytes of K) comes from memory into registers, DEPTH k-tiles
// ahead, and goes to one of two LDS buffers just before its turn.  With groups of
// a hundred rows a k-tile's instructions take a few hundred cycles and the loads
// some thousands, so the time goes with the bytes in flight.  Registers hold
// more of them than LDS: at 128 x 128, two workgroups to a CU and four k-tiles
// each, 256 KB, where ragged_tile.hpp's direct copies have one k-tile each, 64 KB.
// Half of the tiles' LDS traffic is the price.
//
// LDS layouts and fragment reads are tile_gemm.hpp's and frag16's; without direct
// copies in flight the compiler lets the transposing reads run freely.
//
// FAST: operands whose 16-byte granules are aligned and whole, read through
// descriptors that turn what is out of range into zeros.  Otherwise a lane loads
// its granule wherever it lies (unaligned 16-byte loads are allowed on global
// memory), element by element only where it crosses the operand's end.
#pragma once
#include "ragged_tile.hpp"

namespace dmp {

// This lane's granules of one k-tile of an operand: chunks j = 0 .. CPW - 1, in the
// places of Operand::issue.
template <class DT, int R, bool KCONTIG, bool FAST>
struct Staged {
    using Op = Operand<DT, R, 4, KCONTIG>;
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
                const bool ok = KCONTIG ? op.row_or_k + 32 * j < rows && op.fixed < kleft
                                        : op.fixed < rows && op.row_or_k + Op::KSTEP * j < kleft;
                v[j] = __builtin_bit_cast(
                    intx4, __builtin_amdgcn_raw_buffer_load_b128(rs, ok ? op.off0 + j * op.step : OOB_OFFSET, 0, 0));
            }
        } else {
            constexpr int EPW = 4 / DT::ESZ;
#pragma unroll
            for (int j = 0; j < CPW; ++j) {
                const int r = KCONTIG ? op.row_or_k + 32 * j : op.fixed;
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
        for (int j = 0; j < CPW; ++j) *(DMP_LDS intx4 *)(lds + Op::chunk_offset(j * 4 + wave) + lane * 16) = v[j];
    }
};

template <class DT, int BM, int BN, bool AK, bool BKC, int MODE, bool FAST, int DEPTH>
__global__ __launch_bounds__(256, 2) void ragged_staged(const RaggedArgs p) {
    constexpr int WN = 2, WTM = BM / 2, WTN = BN / 2, TM = WTM / 16, TN = WTN / 16, KT = 128 / DT::ESZ;
    static_assert(DEPTH % 2 == 0, "a trip of DEPTH k-tiles ends on the buffer it began on");
    using SA = Staged<DT, BM, AK, FAST>;
    using SB = Staged<DT, BN, BKC, FAST>;
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
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            intx4 fa[TM], fb[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[i] = frag16<DT, typename SA::Op, BM, AK>(la, wm * WTM + i * 16, s, lane);
#pragma unroll
            for (int j = 0; j < TN; ++j) fb[j] = frag16<DT, typename SB::Op, BN, BKC>(lb, wn * WTN + j * 16, s, lane);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mma16<DT>(fa[i], fb[j], acc[i][j]);
        }
    };
    if (nkt > 0) {
        // (k-tiles past the end: a branch that every lane takes or none, so that short
        // sums do not load zeros)
#pragma unroll
        for (int s = 0; s < DEPTH; ++s)
            if (s < nkt) fetch(s, s);
        put(0, 0);
        barrier_vmcnt<63>();
        for (int kt = 0; kt < nkt; kt += DEPTH) {
#pragma unroll
            for (int s = 0; s < DEPTH; ++s) {
                // k-tile kt + s is in LDS buffer s % 2, the next DEPTH - 1 are on their way
                if (kt + s < nkt) {
                    if (kt + s + DEPTH < nkt) fetch(kt + s + DEPTH, s);
                    multiply(s % 2);
                    if (kt + s + 1 < nkt) put((s + 1) % DEPTH, (s + 1) % 2);
                    barrier_vmcnt<63>();
                }
            }
        }
    }
    __syncthreads();
    constexpr int SLAB = 32 * (WTN + 4) * 4;
    static_assert(2 * SLAB <= 2 * SA::Op::BYTES && 2 * SLAB <= 2 * SB::Op::BYTES, "slabs must fit");
    DMP_LDS char *slab = wave < 2 ? (DMP_LDS char *)&lds_a[0][0] + wave * SLAB : (DMP_LDS char *)&lds_b[0][0] + (wave - 2) * SLAB;
    const int64_t first = (MODE == RAGGED_WGRAD ? at.group * p.sC : 0) + at.row0 * p.ldc + at.col0;
    store_wave_tile<WTM, WTN>((DMP_LDS float *)slab, p.ep, (const char *)p.C + first * out_size(p.ep.c_type),
                              (char *)p.D + first * out_size(p.ep.d_type), p.ldc, at.rows, at.cols, wm * WTM,
                              wn * WTN, lane, [&](int i, int j) { return acc[i][j]; });
}

}  // namespace dmp
