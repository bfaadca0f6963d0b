// wgrad8.hpp -- weight gradients from 8-bit checkpoints of activations:
// D_g = alpha * X_g^T Y_g + beta * C_g, X in 8-bit floats with a factor for every 128
// columns of a row, Y in 16 bits.
//
// The sum runs over the rows, and a factor belongs to a row, so it cannot be taken out
// of the sum: X's values are widened to Y's type on their way into LDS, x = q * s in 32 bits
// and rounded once (exact for powers of two).  A lane loads 16 bytes, 16 columns of one
// row; widened they are a row of the 128-byte blocks (4 rows x 16 columns) that the
// transposing LDS reads take, so that from LDS on everything is as in the 16-bit
// gradients (ragged_staged.hpp): the panels, the fragments, two k-tiles (of 64 rows)
// ahead in registers, two LDS buffers.  Four neighbouring lanes take the four rows of a
// block: a wave's writes are one contiguous run of LDS.
//
// Rows are split where the gradients' tiles alone would leave CUs idle (wgrad8_plan);
// each part's sums go to memory in 32 bits, and wgrad8_join adds them in their order.
//
// Large gradients are bound by the matrix units and, beside them, LDS (4096 x 4096 of 8192 rows, bf16: 250
// us of a long loop, 1.1 PFLOP/s, a library product of 16-bit operands 1.2; 45 % of the matrix units'
// cycles after a pause, 293 us); many small ones by memory (24 of 520 x 1032, 3001 rows, fp16 with C and D in 32
// bits: 111 MB in 30 us).
#pragma once
#include "ragged_staged.hpp"
#include "wgrad8_plan.hpp"

namespace dmp {

struct Wgrad8Args {
    RaggedArgs r;       // A: q, lda its row in bytes; sa, sa_row, sa_k: factors
    int splits;
    int units;          // workgroups to a split
    int64_t part;       // elements of a split's partial sums
};

// Sixteen 8-bit values times s, rounded to DT.
template <class DT, int FMT>
__device__ static inline void widen16(const intx4 &q, float s, intx4 (&out)[2]) {
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        float a, b;
        if constexpr (FMT == 0) {
            const auto v = w % 2 ? __builtin_amdgcn_cvt_pk_f32_fp8(q[w / 2], true) : __builtin_amdgcn_cvt_pk_f32_fp8(q[w / 2], false);
            a = v[0];
            b = v[1];
        } else {
            const auto v = w % 2 ? __builtin_amdgcn_cvt_pk_f32_bf8(q[w / 2], true) : __builtin_amdgcn_cvt_pk_f32_bf8(q[w / 2], false);
            a = v[0];
            b = v[1];
        }
        a *= s;
        b *= s;
        if constexpr (std::is_same_v<DT, F16>) {
            typedef _Float16 h2 __attribute__((ext_vector_type(2)));
            out[w / 4][w % 4] = __builtin_bit_cast(int, h2{(_Float16)a, (_Float16)b});
        } else {
            typedef __bf16 b2 __attribute__((ext_vector_type(2)));
            out[w / 4][w % 4] = __builtin_bit_cast(int, b2{(__bf16)a, (__bf16)b});
        }
    }
}

__device__ static inline intx4 load_granule_at(__amdgpu_buffer_rsrc_t r, int off) {
    return __builtin_bit_cast(intx4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// This lane's granules (16 columns of a row) of a k-tile of X, widened into the panel Op.
template <class DT, int FMT, int R, int NW, int PAD>
struct Widened {
    using Op = Operand<DT, R, NW, false, PAD>;
    static constexpr int CPW = R / (16 * NW);          // granules to a lane
    static constexpr int KSTEP = 4 * (NW * 16) / (R / 16);  // rows between them
    static_assert(CPW >= 1 && (NW * 16) % (R / 16) == 0, "whole block rows between a lane's granules");
    const char *base;       // the tile's first byte of q
    const float *sc;        // the factor of this lane's column block in the tile's first row
    int64_t sa_row;
    int ld, k, mn, span, at;
    bool in;                // this lane's columns exist
    __device__ void init(const RaggedArgs &p, const char *q, int64_t row0, int64_t col0, int cols, int span_, int wave, int lane) {
        const int id = wave * 64 + lane, blk = id >> 2, kr = id & 3;
        const int mb = blk % (R / 16), kb = blk / (R / 16);
        k = 4 * kb + kr;
        mn = 16 * mb;
        in = mn < cols;
        base = q;
        ld = (int)p.lda;
        span = span_;
        sa_row = p.sa_row;
        // (a column block that exists, whatever the lane's columns)
        sc = p.sa + row0 * sa_row + ((col0 + (in ? mn : 0)) >> 7) * p.sa_k;
        at = Op::block_offset(kb, mb) + kr * 32;
    }
    __device__ void fetch(int kt, intx4 (&v)[CPW], float (&s)[CPW]) const {
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(base + (int64_t)kt * 64 * ld);
#pragma unroll
        for (int j = 0; j < CPW; ++j) {
            const int kk = k + KSTEP * j, row = kt * 64 + kk;
            const bool ok = in && row < span;
            v[j] = load_granule_at(rs, ok ? kk * ld + mn : OOB_OFFSET);
            s[j] = sc[(int64_t)min(row, span - 1) * sa_row];  // a row that exists
        }
    }
    __device__ void put(int kt, DMP_LDS char *lds, const intx4 (&v)[CPW], const float (&s)[CPW]) const {
#pragma unroll
        for (int j = 0; j < CPW; ++j) {
            intx4 w[2];
            // rows past the end: zeros, also where the last row's factor is none
            widen16<DT, FMT>(v[j], kt * 64 + k + KSTEP * j < span ? s[j] : 0.0f, w);
            DMP_LDS char *to = lds + at + j * (KSTEP / 4) * Op::ROW_BYTES;
            *(DMP_LDS intx4 *)to = w[0];
            *(DMP_LDS intx4 *)(to + 16) = w[1];
        }
    }
};

// This workgroup's tile: as my_tile's for gradients (runs of tiles to an XCD, longest
// groups first), for each split of the rows in turn.
template <class DT, int BM, int BN>
__device__ static inline bool wgrad8_at(const Wgrad8Args &p, int lane, TileAt &at, int &split, int &first_row) {
    const RaggedArgs &r = p.r;
    const int total = (int)r.K, all = workgroup_id();
    split = all / p.units;
    if (split >= p.splits) return false;
    const int id = all - split * p.units;
    const int tiles = r.tiles_m * r.tiles_n, runs = (tiles + r.run - 1) / r.run;
    const int seq = id / 8, s = seq / r.run, xcd = id % 8;
    const int u = 8 * s + (s % 2 ? 7 - xcd : xcd), q = u / runs;
    const int t = (u - q * runs) * r.run + seq - s * r.run;
    if (q >= r.groups || t >= tiles) return false;
    int g = q, r0 = 0, r1 = total;
    if (r.offsets) {
        if (r.groups <= 64) g = longest_first(r, q, total, lane);
        r0 = __builtin_amdgcn_readfirstlane(load_offset(r, g, total));
        r1 = max(r0, __builtin_amdgcn_readfirstlane(load_offset(r, g + 1, total)));
    }
    if (p.splits > 1) {
        const int per = ((r1 - r0 - 1) / p.splits / 64 + 1) * 64;  // whole k-tiles (r1 > r0: at least a share)
        r0 = (int)min((int64_t)r1, r0 + (int64_t)split * per);
        r1 = (int)min((int64_t)r1, (int64_t)r0 + per);
    }
    int tm, tn;
    grouped_order(t, r.tiles_m, r.tiles_n, tm, tn);
    at.group = g;
    at.row0 = (int64_t)tm * BM;
    at.col0 = (int64_t)tn * BN;
    at.rows = (int)r.M - tm * BM;
    at.cols = (int)r.N - tn * BN;
    at.k = r1 - r0;
    first_row = r0;
    at.A = (const char *)r.A + (int64_t)r0 * r.lda + at.row0;
    at.B = (const char *)r.B + ((int64_t)r0 * r.ldb + at.col0) * DT::ESZ;
    return true;
}

template <class DT, int FMT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM *WN * 64, 2) void wgrad8_tile(const Wgrad8Args p) {
    constexpr int NW = WM * WN, WTM = BM / WM, WTN = BN / WN, TM = WTM / 16, TN = WTN / 16, KT = 64;
    constexpr int DEPTH = 2;
    constexpr int PA = BM >= 128 ? 32 : 0, PB = BN >= 128 ? 32 : 0;  // see tile16_gemm
    using SA = Widened<DT, FMT, BM, NW, PA>;
    using SB = Staged<DT, BN, NW, false, true, PB>;
    __shared__ __attribute__((aligned(1024))) char lds_a[2][SA::Op::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b[2][SB::Op::BYTES];
    const int lane = lane_id(), wave = wave_id();
    const int wm = wave / WN, wn = wave % WN;
    TileAt at;
    int split, row0;
    if (!wgrad8_at<DT, BM, BN>(p, lane, at, split, row0)) return;
    const RaggedArgs &r = p.r;
    const int nkt = at.k / KT + (at.k % KT != 0);
    floatx4 acc[TM][TN] = {};
    if (nkt > 0) {
        SA a;
        SB b;
        a.init(r, at.A, row0, at.row0, at.rows, at.k, wave, lane);
        b.init(at.B, wave, lane, r.ldb, at.cols);
        intx4 ra[DEPTH][SA::CPW], rb[DEPTH][SB::CPW];
        float rs[DEPTH][SA::CPW];
        auto fetch = [&](int kt, int slot) {
            a.fetch(kt, ra[slot], rs[slot]);
            b.fetch(kt, at.k - kt * KT, rb[slot]);
        };
        auto put = [&](int kt, int slot, int buf) {
            a.put(kt, (DMP_LDS char *)lds_a[buf], ra[slot], rs[slot]);
            b.put((DMP_LDS char *)lds_b[buf], lane, rb[slot]);
        };
        auto multiply = [&](int buf) {
            const DMP_LDS char *la = (const DMP_LDS char *)lds_a[buf], *lb = (const DMP_LDS char *)lds_b[buf];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                intx4 fa[TM], fb[TN];
#pragma unroll
                for (int j = 0; j < TN; ++j) fb[j] = frag16<DT, typename SB::Op, BN, false>(lb, wn * WTN + j * 16, s, lane);
#pragma unroll
                for (int i = 0; i < TM; ++i) fa[i] = frag16<DT, typename SA::Op, BM, false>(la, wm * WTM + i * 16, s, lane);
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[i][j] = mma16<DT>(fa[i], fb[j], acc[i][j]);
            }
        };
        // k-tiles past the end are fetched as zeros: see ragged_staged
#pragma unroll
        for (int s = 0; s < DEPTH; ++s) fetch(s, s);
        put(0, 0, 0);
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
                put(kt + s + 1, (s + 1) % DEPTH, (s + 1) % 2);
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
    static_assert(NW <= INA || (NW - INA) * SLAB <= 2 * SB::Op::BYTES, "slabs must fit");
    DMP_LDS char *slab = wave < INA ? (DMP_LDS char *)&lds_a[0][0] + wave * SLAB
                                    : (DMP_LDS char *)&lds_b[0][0] + (wave - INA) * SLAB;
    const int64_t first = (int64_t)split * p.part + at.group * r.sC + at.row0 * r.ldc + at.col0;
    store_wave_tile<WTM, WTN, true>((DMP_LDS float *)slab, r.ep, (const char *)r.C + first * out_size(r.ep.c_type),
                              (char *)r.D + first * out_size(r.ep.d_type), r.ldc, at.rows, at.cols, wm * WTM,
                              wn * WTN, lane, [&](int i, int j) { return acc[i][j]; });
}

// 256 x 256 tiles on four waves, each 128 x 128 with its accumulators tied in place
// (tile16_gemm.hpp).  Four waves read 128 KB of fragments from LDS for a k-tile where eight
// of 128 x 64 read 192, next to 64 written: 1536 cycles of LDS beside 2048 of the
// matrix units.  One wave to a SIMD has nothing beside it, so everything is spread
// over the gaps between the matrix instructions (which leave 12 of 16 cycles): in the
// k-tile's first half the fragments of the second, and the next k-tile's granules from
// registers into LDS, X's widened on the way, each followed by the load of the one
// after it; in the second half, behind the barrier, the next k-tile's first fragments.
template <class DT, int FMT>
__global__ __launch_bounds__(256) void wgrad8_large_tile(const Wgrad8Args p) {
    constexpr int BM = 256, BN = 256, WN = 2, NW = 4, WTM = 128, WTN = 128, TM = 8, TN = 8, NI = TM * TN;
    using SA = Widened<DT, FMT, BM, NW, 32>;
    using SB = Staged<DT, BN, NW, false, true, 32>;
    __shared__ __attribute__((aligned(1024))) char lds_a0[SA::Op::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b0[SB::Op::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_a1[SA::Op::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b1[SB::Op::BYTES];
    DMP_LDS char *LA[2] = {(DMP_LDS char *)lds_a0, (DMP_LDS char *)lds_a1};
    DMP_LDS char *LB[2] = {(DMP_LDS char *)lds_b0, (DMP_LDS char *)lds_b1};
    const int lane = lane_id(), wave = wave_id();
    const int wm = wave / WN, wn = wave % WN;
    TileAt at;
    int split, row0;
    if (!wgrad8_at<DT, BM, BN>(p, lane, at, split, row0)) return;
    const RaggedArgs &r = p.r;
    const int nkt = at.k / 64 + (at.k % 64 != 0);
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
    if (nkt > 0) {
        SA a;
        SB b;
        a.init(r, at.A, row0, at.row0, at.rows, at.k, wave, lane);
        b.init(at.B, wave, lane, r.ldb, at.cols);
        intx4 ra[SA::CPW], rb[SB::CPW];
        float rs[SA::CPW];
        const int srow = (int)r.sa_row * 4;
        auto load_a = [&](int kt, int j) {
            const __amdgpu_buffer_rsrc_t q = make_rsrc(a.base + (int64_t)kt * 64 * a.ld);
            const __amdgpu_buffer_rsrc_t f = make_rsrc(r.sa + (row0 + (int64_t)kt * 64) * r.sa_row + (at.row0 >> 7) * r.sa_k);
            const int kk = a.k + SA::KSTEP * j;
            const bool ok = a.in && kt * 64 + kk < at.k;
            ra[j] = load_granule_at(q, ok ? kk * a.ld + a.mn : OOB_OFFSET);
            // (a row past the end: the factor 0)
            rs[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(f, ok ? kk * srow + (a.mn >> 7) * (int)r.sa_k * 4 : OOB_OFFSET, 0, 0));
        };
        auto load_b = [&](int kt, int j) {
            const __amdgpu_buffer_rsrc_t q = make_rsrc(SB::Op::tile_base(b.base, b.ld, 0, (int64_t)kt * 64));
            const bool ok = b.op.fixed < at.cols && b.op.row_or_k + SB::Op::KSTEP * j < at.k - kt * 64;
            rb[j] = load_granule_at(q, ok ? b.op.off0 + j * b.op.step : OOB_OFFSET);
        };
        auto put_a = [&](int buf, int j) {
            intx4 w[2];
            widen16<DT, FMT>(ra[j], rs[j], w);
            DMP_LDS char *to = LA[buf] + a.at + j * (SA::KSTEP / 4) * SA::Op::ROW_BYTES;
            *(DMP_LDS intx4 *)to = w[0];
            *(DMP_LDS intx4 *)(to + 16) = w[1];
        };
        auto put_b = [&](int buf, int j) {
            *(DMP_LDS intx4 *)(LB[buf] + SB::Op::chunk_offset(j * NW + wave) + lane * 16) = rb[j];
        };
        intx4 fa[2][TM], fb[2][TN];
        auto read_one = [&](int buf, int s, int x) {
            if (x < TN) fb[s][x] = frag16<DT, typename SB::Op, BN, false>(LB[buf], wn * WTN + x * 16, s, lane);
            else fa[s][x - TN] = frag16<DT, typename SA::Op, BM, false>(LA[buf], wm * WTM + (x - TN) * 16, s, lane);
        };
        auto ktile = [&](int kt, int cur) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    Mma16<DT>::run(acc[i][j], fa[0][i], fb[0][j]);
                    const int q = i * TN + j;
                    if (slot_has(q, TM + TN, NI)) read_one(cur, 1, q * (TM + TN) / NI);
                    if (slot_has(q, SB::CPW, NI)) {
                        const int c = q * SB::CPW / NI;
                        put_b(cur ^ 1, c);
                        load_b(kt + 2, c);
                    }
                    if (slot_has(q, SA::CPW, NI)) {
                        const int c = q * SA::CPW / NI;
                        put_a(cur ^ 1, c);
                        load_a(kt + 2, c);
                    }
                }
            step_sync();
            barrier_vmcnt<63>();
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    Mma16<DT>::run(acc[i][j], fa[1][i], fb[1][j]);
                    const int q = i * TN + j;
                    if (slot_has(q, TM + TN, NI)) read_one(cur ^ 1, 0, q * (TM + TN) / NI);
                }
            step_sync();
        };
#pragma unroll
        for (int j = 0; j < SA::CPW; ++j) load_a(0, j);
#pragma unroll
        for (int j = 0; j < SB::CPW; ++j) load_b(0, j);
#pragma unroll
        for (int j = 0; j < SA::CPW; ++j) {
            put_a(0, j);
            load_a(1, j);
        }
#pragma unroll
        for (int j = 0; j < SB::CPW; ++j) {
            put_b(0, j);
            load_b(1, j);
        }
        barrier_vmcnt<63>();
#pragma unroll
        for (int x = 0; x < TM + TN; ++x) read_one(0, 0, x);
        pin_acc();
        asm volatile("s_nop 7" ::);
        // two k-tiles to a trip so that each buffer is named statically; an odd count
        // runs one zero-filled k-tile more
        for (int kt = 0; kt < nkt; kt += 2) {
            ktile(kt, 0);
            ktile(kt + 1, 1);
        }
        mma_drain();
        pin_acc();
    }
    __syncthreads();
    DMP_LDS char *slab = wave == 0 ? LA[0] : wave == 1 ? LB[0] : wave == 2 ? LA[1] : LB[1];
    static_assert(32 * (WTN + 4) * 4 <= SA::Op::BYTES && 32 * (WTN + 4) * 4 <= SB::Op::BYTES, "slab must fit");
    const int64_t first = (int64_t)split * p.part + at.group * r.sC + at.row0 * r.ldc + at.col0;
    store_wave_tile<WTM, WTN, true>((DMP_LDS float *)slab, r.ep, (const char *)r.C + first * out_size(r.ep.c_type),
                              (char *)r.D + first * out_size(r.ep.d_type), r.ldc, at.rows, at.cols, wm * WTM,
                              wn * WTN, lane, [&](int i, int j) { return acc[i][j]; });
}

struct Wgrad8JoinArgs {
    const float *part;
    const void *C;
    void *D;
    int64_t rows, N, ldc;   // rows: of all groups
    int splits;
    EpiParams ep;
};

// D = the output stage of the splits' sums, added in their order: four values to a thread.
__global__ __launch_bounds__(256) void wgrad8_join(const Wgrad8JoinArgs p) {
    const int64_t quads = (p.N + 3) / 4, i = (int64_t)workgroup_id() * 256 + threadIdx.x;
    const int64_t row = i / quads, col = (i - row * quads) * 4;
    if (row >= p.rows) return;
    const int n = (int)min((int64_t)4, p.N - col);
    floatx4 v = {0, 0, 0, 0};
    for (int s = 0; s < p.splits; ++s)
        v += load4s<float, 4, true>(p.part, ((int64_t)s * p.rows + row) * p.N + col, false, true, n);
    const int64_t at = row * p.ldc + col;
    const floatx4 c = p.ep.use_c ? load4<float, true>(p.C, at, p.ep.c_type, true, n) : floatx4{0, 0, 0, 0};
    store4<float, true>(p.D, at, finish4(v, c, p.ep), p.ep.d_type, true, n);
}

}  // namespace dmp
