// ragged.hpp -- what the products over ragged groups of rows share: arguments,
// 8-bit float types, the search for a tile's group, and the kernel that takes
// any size, alignment and layout.
//
// Rows (tokens) are sorted by group (expert); offsets[g] .. offsets[g+1] are the
// rows of group g.  Three products use them:
//   ROWS    D[i] = alpha * A[i] B_g + beta * C[i] for the rows i of group g.
//           The rows are ragged, N and K are common.  (Forward, and with the
//           other layout of B the input gradient.)
//   WGRAD   D_g = alpha * X_g^T Y_g + beta * C_g: the reduction is ragged, the
//           M x N outputs are common.
//   SCALED  ROWS on 8-bit float operands with a factor for every 128 k of a row
//           of A and for every 128 x 128 block of B.
// The offsets stay on the device: the host knows only their number and the
// total of the rows, so it launches a grid from these two, and a workgroup
// finds its tiles by scanning the offsets (one wave-wide load and two prefix
// scans for each 64 groups).
#pragma once
#include "common.hpp"
#include "tile16_gemm.hpp"

namespace dmp {

enum { RAGGED_ROWS = 0, RAGGED_WGRAD = 1, RAGGED_SCALED = 2 };

typedef int32_t intx8 __attribute__((ext_vector_type(8)));

// 8-bit floats, by the operand format codes of the mixed 8/6/4-bit matrix
// instructions (0: e4m3, 1: e5m2).  FA, FB: the formats of A and B.  Staging
// and fragments are those of any one-byte type.
template <int FA, int FB> struct F8 {
    using elem = uint8_t;
    using acc = float;
    static constexpr int ESZ = 1;
    static constexpr int G = 16;
    // One 16 x 16 x 128 step: a whole block of 128 k.  Lane L supplies row (A) or
    // column (B) L % 16 and 32 of the 128 k; which 32 is free as long as A and B agree.
    __device__ static inline floatx4 mma(const intx8 &a, const intx8 &b, const floatx4 &c) {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, FA, FB, 0, 0, 0, 0);
    }
};

struct RaggedArgs {
    const void *A, *B, *C;
    void *D;
    const void *offsets;     // groups + 1 row numbers on the device; NULL: one group of all rows
    const float *sa, *sb;    // SCALED: factors of A and B
    int64_t M, N, K;         // ROWS, SCALED: M rows in all.  WGRAD: K rows in all
    int64_t lda, ldb, ldc;
    int64_t sB, sC;          // elements between the groups' B (WGRAD: between their C and D: sC)
    int64_t sa_row, sa_k;    // SCALED: elements between A's factors of neighbouring rows / k-blocks
    int64_t sb_col, sb_k, sb_group;  // SCALED: the same of B's, by blocks of 128 columns
    int groups, off32;       // off32: the offsets are int32_t, else int64_t
    int tiles_m, tiles_n;    // WGRAD: both; ROWS, SCALED: tiles_n
    int cut;                 // ragged_tile: workgroups in a round, or 0
    EpiParams ep;
};

// Row number i of the offsets, brought into 0 .. total.  (In 32-bit steps: the
// scalar unit cannot compare 64-bit values, and one vector comparison would take
// everything that a tile derives from its rows into vector registers.)
__device__ static inline int load_offset(const RaggedArgs &p, int i, int total) {
    int lo, hi;
    if (p.off32) {
        lo = ((const int32_t *)p.offsets)[i];
        hi = lo >> 31;
    } else {
        const intx2 v = ((const intx2 *)p.offsets)[i];
        lo = v[0];
        hi = v[1];
    }
    return hi < 0 ? 0 : (hi > 0 || (uint32_t)lo > (uint32_t)total) ? total : lo;
}

__device__ static inline int wave_scan_add(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d, 64);
        if (lane >= d) v += o;
    }
    return v;
}
__device__ static inline int wave_scan_max(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d, 64);
        if (lane >= d) v = max(v, o);
    }
    return v;
}

// Walks the row tiles of all groups in ascending order, 64 groups at a time.
// Whatever the offsets hold, the rows that it hands out lie in 0 .. total and
// no two groups share one: each group's end is the largest offset so far.
// (So the number of row tiles is at most total / BM + groups.)
template <int BM>
struct GroupWalk {
    int chunk = 0, row_floor = 0;  // this chunk's first group; where its first group starts
    int first = 0;                 // row tiles before this chunk
    int lo, hi, upto;              // this lane's group: its rows, row tiles up to and with it
    int count;                     // row tiles in this chunk

    __device__ void load(const RaggedArgs &p, int total, int lane) {
        const int g = chunk + lane;
        if (p.offsets) {
            int e = g < p.groups ? load_offset(p, g + 1, total) : 0;
            int s = lane == 0 && chunk == 0 ? load_offset(p, 0, total) : row_floor;
            s = __builtin_amdgcn_readfirstlane(s);
            hi = max(wave_scan_max(e, lane), s);
            lo = __shfl_up(hi, 1, 64);
            if (lane == 0) lo = s;
        } else {
            lo = 0;
            hi = g == 0 ? total : 0;
        }
        const int t = hi > lo ? (hi - lo - 1) / BM + 1 : 0;
        upto = wave_scan_add(t, lane);
        count = __builtin_amdgcn_readlane(upto, 63);
    }
    __device__ bool next(const RaggedArgs &p, int total, int lane) {
        if (chunk + 64 >= p.groups) return false;
        first += count;
        row_floor = __builtin_amdgcn_readlane(hi, 63);
        chunk += 64;
        load(p, total, lane);
        return true;
    }
    // The group (and its rows) that holds row tile `t`, which is not before this chunk.
    __device__ bool find(const RaggedArgs &p, int total, int lane, int t, int &g, int &r0, int &r1,
                         int &tile0) {
        while (t >= first + count)
            if (!next(p, total, lane)) return false;
        const uint64_t before = __ballot(first + upto <= t);
        const int l = __builtin_amdgcn_readfirstlane(__popcll(before));
        g = chunk + l;
        r0 = __builtin_amdgcn_readlane(lo, l);
        r1 = __builtin_amdgcn_readlane(hi, l);
        tile0 = l == 0 ? first : first + __builtin_amdgcn_readlane(upto, l - 1);
        return true;
    }
    // All row tiles (walks to the last chunk).
    __device__ int all(const RaggedArgs &p, int total, int lane) {
        while (next(p, total, lane)) {}
        return first + count;
    }
};

// ---------------------------------------------------------------------------
// Any size, alignment and layout: 64 x 64 tiles of four waves, each 32 x 32 in
// 16 x 16 instructions.  A k-tile (128 bytes of K) comes through registers: a
// lane loads a 16-byte granule wherever it lies (unaligned 16-byte loads are
// allowed on global memory), element by element only where the granule crosses
// the operand's end, and writes it to the LDS place that the direct copies of
// the aligned kernels use.  The next k-tile's loads are in flight while this
// one is multiplied.  A K that is not a multiple of 8 leaves no other way than
// unaligned rows; the aligned kernels take everything else.
// ---------------------------------------------------------------------------
template <class DT, int R, bool KCONTIG>
struct AnyOperand {
    using Op = Operand<DT, R, 4, KCONTIG>;
    using elem = typename DT::elem;
    static constexpr int G = DT::G, CPW = Op::CPW;

    // granule of this lane in chunk j: rows / mn from `base` (element (row0, k0)),
    // `rows` valid rows, `kleft` valid k
    __device__ static intx4 load(const elem *base, int64_t ld, int wave, int lane, int j, int rows,
                                 int kleft) {
        const int bid = (j * 4 + wave) * 8 + (lane >> 3);
        int r, k, n;  // K-contiguous: row r, k .. k + n - 1; else row r .. r + n - 1, k
        const elem *q;
        if constexpr (KCONTIG) {
            r = bid;
            k = ((lane & 7) ^ swz(r)) * G;
            n = r < rows ? kleft - k : 0;
            q = base + r * ld + k;
        } else {
            const int kb = bid / (R / 16), mb = bid % (R / 16);
            k = DT::ESZ == 2 ? kb * 4 + ((lane & 7) >> 1) : kb * 8 + (lane & 7);
            r = mb * 16 + (DT::ESZ == 2 ? (lane & 1) * 8 : 0);
            n = k < kleft ? min(G, rows - r) : 0;
            q = base + (int64_t)k * ld + r;
        }
        intx4 v = {0, 0, 0, 0};
        if (n >= G) {
            __builtin_memcpy(&v, q, 16);
        } else if (n > 0) {
            constexpr int EPW = 4 / DT::ESZ;
#pragma unroll
            for (int e = 0; e < G; ++e)
                if (e < n) v[e / EPW] |= (int)((uint32_t)q[e] << (e % EPW * 8 * DT::ESZ));
        }
        return v;
    }
    __device__ static void store(DMP_LDS char *lds, int wave, int lane, int j, const intx4 &v) {
        *(DMP_LDS intx4 *)(lds + Op::chunk_offset(j * 4 + wave) + lane * 16) = v;
    }
};

template <class DT>
__device__ static inline floatx4 mma16(const intx4 &a, const intx4 &b, const floatx4 &c) {
    if constexpr (std::is_same_v<DT, F16>)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                      __builtin_bit_cast(half8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// What a tile of the three products is: its operands' corners and valid extents.
struct TileAt {
    const char *A, *B;       // element (first row, first k) of A, (first k, first column) of B
    int rows, cols, k;       // valid rows of A, columns of B (to the operand's end), k
    int64_t row0, col0;      // in D
    int group;
};

template <class DT, bool AK, bool BKC, int MODE, int BM, int BN>
__device__ static inline TileAt tile_at(const RaggedArgs &p, int g, int r0, int r1, int tm, int tn) {
    TileAt t;
    t.group = g;
    t.col0 = (int64_t)tn * BN;
    t.cols = (int)p.N - tn * BN;
    if constexpr (MODE == RAGGED_WGRAD) {
        t.row0 = (int64_t)tm * BM;
        t.rows = (int)p.M - tm * BM;
        t.k = r1 - r0;
        t.A = (const char *)p.A + ((int64_t)r0 * p.lda + t.row0) * DT::ESZ;
        t.B = (const char *)p.B + ((int64_t)r0 * p.ldb + t.col0) * DT::ESZ;
    } else {
        t.row0 = r0 + (int64_t)tm * BM;
        t.rows = r1 - r0 - tm * BM;
        t.k = (int)p.K;
        t.A = (const char *)p.A + t.row0 * p.lda * DT::ESZ;
        t.B = (const char *)p.B + (g * p.sB + (BKC ? t.col0 * p.ldb : t.col0)) * DT::ESZ;
    }
    return t;
}

template <class DT, bool AK, bool BKC, int MODE>
__global__ __launch_bounds__(256) void ragged_any(const RaggedArgs p) {
    constexpr int BM = 64, BN = 64, TM = 2, TN = 2;
    constexpr int KT = 128 / DT::ESZ;
    using LA = AnyOperand<DT, BM, AK>;
    using LB = AnyOperand<DT, BN, BKC>;
    using elem = typename DT::elem;
    __shared__ __attribute__((aligned(1024))) char lds_a[2][LA::Op::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b[2][LB::Op::BYTES];
    const int lane = lane_id(), wave = wave_id();
    const int wm = wave >> 1, wn = wave & 1;
    const int total = (int)(MODE == RAGGED_WGRAD ? p.K : p.M);

    TileAt at;
    if constexpr (MODE == RAGGED_WGRAD) {
        const int tiles = p.tiles_m * p.tiles_n;
        const int g = blockIdx.x / tiles, t = blockIdx.x - g * tiles;
        const int r0 = load_offset(p, g, total), r1 = max(r0, load_offset(p, g + 1, total));
        at = tile_at<DT, AK, BKC, MODE, BM, BN>(p, g, r0, r1, t / p.tiles_n, t % p.tiles_n);
    } else {
        GroupWalk<BM> walk;
        walk.load(p, total, lane);
        int g, r0, r1, tile0;
        const int t = blockIdx.x / p.tiles_n;
        if (!walk.find(p, total, lane, t, g, r0, r1, tile0)) return;
        at = tile_at<DT, AK, BKC, MODE, BM, BN>(p, g, r0, r1, t - tile0, blockIdx.x % p.tiles_n);
    }
    const int nkt = at.k / KT + (at.k % KT != 0);

    floatx4 acc[TM][TN] = {};
    intx4 ra[LA::CPW], rb[LB::CPW];
    auto fetch = [&](int kt) {
        const int64_t k0 = (int64_t)kt * KT;
        const int kleft = min(KT, at.k - kt * KT);
        const elem *A = (const elem *)at.A + (AK ? k0 : k0 * p.lda);
        const elem *B = (const elem *)at.B + (BKC ? k0 : k0 * p.ldb);
#pragma unroll
        for (int j = 0; j < LA::CPW; ++j) ra[j] = LA::load(A, p.lda, wave, lane, j, at.rows, kleft);
#pragma unroll
        for (int j = 0; j < LB::CPW; ++j) rb[j] = LB::load(B, p.ldb, wave, lane, j, at.cols, kleft);
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int j = 0; j < LA::CPW; ++j) LA::store((DMP_LDS char *)lds_a[buf], wave, lane, j, ra[j]);
#pragma unroll
        for (int j = 0; j < LB::CPW; ++j) LB::store((DMP_LDS char *)lds_b[buf], wave, lane, j, rb[j]);
    };
    if (nkt > 0) {
        fetch(0);
        put(0);
    }
    __syncthreads();
    for (int kt = 0; kt < nkt; ++kt) {
        if (kt + 1 < nkt) fetch(kt + 1);
        const DMP_LDS char *la = (const DMP_LDS char *)lds_a[kt & 1];
        const DMP_LDS char *lb = (const DMP_LDS char *)lds_b[kt & 1];
        intx4 fa[TM][2], fb[TN][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
                fa[i][s] = frag16<DT, typename LA::Op, BM, AK>(la, wm * 32 + i * 16, s, lane);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                fb[j][s] = frag16<DT, typename LB::Op, BN, BKC>(lb, wn * 32 + j * 16, s, lane);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mma16<DT>(fa[i][s], fb[j][s], acc[i][j]);
        if (kt + 1 < nkt) put((kt + 1) & 1);
        __syncthreads();
    }
    const int64_t base = MODE == RAGGED_WGRAD ? at.group * p.sC : 0;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = wm * 32 + i * 16 + 4 * (lane >> 4) + q, c = wn * 32 + j * 16 + (lane & 15);
                if (r >= at.rows || c >= at.cols) continue;
                const int64_t idx = base + (at.row0 + r) * p.ldc + at.col0 + c;
                const floatx4 a = {acc[i][j][q], 0, 0, 0};
                const floatx4 cv = p.ep.use_c ? load4<float>(p.C, idx, p.ep.c_type, false, 1)
                                              : floatx4{0, 0, 0, 0};
                store4<float>(p.D, idx, finish4(a, cv, p.ep), p.ep.d_type, false, 1);
            }
}

}  // namespace dmp
