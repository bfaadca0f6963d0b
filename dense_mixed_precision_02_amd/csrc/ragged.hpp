// ragged.hpp -- what the products over ragged groups of rows share: arguments,
// 8-bit float types and the search for a tile's group.
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
#include "ragged_plan.hpp"
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

// This workgroup's number in a grid of plan::grid_shape.
__device__ static inline int workgroup_id() { return (int)(blockIdx.y << plan::GRID_ROW_BITS | blockIdx.x); }

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
    int cut;                 // ragged_tile, ROWS: workgroups in a round, or 0
    int run;                 // ragged_tile, WGRAD: tiles in a run (on one XCD)
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

}  // namespace dmp
