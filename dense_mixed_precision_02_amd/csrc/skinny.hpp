// skinny.hpp -- products of few rows by large K-contiguous matrices (decoding).
//
// With a few rows to a group the time is that of reading every B_g once.  A
// workgroup takes 16 TN columns of one group; its NW waves split K and each
// streams its share of the columns from memory straight into matrix-instruction
// operands (lane L: column L % 16, granules L / 16 and L / 16 + 4 of a 128-byte
// k-tile), two stages of U k-tiles in registers, so that a stage's loads are in flight
// while the one before is multiplied.  No LDS on the way; A's rows come the
// same way out of the caches.  At the end the waves' sums meet in LDS and are
// added in the order of the waves (the same result every run).  Rows go 16 or
// 32 at a time (16-bit operands with TN = 2: 32 or 64; the widened 8-bit ones
// would not fit the registers); a group with more reads its B again, by then
// from the caches, one pass after the other (which a long group makes slow: grouped_cfg
// has the figures).  64 groups of one row, bf16 4096 x 1024: 92 us, 5.8 TB/s.
//
// skinny_n does the same for N-contiguous B (16-bit operands): 92 us.
//
// 8-bit operands (SCALED) are widened to bf16 exactly as in scaled_tile.hpp:
// the matrix units idle here anyway, so every D type gets exact products.
// (64 groups of one row, 1024 x 4096: 56 us, 4.8 TB/s.)  Whether a factor has to be taken
// apart is noted in the loop and done after it (scaled_tile.hpp's Factor; 16 rows by 4096
// x 8192 with warm weights 8.6 us, 8.3 without).
#pragma once
#include "scaled_tile.hpp"

namespace dmp {

__device__ static inline intx4 load_granule(__amdgpu_buffer_rsrc_t r, int off) {
    return __builtin_bit_cast(intx4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// The sums of the waves (lds[wave][row][column]), added in the order of the waves,
// through the output stage.
template <int NW, int CW, int SZ>
__device__ static inline void join_waves(const RaggedArgs &p, const float *lds, int64_t row0, int rows,
                                         int64_t col0, int cols) {
    step_sync();
    __syncthreads();
    for (int e = threadIdx.x; e < rows * CW; e += NW * 64) {
        const int r = e / CW, c = e % CW;
        if (c >= cols) continue;
        float v = lds[e];
        for (int w = 1; w < NW; ++w) v += lds[w * SZ + e];
        const int64_t idx = (row0 + r) * p.ldc + col0 + c;
        const floatx4 cv = p.ep.use_c ? load4<float>(p.C, idx, p.ep.c_type, false, 1) : floatx4{0, 0, 0, 0};
        store4<float>(p.D, idx, finish4(floatx4{v, 0, 0, 0}, cv, p.ep), p.ep.d_type, false, 1);
    }
    step_sync();
}

// One group's rows [row0, row0 + rows), rows <= 16 TM, times this workgroup's columns.
template <class DT, int MODE, int TM, int TN, int NW, int FA, int FB>
__device__ static inline void skinny_rows(const RaggedArgs &p, float *lds, int g, int64_t row0, int rows,
                                          int64_t col0, int cols) {
    constexpr int U = TM + TN <= 2 ? 4 : TM + TN <= 3 ? 2 : 1;  // k-tiles in a stage
    constexpr int ESZ = DT::ESZ, KT = 128 / ESZ;
    const int lane = lane_id(), wave = wave_id();
    const int nkt = (int)((p.K + KT - 1) / KT);
    const int per = (nkt + NW - 1) / NW, kt0 = min(wave * per, nkt), kt1 = min(kt0 + per, nkt);
    const int kbytes = (int)(p.K * ESZ);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc((const char *)p.A + row0 * p.lda * ESZ);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc((const char *)p.B + (g * p.sB + col0 * p.ldb) * ESZ);
    const int r16 = lane & 15, gr = (lane >> 4) * 16;  // this lane's row or column; byte of its first granule

    floatx4 acc[TM][TN] = {};
    intx4 fa[2][U][TM][2], fb[2][U][TN][2];
    float fs[2][U][TM];  // SCALED: lane L holds the factor of row L % 16
    float fsb[2][U];
    auto load = [&](int st, int kt) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (kt + u) * 128 + gr;
            const bool in = kt + u < kt1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kb = k + 64 * h;
                const bool ok = in && kb < kbytes;
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int c = j * 16 + r16;
                    fb[st][u][j][h] = load_granule(rb, ok && c < cols ? c * (int)(p.ldb * ESZ) + kb : OOB_OFFSET);
                }
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int r = i * 16 + r16;
                    fa[st][u][i][h] = load_granule(ra, ok && r < rows ? r * (int)(p.lda * ESZ) + kb : OOB_OFFSET);
                }
            }
            if constexpr (MODE == RAGGED_SCALED) {
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int r = i * 16 + r16;
                    fs[st][u][i] = in && r < rows ? p.sa[(row0 + r) * p.sa_row + (kt + u) * p.sa_k] : 0.0f;
                }
                fsb[st][u] = in ? p.sb[g * p.sb_group + (col0 >> 7) * p.sb_col + (kt + u) * p.sb_k] : 0.0f;
            }
        }
    };
    bool leaves = false;  // SCALED: this lane's factors left the normal numbers (scaled_tile.hpp's Factor)
    auto multiply = [&](auto split, int st) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (MODE == RAGGED_SCALED) {
                intx4 b[TN][4];
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int h = 0; h < 4; ++h) b[j][h] = widen8<FB>(fb[st][u][j][h >> 1], h & 1);
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const float own = fs[st][u][i] * fsb[st][u];
                    leaves |= factor_leaves(fs[st][u][i], fsb[st][u], own);
                    floatx4 s;
                    int e[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int from = 4 * (lane >> 4) + q;
                        if constexpr (decltype(split)::value) {
                            const Factor f = split_factor(__shfl(fs[st][u][i], from, 64), fsb[st][u]);
                            s[q] = f.s;
                            e[q] = f.e;
                        } else {
                            s[q] = __shfl(own, from, 64);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        floatx4 c = {0, 0, 0, 0};
#pragma unroll
                        for (int h = 0; h < 4; ++h)
                            c = mma16<BF16>(widen8<FA>(fa[st][u][i][h >> 1], h & 1), b[j][h], c);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if constexpr (decltype(split)::value) acc[i][j][q] = add_scaled(s[q], e[q], c[q], acc[i][j][q]);
                            else acc[i][j][q] = __builtin_fmaf(s[q], c[q], acc[i][j][q]);
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j) acc[i][j] = mma16<DT>(fa[st][u][i][h], fb[st][u][j][h], acc[i][j]);
            }
        }
    };
    if (kt0 < kt1) {
        load(0, kt0);
        for (int kt = kt0; kt < kt1; kt += 2 * U) {
            load(1, kt + U);
            multiply(std::false_type{}, 0);
            load(0, kt + 2 * U);
            multiply(std::false_type{}, 1);
        }
    }
    if constexpr (MODE == RAGGED_SCALED) {
        if (__builtin_expect(__ballot(leaves) != 0, 0)) {  // once more with split factors
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = floatx4{0, 0, 0, 0};
            for (int kt = kt0; kt < kt1; kt += U) {
                load(0, kt);
                multiply(std::true_type{}, 0);
            }
        }
    }
    // sums of the waves, [wave][row][column]
    constexpr int CW = 16 * TN, SZ = 16 * TM * CW;
    step_sync();
    __syncthreads();  // the sums of the rows before are read
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                lds[wave * SZ + (i * 16 + 4 * (lane >> 4) + q) * CW + j * 16 + (lane & 15)] = acc[i][j][q];
    join_waves<NW, CW, SZ>(p, lds, row0, rows, col0, cols);
}

// The same with N-contiguous B_g, on 128 columns: lane L loads eight rows of B, k =
// 8 (L / 16) .. + 7 of a step of 32, at columns 8 (L % 16) .. + 7, and turns the
// block in registers.  The t-th of its columns is then its operand of the t-th
// instruction, which so computes the columns t, 8 + t, ..., 120 + t.
template <class DT, int TM, int NW>
__device__ static inline void skinny_rows_n(const RaggedArgs &p, float *lds, int g, int64_t row0, int rows,
                                            int64_t col0, int cols) {
    constexpr int U = TM == 1 ? 2 : 1;  // steps in a stage
    const int lane = lane_id(), wave = wave_id();
    const int ns = (int)((p.K + 31) / 32);
    const int per = (ns + NW - 1) / NW, s0 = min(wave * per, ns), s1 = min(s0 + per, ns);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc((const char *)p.A + row0 * p.lda * 2);
    const char *Bg = (const char *)p.B + (g * p.sB + col0) * 2;
    const int r16 = lane & 15, k8 = 8 * (lane >> 4), c8 = 8 * r16;
    const int ld = (int)p.ldb * 2, boff = k8 * ld + c8 * 2;

    floatx4 acc[TM][8] = {};
    intx4 fa[2][U][TM], fb[2][U][8];
    auto load = [&](int st, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * 32 + k8;
            const bool ok = s + u < s1 && k < (int)p.K;
            const __amdgpu_buffer_rsrc_t rb = make_rsrc(Bg + (int64_t)(s + u) * 32 * ld);
#pragma unroll
            for (int r = 0; r < 8; ++r) fb[st][u][r] = load_granule(rb, ok && c8 < cols ? boff + r * ld : OOB_OFFSET);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int r = i * 16 + r16;
                fa[st][u][i] = load_granule(ra, ok && r < rows ? r * (int)(p.lda * 2) + k * 2 : OOB_OFFSET);
            }
        }
    };
    auto multiply = [&](int st) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                intx4 b;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    b[d] = (int)__builtin_amdgcn_perm((uint32_t)fb[st][u][2 * d + 1][t / 2], (uint32_t)fb[st][u][2 * d][t / 2],
                                                      t % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
                for (int i = 0; i < TM; ++i) acc[i][t] = mma16<DT>(fa[st][u][i], b, acc[i][t]);
            }
    };
    if (s0 < s1) {
        load(0, s0);
        for (int s = s0; s < s1; s += 2 * U) {
            load(1, s + U);
            multiply(0);
            load(0, s + 2 * U);
            multiply(1);
        }
    }
    constexpr int CW = 128, SZ = 16 * TM * CW;
    step_sync();
    __syncthreads();  // the sums of the rows before are read
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float *at = lds + wave * SZ + (i * 16 + 4 * (lane >> 4) + q) * CW + c8;
#pragma unroll
            for (int t = 0; t < 8; ++t) at[t] = acc[i][t][q];
        }
    join_waves<NW, CW, SZ>(p, lds, row0, rows, col0, cols);
}

template <class DT, int MODE, int TN, int NW, int FA, int FB>
__global__ __launch_bounds__(NW * 64, 2) void skinny(const RaggedArgs p) {
    constexpr int TS = TN == 1 || MODE == RAGGED_SCALED ? 1 : 2;  // passes of 16 TS and 32 TS rows
    __shared__ float lds[NW * 32 * TS * 16 * TN];
    const int total = (int)p.M, id = workgroup_id();
    const int g = id / p.tiles_n;
    if (g >= p.groups) return;
    const int64_t col0 = (int64_t)(id - g * p.tiles_n) * 16 * TN;
    const int cols = (int)min((int64_t)16 * TN, p.N - col0);
    int r0 = 0, r1 = total;
    if (p.offsets) {
        r0 = load_offset(p, g, total);
        r1 = load_offset(p, g + 1, total);
    }
    for (int r = r0; r < r1; r += 32 * TS) {
        const int n = min(32 * TS, r1 - r);
        if (n <= 16 * TS) skinny_rows<DT, MODE, TS, TN, NW, FA, FB>(p, lds, g, r, n, col0, cols);
        else skinny_rows<DT, MODE, 2 * TS, TN, NW, FA, FB>(p, lds, g, r, n, col0, cols);
    }
}

// 16-bit operands, N-contiguous B: 128 columns to a workgroup.
template <class DT, int NW>
__global__ __launch_bounds__(NW * 64, 8 / NW) void skinny_n(const RaggedArgs p) {
    __shared__ __attribute__((aligned(16))) float lds[NW * 32 * 128];
    const int total = (int)p.M, id = workgroup_id();
    const int g = id / p.tiles_n;
    if (g >= p.groups) return;
    const int64_t col0 = (int64_t)(id - g * p.tiles_n) * 128;
    const int cols = (int)min((int64_t)128, p.N - col0);
    const int r0 = load_offset(p, g, total), r1 = load_offset(p, g + 1, total);
    for (int r = r0; r < r1; r += 32) {
        const int n = min(32, r1 - r);
        if (n <= 16) skinny_rows_n<DT, 1, NW>(p, lds, g, r, n, col0, cols);
        else skinny_rows_n<DT, 2, NW>(p, lds, g, r, n, col0, cols);
    }
}

}  // namespace dmp
