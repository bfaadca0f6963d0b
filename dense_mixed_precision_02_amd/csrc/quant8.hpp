// quant8.hpp -- 8-bit float operands with a scale for each block.
//
// A block is 128 consecutive k of one row (block == 1) or of 128 rows
// (block == 128).  With top the type's largest value (e4m3 448, e5m2 57344)
// and a = max(largest magnitude of the block, 2^-100),
//     scale = a / top,   q = round8(x * (top / a)),
// every step a 32-bit float operation, round8 to nearest even.  The floor of
// 2^-100 keeps top / a finite for blocks of zeros and of vanishing values.  A
// block that holds an infinity or a NaN gets the scale NaN and zeros, so that
// every product that uses it shows it.  Magnitudes are compared as the bit
// patterns of |x|, whose order is that of the values with infinity and then
// NaN above them all.
//
// Output: Q[b][i][k], rows of Kp = 16 ceil(K / 16) bytes, zeros past K (the
// products read whole 16-byte granules), and scale[b][k / 128][i / block]: for
// one k-block the factors of neighbouring rows lie next to each other, which is
// how a product's tile reads them.
//
// Both kernels are bound by HBM: one read of X and one write of Q (bf16: 8192 x 4096 by
// rows 19.7 us, 5.2 TB/s, from a column-major X 28 us, 3.6 TB/s; 8 x 4096 x 2048 by blocks
// of 128 rows 42 us, 4.8 TB/s).  Rows shorter than the 1024 k that a wave of quant8_rows
// spans leave lanes idle: the same 32M elements as rows of 1024: 22 us, of 256: 43, of 128: 78.
#pragma once
#include "common.hpp"
#include "ragged.hpp"

namespace dmp {

struct Quant8Args {
    const void *X;
    uint8_t *Q;
    float *scale;
    int64_t M, K, ldx, Kp, sX;  // sX: elements between batch entries
    int KB;                     // k-blocks
    int64_t MB;                 // row blocks (rows, or ceil(M / 128))
    int64_t tiles_m;
    int batch;
};

template <int FMT> constexpr float F8_TOP = FMT == 0 ? 448.0f : 57344.0f;
constexpr float QUANT8_LEAST = 0x1p-100f;
constexpr uint32_t F32_INF_BITS = 0x7f800000u;

// Sixteen consecutive elements as floats; n of them exist.  XT: OUT_F32, OUT_F16 or OUT_BF16.
template <int XT>
__device__ static inline void load16(const void *base, int64_t idx, int n, float (&x)[16]) {
    if constexpr (XT == OUT_F32) {
        const float *q = (const float *)base + idx;
        if (n >= 16) {
            floatx4 v[4];
            __builtin_memcpy(v, q, 64);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = v[e >> 2][e & 3];
            return;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = e < n ? q[e] : 0.0f;
    } else {
        const uint16_t *q = (const uint16_t *)base + idx;
        if (n >= 16) {
            intx4 v[2];
            __builtin_memcpy(v, q, 32);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t w = (uint32_t)v[e >> 3][(e & 7) >> 1];
                x[e] = decode16((uint16_t)(e & 1 ? w >> 16 : w), XT == OUT_F16);
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = e < n ? decode16(q[e], XT == OUT_F16) : 0.0f;
    }
}

__device__ static inline uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

// A block's scale and the factor its elements are multiplied by, from the bit
// pattern of its largest magnitude; a factor of zero stands for "store zeros".
template <int FMT>
__device__ static inline void block_scale(uint32_t amax_bits, float &scale, float &factor) {
    if (amax_bits >= F32_INF_BITS) {
        scale = __builtin_bit_cast(float, 0x7fc00000u);
        factor = 0.0f;
        return;
    }
    const float a = fmaxf(__builtin_bit_cast(float, amax_bits), QUANT8_LEAST);
    scale = a / F8_TOP<FMT>;
    factor = F8_TOP<FMT> / a;
}

// Four values times the factor, rounded to 8 bits, in one word.
template <int FMT>
__device__ static inline uint32_t encode8(float x0, float x1, float x2, float x3, float f) {
    if (f == 0.0f) return 0;
    x0 *= f; x1 *= f; x2 *= f; x3 *= f;
    int w = 0;
    if constexpr (FMT == 0) {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(x0, x1, w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(x2, x3, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(x0, x1, w, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(x2, x3, w, true);
    }
    return (uint32_t)w;
}

// Row-major X, blocks of one row: eight lanes to a block, sixteen elements to a
// lane, so a wave takes 1024 consecutive elements of a row; a workgroup takes
// those columns of 16 rows, and writes their 8 x 16 scales row by row of the
// [k-block][row] table.
constexpr int QUANT_ROWS = 16;
template <int XT, int FMT>
__global__ __launch_bounds__(256) void quant8_rows(const Quant8Args p) {
    __shared__ float sc[8][QUANT_ROWS];
    const int kgroups = (p.KB + 7) / 8;
    const int id = workgroup_id(), kg = id % kgroups;
    const int64_t rest = id / kgroups;
    const int64_t b = rest / p.tiles_m, m0 = (rest % p.tiles_m) * QUANT_ROWS;
    if (b >= p.batch) return;
    const int lane = lane_id(), wave = wave_id();
    const int64_t k = (int64_t)kg * 1024 + lane * 16;
    const int64_t left = p.K - k;
    const int n = left >= 16 ? 16 : left > 0 ? (int)left : 0;
    constexpr int PER = QUANT_ROWS / 4;
    float x[PER][16];
#pragma unroll
    for (int t = 0; t < PER; ++t) {
        const int64_t i = m0 + wave * PER + t;
        load16<XT>(p.X, b * p.sX + i * p.ldx + k, i < p.M ? n : 0, x[t]);
    }
#pragma unroll
    for (int t = 0; t < PER; ++t) {
        uint32_t am = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) am = max(am, abs_bits(x[t][e]));
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) am = max(am, (uint32_t)__shfl_xor((int)am, d, 64));
        float s, f;
        block_scale<FMT>(am, s, f);
        if ((lane & 7) == 0) sc[lane >> 3][wave * PER + t] = s;
        const int64_t i = m0 + wave * PER + t;
        if (i < p.M && k < p.Kp) {
            intx4 v;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                v[w] = (int)encode8<FMT>(x[t][4 * w], x[t][4 * w + 1], x[t][4 * w + 2], x[t][4 * w + 3], f);
            *(intx4 *)(p.Q + (b * p.M + i) * p.Kp + k) = v;
        }
    }
    __syncthreads();
    if (threadIdx.x < 8 * QUANT_ROWS) {
        const int kb = kg * 8 + threadIdx.x / QUANT_ROWS, r = threadIdx.x % QUANT_ROWS;
        if (kb < p.KB && m0 + r < p.M)
            p.scale[(b * p.KB + kb) * p.MB + m0 + r] = sc[threadIdx.x / QUANT_ROWS][r];
    }
}

// 128 rows x 128 k of X: blocks of 128 rows, and column-major X (element (i, k)
// at X[i + k * ldx]) with either block.  Sixteen consecutive elements to a lane
// and load, eight lanes to a run of 128, four runs to a thread, all in
// registers between the maximum and the rounding.  A column-major X has its
// runs along the rows: the four k that a thread holds are neighbours, so it
// packs them into words, and the words pass through LDS to become rows.
template <int XT, int FMT, bool COL, bool ROWS128>
__global__ __launch_bounds__(256) void quant8_tile(const Quant8Args p) {
    constexpr int PITCH = 33;  // words to an LDS row: 8 lanes that write one word of rows 16 apart meet two banks
    __shared__ uint32_t am[128];
    __shared__ uint32_t q[COL ? 128 * PITCH : 1];
    const int id = workgroup_id(), kb = id % p.KB;
    const int64_t rest = id / p.KB;
    const int64_t b = rest / p.tiles_m, i0 = (rest % p.tiles_m) * 128;
    if (b >= p.batch) return;
    const int64_t k0 = (int64_t)kb * 128;
    const int tid = threadIdx.x, piece = tid & 7, line = tid >> 3;  // 32 lines
    const int rows = (int)min((int64_t)128, p.M - i0), ks = (int)min((int64_t)128, p.K - k0);
    if (tid < 128) am[tid] = 0;
    float x[4][16];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int l = line * 4 + t;  // row (row-major) or k (column-major) of the tile
        const int n = (COL ? l < ks : l < rows) ? (COL ? rows : ks) - 16 * piece : 0;
        const int64_t at = COL ? (k0 + l) * p.ldx + i0 : (i0 + l) * p.ldx + k0;
        load16<XT>(p.X, b * p.sX + at + 16 * piece, n, x[t]);
    }
    __syncthreads();
    if constexpr (ROWS128) {
        uint32_t m = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) m = max(m, abs_bits(x[t][e]));
        for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
        if ((tid & 63) == 0) am[tid >> 6] = m;
    } else {
        static_assert(COL || ROWS128, "row-major rows have their own kernel");
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            uint32_t m = 0;
#pragma unroll
            for (int t = 0; t < 4; ++t) m = max(m, abs_bits(x[t][e]));
#pragma unroll
            for (int d = 8; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
            if ((tid & 63) < 8) atomicMax(&am[16 * piece + e], m);
        }
    }
    __syncthreads();
    float s, f[ROWS128 ? 1 : 16];
    if constexpr (ROWS128) {
        block_scale<FMT>(max(max(am[0], am[1]), max(am[2], am[3])), s, f[0]);
        if (tid == 0) p.scale[(b * p.KB + kb) * p.MB + i0 / 128] = s;
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) block_scale<FMT>(am[16 * piece + e], s, f[e]);
        if (tid < rows) {
            float unused;
            block_scale<FMT>(am[tid], s, unused);
            p.scale[(b * p.KB + kb) * p.MB + i0 + tid] = s;
        }
    }
    if constexpr (COL) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            q[(16 * piece + e) * PITCH + line] =
                encode8<FMT>(x[0][e], x[1][e], x[2][e], x[3][e], f[ROWS128 ? 0 : e]);
        __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int r = line * 4 + t;
        if (r >= rows || k0 + 16 * piece >= p.Kp) continue;
        intx4 v;
#pragma unroll
        for (int w = 0; w < 4; ++w)
            v[w] = COL ? (int)q[r * PITCH + 4 * piece + w]
                       : (int)encode8<FMT>(x[t][4 * w], x[t][4 * w + 1], x[t][4 * w + 2], x[t][4 * w + 3], f[0]);
        *(intx4 *)(p.Q + (b * p.M + i0 + r) * p.Kp + k0 + 16 * piece) = v;
    }
}

}  // namespace dmp
