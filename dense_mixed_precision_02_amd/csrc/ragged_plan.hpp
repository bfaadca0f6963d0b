// ragged_plan.hpp -- host-side argument checks and kernel choice of the
// products over ragged groups, the 8-bit block-scaled products and the 8-bit
// quantization (plain C++: no HIP types).
#pragma once
#include "plan.hpp"

namespace dmp {
namespace plan {

constexpr unsigned GROUPED_FLAGS = GEMM_B_COLMAJOR | GEMM_OFFSETS_I32;
constexpr int64_t SIZE_MAX_1 = (1ll << 31) - 1024, LD_MAX = 1ll << 48, GROUPS_MAX = 1ll << 20;

// A grid's shape.  A launch takes fewer than 2^32 threads along x, so a grid has rows
// of 2^22 workgroups (of up to 512 threads); workgroup i is the (i % 2^22)-th of row
// i / 2^22 (workgroup_id()).  A last row that is not full ends in workgroups past the
// count, which the kernels let return.
constexpr int GRID_ROW_BITS = 22;
struct GridShape {
    unsigned x, y;
};
inline bool grid_shape(int64_t workgroups, GridShape &g) {
    if (workgroups < 1 || workgroups > 0x7fffffff) return false;
    const int64_t row = 1ll << GRID_ROW_BITS;
    g.x = (unsigned)std::min(workgroups, row);
    g.y = (unsigned)cdiv(workgroups, row);
    return true;
}

inline bool float_out(int t) { return t == GEMM_OUT_F32 || t == GEMM_OUT_F16 || t == GEMM_OUT_BF16; }

// The output stage's types and pointers (D, and C where it is read).
inline int check_outputs(const void *C, const void *D, const EpiParams &ep) {
    if (!D || (ep.use_c && !C)) return GEMM_ERR_INVALID_ARG;
    if (C == D && ep.use_c && ep.c_type != ep.d_type) return GEMM_ERR_INVALID_ARG;
    if ((ep.use_c && (uintptr_t)C % (uintptr_t)out_bytes(ep.c_type)) ||
        (uintptr_t)D % (uintptr_t)out_bytes(ep.d_type))
        return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

inline int check_sizes(gemm_handle_t h, int64_t groups, int64_t M, int64_t N, int64_t K,
                       int64_t ldc, const EpiParams &ep) {
    if (!h || M < 0 || N < 0 || K < 0 || groups < 0 || groups > GROUPS_MAX) return GEMM_ERR_INVALID_ARG;
    if (M > SIZE_MAX_1 || N > SIZE_MAX_1 || K > SIZE_MAX_1) return GEMM_ERR_INVALID_ARG;
    if (ldc < std::max<int64_t>(1, N) || ldc > LD_MAX) return GEMM_ERR_INVALID_ARG;
    if (!float_out(ep.c_type) || !float_out(ep.d_type)) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

inline bool offsets_ok(const void *offsets, unsigned flags) {
    return offsets && (uintptr_t)offsets % ((flags & GEMM_OFFSETS_I32) ? 4 : 8) == 0;
}

// D[i] = alpha A[i] B_g + beta C[i]: A M x K row-major, B_g K x N or N x K, D M x N.
inline int validate_grouped(gemm_handle_t h, const void *A, const void *B, const void *C, const void *D,
                            const void *offsets, int64_t groups, int64_t M, int64_t N, int64_t K,
                            int64_t lda, int64_t ldb, int64_t ldc, int dtype, unsigned flags,
                            const EpiParams &ep) {
    int rc = check_sizes(h, groups, M, N, K, ldc, ep);
    if (rc != GEMM_OK) return rc;
    if (dtype != GEMM_F16 && dtype != GEMM_BF16) return GEMM_ERR_INVALID_ARG;
    if (flags & ~GROUPED_FLAGS) return GEMM_ERR_INVALID_ARG;
    const bool bc = flags & GEMM_B_COLMAJOR;
    if (K > 0 && (lda < K || lda > LD_MAX || ldb < std::max<int64_t>(1, bc ? K : N) || ldb > LD_MAX))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0 || groups == 0) return GEMM_OK;
    if (!extent_ok(1, M, ldc, N)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!extent_ok(1, M, lda, K) || !extent_ok(groups, bc ? N : K, ldb, bc ? K : N)))
        return GEMM_ERR_INVALID_ARG;
    if (!offsets_ok(offsets, flags)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!A || !B || (uintptr_t)A % 2 || (uintptr_t)B % 2)) return GEMM_ERR_INVALID_ARG;
    return check_outputs(C, D, ep);
}

// D_g = alpha X_g^T Y_g + beta C_g: X K x M and Y K x N row-major, D_g M x N.
inline int validate_wgrad(gemm_handle_t h, const void *X, const void *Y, const void *C, const void *D,
                          const void *offsets, int64_t groups, int64_t M, int64_t N, int64_t K,
                          int64_t ldx, int64_t ldy, int64_t ldc, int dtype, unsigned flags,
                          const EpiParams &ep) {
    int rc = check_sizes(h, groups, M, N, K, ldc, ep);
    if (rc != GEMM_OK) return rc;
    if (dtype != GEMM_F16 && dtype != GEMM_BF16) return GEMM_ERR_INVALID_ARG;
    if (flags & ~(unsigned)GEMM_OFFSETS_I32) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (ldx < std::max<int64_t>(1, M) || ldx > LD_MAX || ldy < std::max<int64_t>(1, N) || ldy > LD_MAX))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0 || groups == 0) return GEMM_OK;
    if (!extent_ok(groups, M, ldc, N)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!extent_ok(1, K, ldx, M) || !extent_ok(1, K, ldy, N))) return GEMM_ERR_INVALID_ARG;
    if (!offsets_ok(offsets, flags)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!X || !Y || (uintptr_t)X % 2 || (uintptr_t)Y % 2)) return GEMM_ERR_INVALID_ARG;
    return check_outputs(C, D, ep);
}

inline int64_t k16(int64_t K) { return cdiv(K, 16) * 16; }

inline bool q8_operand_ok(const gemm_q8_t &o, int64_t K, int64_t groups, int64_t rows, int64_t blocks) {
    if (o.type != GEMM_E4M3 && o.type != GEMM_E5M2) return false;
    if (!o.q || !aligned16(o.q) || !o.scale || (uintptr_t)o.scale % 4) return false;
    if (o.ld < k16(K) || o.ld % 16 || o.ld > LD_MAX) return false;
    if (o.scale_row < 0 || o.scale_k < 0 || o.scale_row > LD_MAX || o.scale_k > LD_MAX) return false;
    if (groups > 1 && (o.group < 0 || o.group % 16 || o.group > LD_MAX || o.scale_group < 0 ||
                       o.scale_group > LD_MAX))
        return false;
    const __int128 lim = (__int128)1 << 48;
    return (__int128)(groups - 1) * (groups > 1 ? o.group : 0) + (__int128)rows * o.ld <= lim &&
           (__int128)(groups - 1) * (groups > 1 ? o.scale_group : 0) + (__int128)blocks * o.scale_row +
                   (__int128)cdiv(K, 128) * o.scale_k <= lim &&
           256 * o.ld < (1ll << 31) - (1ll << 22);  // offsets inside a tile fit 31 bits
}

inline int validate_scaled8(gemm_handle_t h, const gemm_q8_t *A, const gemm_q8_t *B, const void *C,
                            const void *D, const void *offsets, int64_t groups, int64_t M, int64_t N,
                            int64_t K, int64_t ldc, unsigned flags, const EpiParams &ep) {
    int rc = check_sizes(h, groups, M, N, K, ldc, ep);
    if (rc != GEMM_OK) return rc;
    if (flags & ~(unsigned)GEMM_OFFSETS_I32) return GEMM_ERR_INVALID_ARG;
    if (!offsets && groups != 1) return GEMM_ERR_INVALID_ARG;
    if (!A || !B) return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0 || groups == 0) return GEMM_OK;
    if (!extent_ok(1, M, ldc, N)) return GEMM_ERR_INVALID_ARG;
    if (offsets && !offsets_ok(offsets, flags)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!q8_operand_ok(*A, K, 1, M, M) || !q8_operand_ok(*B, K, groups, N, cdiv(N, 128))))
        return GEMM_ERR_INVALID_ARG;
    return check_outputs(C, D, ep);
}

inline int validate_quant8(gemm_handle_t h, const void *X, int64_t M, int64_t K, int64_t ldx, int x_type,
                           unsigned flags, int64_t batch, int block, int q_type, const void *Q,
                           const void *scale) {
    if (!h || M < 0 || K < 0 || batch < 0 || batch > (1ll << 30) || M > SIZE_MAX_1 || K > SIZE_MAX_1)
        return GEMM_ERR_INVALID_ARG;
    if (!float_out(x_type) || (flags & ~(unsigned)(GEMM_A_COLMAJOR | GEMM_SCALE_POW2))) return GEMM_ERR_INVALID_ARG;
    if ((block != 1 && block != 128) || (q_type != GEMM_E4M3 && q_type != GEMM_E5M2))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0 || batch == 0) return GEMM_OK;
    const bool col = flags & GEMM_A_COLMAJOR;
    if (ldx < (col ? M : K) || ldx > LD_MAX) return GEMM_ERR_INVALID_ARG;
    if (!extent_ok(batch, col ? K : M, ldx, col ? M : K) || !extent_ok(batch, M, k16(K), k16(K)))
        return GEMM_ERR_INVALID_ARG;
    if (!X || !Q || !scale || (uintptr_t)X % (uintptr_t)out_bytes(x_type) || !aligned16(Q) ||
        (uintptr_t)scale % 4)
        return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

// ---------------------------------------------------------------------------
// Which kernel.  The host knows the rows in all and the number of groups, not
// how the rows are spread; the rules go by the mean.
// ---------------------------------------------------------------------------

// K-contiguous B with 16, 32 and 64 columns to a workgroup; N-contiguous B.
enum { CFG_SKINNY1 = 16, CFG_SKINNY2 = 17, CFG_SKINNY4 = 18, CFG_SKINNY_N = 19 };

// Few rows to a group, K-contiguous B: the widest columns whose workgroups fill the
// device (us with 16 / 32 / 64 columns, weights from memory; 16 bits: 64 groups of one
// row, 1024 x 4096: 151 / 92 / 98, 2048 x 2048: 98 / 94 / 102; 8 bits: 64 groups of one
// row, 1024 x 4096: 143 / 78 / 56; 16 groups of 32 rows, 4096 x 512: 17 / 14.5 / 18.5; 16
// rows, 4096 x 8192: 12.8 / 10.8 / 15.3).  64 columns of 16 bits never gained much.
// A few 16-bit rows and a long K take 16 columns: the rows are cheap to read again
// and smaller pieces spread evener.  Their loop takes 8 k-tiles of a wave's quarter of K
// to a trip, so K is long where the second trip is all but full, 15 k-tiles to a wave
// (64 groups by 1024 columns, us with 16 / 32 columns, 64 rows one to a group / on
// 34 of the groups / 256 rows; K 3584, 14 k-tiles: 88.6 / 85.3, 50.5 / 53.2, 98.7 / 91.0;
// 3712, 15: 92.2 / 91.2, 52.0 / 57.2, 100.0 / 96.7; 3840: 92.7 / 96.4, 53.0 / 60.6, 103.1 /
// 103.9; 4096, 16: 92.4 / 92.8, 52.3 / 57.8, 100.6 / 98.5; 5120, 20: 126 / 133, 72.0 / 83.3,
// 139 / 144; 8192, 32: 190 / 207, 107 / 125, 203 / 211; and on the way a third trip that
// is mostly empty, 4608, 18: 117 / 108, 66.7 / 67.4, 129 / 116.  With 384 rows 4096 takes 106 / 102).
inline int skinny_cfg(int num_cus, int64_t groups, int64_t M, int64_t N, int64_t K, bool eight_bits) {
    if (eight_bits && groups * cdiv(N, 64) >= num_cus) return CFG_SKINNY4;
    if (!eight_bits && M <= 4 * groups && cdiv(cdiv(K, 64), 4) >= 15) return CFG_SKINNY1;
    return groups * cdiv(N, 32) >= num_cus ? CFG_SKINNY2 : CFG_SKINNY1;
}

// Grouped rows: 16-byte granules need aligned operands, whole granules along
// the contiguous extents and 31-bit offsets inside a tile.
inline int grouped_cfg(int num_cus, const void *A, const void *B, int64_t groups, int64_t M, int64_t N,
                       int64_t K, int64_t lda, int64_t ldb, bool b_col) {
    if (K == 0 || !granule_ok(A, B, M, N, K, lda, ldb, GEMM_F16, false, b_col, true)) return CFG_GENERIC;
    // Few rows to a group: kernels that stream B into registers, as long as they need
    // not pass over it often or the tiles would leave most of the device idle (us,
    // streamed against 128 x 128 tiles, weights from memory; B column-major: 64 groups of
    // one row, 4096 x 1024: 92 / 110, 8 groups of 64 rows, 1024 x 1024: 11 / 18, 4096 x
    // 4096: 100 / 65; row-major: 8 groups of one row, 4096 x 4096: 50 / 54, of 32 rows:
    // 54 / 56, of 64 rows: 94 / 57, 16 groups of 64 rows, 4096 x 512: 58 / 55).  That goes for
    // rows that are spread.  A workgroup takes a group's passes one after the other, so a long
    // group sets the time, and the host cannot see it (64 groups, 1024 rows, 4096 x 1024,
    // column- and row-major: shares that fall with the rank to the power of 0.7, longest
    // 148: 129 / 148 and 179 / 140; of 1.5, longest 463: 227 / 105 and 380 / 100; all in one
    // group: 364 / 51 and 592 / 55).
    const int64_t t128 = groups * cdiv(N, 128);
    if (b_col && (M <= 16 * groups || (M <= 64 * groups && 2 * t128 <= num_cus)))
        return skinny_cfg(num_cus, groups, M, N, K, false);
    if (!b_col && (M <= 32 * groups || (M <= 64 * groups && 4 * t128 <= num_cus))) return CFG_SKINNY_N;
    // 256 x 256 tiles where the mean group fills most of one and 128 x 128 ones, two to a
    // CU, would take more than one round of the device (us, 256 x 256 / 128 x 128 tiles,
    // column-major B, rows by chance over the groups; 8 groups by 4096 x 4096, 1536 rows, 512
    // small tiles: 125 / 85, 2048 rows, 640: 100 / 120, 4096 rows: 156 / 187; one group, 2000
    // rows, 512: 99 / 80, 2100 rows, 544: 88 / 114; 32 groups by 2048 x 1024, 6144 rows, 512:
    // 70 / 47, 7168 rows, 576: 59 / 66.  By the mean: 64 groups by 1024 x 2048, of 96 rows: 73 /
    // 59, of 192: 82 / 97, in shares that fall with the root of the rank 109 / 99)
    const int64_t small = (cdiv(M, 128) + groups / 2) * cdiv(N, 128);
    return M / groups >= 192 && small > 2 * (int64_t)num_cus ? CFG_L : CFG_M;
}

// Weight gradients: 256 x 256 tiles where they fill the device and lie mostly
// inside the outputs, else 64 x 128 ones (us, 256 x 256 / 64 x 128, bf16 results: 8
// groups of 1024 x 1024, half the device, 4096 rows: 30 / 22, 16384 rows: 62 / 60; 16 groups
// of them, 4096 rows: 25 / 26, 16384 rows: 42 / 59; 24 groups, 3000 rows: 37 / 30, the same of
// 520 x 1032, of which 0.55 of the tiles is useful: 43 / 23; 20 groups of 800 x 1100, 0.67,
// 6000 rows: 59 / 59; 12 groups of 1000 x 1500, 0.95: 80 / 80).
inline int wgrad_cfg(int num_cus, const void *X, const void *Y, int64_t groups, int64_t M, int64_t N,
                     int64_t K, int64_t ldx, int64_t ldy) {
    if (K == 0 || !granule_ok(X, Y, M, N, K, ldx, ldy, GEMM_F16, true, false, true)) return CFG_GENERIC;
    const int64_t t256 = cdiv(M, 256) * cdiv(N, 256);
    const double useful = (double)M * (double)N / ((double)t256 * 65536.0);
    return groups * t256 >= num_cus && useful >= 0.75 ? CFG_L : CFG_S;
}

inline int scaled_cfg(int num_cus, int64_t groups, int64_t M, int64_t N) {
    // as for 16 bits (us, streamed against 128 x 128 tiles, weights from memory: 8 groups of
    // 16 rows, 4096 x 4096: 32 / 40, of 32 rows: 38 / 41; 8 groups of 64 rows, 2048 x 1024:
    // 14 / 20; 16 such groups: 22 / 21; and as there a long group loses: 64 groups, 1024 rows,
    // 4096 x 1024, longest 463: 214 / 62, all in one: 405 / 26)
    if (M <= 16 * groups || (M <= 64 * groups && 4 * groups * cdiv(N, 128) <= num_cus))
        return skinny_cfg(num_cus, groups, M, N, 0, true);
    // 256 x 256 (fp32 results: 256 x 128) tiles where the mean group fills most of one
    // and they fill the device (us, large / 128 x 128 tiles, 4096 x 4096, 16-bit results: 8
    // equal groups, 2048 rows: 64 / 54, 4096 rows: 75 / 92; rows by chance, 2048: 64 / 83, 2560:
    // 65 / 81, 4096: 119 / 115; one group, 2000 rows: 57 / 42, 4096 rows: 63 / 80; 16 equal
    // groups, 8000 rows, 2064 x 4096: 93 / 128; fp32 results: 65 / 70 and 127 / 133; 111 / 94,
    // 113 / 99 and 168 / 149; 62 / 64 and 122 / 122; 149 / 158)
    const int64_t tiles = (cdiv(M, 256) + groups / 2) * cdiv(N, 256);
    return M / groups >= 192 && tiles >= num_cus ? CFG_L : CFG_M;
}

}  // namespace plan
}  // namespace dmp
