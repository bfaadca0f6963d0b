// wgrad8_plan.hpp -- host-side argument checks and kernel choice of the weight gradients
// from 8-bit checkpoints (plain C++: no HIP types).
#pragma once
#include "ragged_plan.hpp"

namespace dmp {
namespace plan {

// 256 x 256 tiles where they fill the device and lie mostly inside the gradients, else 64 x 128.
inline bool wgrad8_large(int num_cus, int64_t groups, int64_t M, int64_t N) {
    const int64_t t256 = cdiv(M, 256) * cdiv(N, 256);
    return groups * t256 >= num_cus && (double)M * (double)N >= 0.75 * 65536.0 * (double)t256;
}

// Parts that the rows are split into: by the number of rows and the gradients' 64 x 128
// tiles, two to a CU, in parts of 256 rows at least.
inline int wgrad8_splits(int num_cus, int64_t groups, int64_t M, int64_t N, int64_t K) {
    if (groups == 0 || M == 0 || N == 0 || wgrad8_large(num_cus, groups, M, N)) return 1;
    const int64_t tiles = groups * cdiv(M, 64) * cdiv(N, 128);
    const int64_t s = std::min<int64_t>(2 * (int64_t)num_cus / tiles, K / groups / 256);
    return (int)std::max<int64_t>(1, std::min<int64_t>(s, 32));
}

inline bool wgrad8_sizes_ok(int64_t groups, int64_t M, int64_t N, int64_t K) {
    return groups >= 0 && groups <= GROUPS_MAX && M >= 0 && N >= 0 && K >= 0 && M <= SIZE_MAX_1 && N <= SIZE_MAX_1 &&
           K <= SIZE_MAX_1;
}

// (splits only of few tiles: the product is below 2^31)
inline int64_t wgrad8_work(int num_cus, int64_t groups, int64_t M, int64_t N, int64_t K) {
    const int s = wgrad8_splits(num_cus, groups, M, N, K);
    return s > 1 ? (int64_t)s * groups * M * N * 4 : 0;
}

inline int validate_wgrad8(gemm_handle_t h, const gemm_q8_t *X, const void *Y, const void *C, const void *D,
                           const void *offsets, int64_t groups, int64_t M, int64_t N, int64_t K, int64_t ldy,
                           int64_t ldc, int dtype, unsigned flags, const EpiParams &ep) {
    int rc = check_sizes(h, groups, M, N, K, ldc, ep);
    if (rc != GEMM_OK) return rc;
    if (dtype != GEMM_F16 && dtype != GEMM_BF16) return GEMM_ERR_INVALID_ARG;
    if (flags & ~(unsigned)GEMM_OFFSETS_I32) return GEMM_ERR_INVALID_ARG;
    if (!X || (!offsets && groups != 1)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (ldy < std::max<int64_t>(1, N) || ldy > LD_MAX)) return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0 || groups == 0) return GEMM_OK;
    if (!extent_ok(groups, M, ldc, N)) return GEMM_ERR_INVALID_ARG;
    if (offsets && !offsets_ok(offsets, flags)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!extent_ok(1, K, ldy, N) || !q8_operand_ok(*X, M, 1, K, K) || !Y || (uintptr_t)Y % 2))
        return GEMM_ERR_INVALID_ARG;
    return check_outputs(C, D, ep);
}

// The large tiles read X's factors by 31-bit offsets inside a k-tile.
inline bool wgrad8_narrow(const gemm_q8_t &X) { return X.scale_row < (1ll << 22) && X.scale_k < (1ll << 26); }

// Can Y's 16-byte granules be loaded whole?
inline bool wgrad8_fast(const void *Y, int64_t N, int64_t ldy) {
    return aligned16(Y) && N % 8 == 0 && ldy % 8 == 0 && 128 * ldy < (1ll << 31) - (1ll << 22);
}

}  // namespace plan
}  // namespace dmp
