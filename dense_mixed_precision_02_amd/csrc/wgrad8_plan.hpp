// wgrad8_plan.hpp -- host-side argument checks and kernel choice of the weight gradients
// from 8-bit checkpoints (plain C++: no HIP types).
#pragma once
#include "ragged_plan.hpp"

namespace dmp {
namespace plan {

// Tiles, and the parts that the rows are split into.
struct Wgrad8Plan {
    int edge;     // 256: 256 x 256 tiles; 128: 128 x 128; 64: 64 x 128
    int splits;
};
inline Wgrad8Plan wgrad8_plan(int num_cus, int64_t groups, int64_t M, int64_t N, int64_t K) {
    if (groups == 0 || M == 0 || N == 0) return {64, 1};
    const int64_t rows = K / groups, t256 = groups * cdiv(M, 256) * cdiv(N, 256);
    const bool inside = (double)M * (double)N >= 0.75 * 65536.0 * (double)(cdiv(M, 256) * cdiv(N, 256));
    // In us with the join, 256 x 256 / 128 x 128 / 64 x 128 tiles, bf16, the parts as below.
    // 256 x 256 tiles where, with parts of 1024 rows at least, they fill most of the device and lie mostly
    // inside the gradients, and their rows are worth a large tile's start and end (4096 x 4096 of 2048 rows:
    // 80 / 111 / 123, of 512: 33 / 37 / 41; 2048 x 2048 of 8192: 94 / 113 / 126; 2000 x 3000 of 4096: 91 / 100 / 123;
    // 16 of 1024 x 1024, 1024 rows each: 51 / 60 / 72; 8 of 2048 x 2048, 512 rows each: 64 / 67 / 78)
    const int64_t large = t256 >= num_cus ? 1 : std::max<int64_t>(1, std::min(num_cus / t256, rows / 1024));
    if (inside && rows >= 512 && 4 * t256 * large >= 3 * num_cus) return {256, (int)large};
    // smaller ones, two to a CU, in parts of 512 and 256 rows at least (128 x 128 / 64 x 128: 1504 x 1504 of 4096
    // rows: 48 / 62; 1024 x 1024 of 8192: 39 / 41; 24 of 520 x 1032, 512 rows each: 43 / 42)
    const int64_t t128 = groups * cdiv(M, 128) * cdiv(N, 128), tiles = groups * cdiv(M, 64) * cdiv(N, 128);
    const int64_t s128 = std::max<int64_t>(1, std::min<int64_t>({2 * (int64_t)num_cus / t128, rows / 512, 16}));
    if (rows >= 512 && 4 * t128 * s128 >= 3 * num_cus) return {128, (int)s128};
    return {64, (int)std::max<int64_t>(1, std::min<int64_t>({2 * (int64_t)num_cus / tiles, rows / 256, 32}))};
}

constexpr int64_t WGRAD8_LD_MAX = 1ll << 23;

inline bool wgrad8_sizes_ok(int64_t groups, int64_t M, int64_t N, int64_t K) {
    return groups >= 0 && groups <= GROUPS_MAX && M >= 0 && N >= 0 && K >= 0 && M <= SIZE_MAX_1 && N <= SIZE_MAX_1 &&
           K <= SIZE_MAX_1;
}

// Can Y's 16-byte granules be loaded whole?  (Else it is copied first: pack.hpp.)
inline bool wgrad8_fast(const void *Y, int64_t N, int64_t ldy) { return aligned16(Y) && N % 8 == 0 && ldy % 8 == 0; }

// Scratch: Y's copy, and the parts' sums.
inline int64_t wgrad8_pack(const void *Y, int64_t N, int64_t K, int64_t ldy) {
    return wgrad8_fast(Y, N, ldy) ? 0 : K * cdiv(N, 8) * 16;
}
inline int64_t wgrad8_work(int num_cus, const void *Y, int64_t groups, int64_t M, int64_t N, int64_t K, int64_t ldy) {
    const int s = wgrad8_plan(num_cus, groups, M, N, K).splits;
    return wgrad8_pack(Y, N, K, ldy) + (s > 1 ? s * groups * M * N * 4 : 0);
}

inline int validate_wgrad8(gemm_handle_t h, const gemm_q8_t *X, const void *Y, const void *C, const void *D,
                           const void *offsets, int64_t groups, int64_t M, int64_t N, int64_t K, int64_t ldy,
                           int64_t ldc, int dtype, unsigned flags, const EpiParams &ep) {
    int rc = check_sizes(h, groups, M, N, K, ldc, ep);
    if (rc != GEMM_OK) return rc;
    if (dtype != GEMM_F16 && dtype != GEMM_BF16) return GEMM_ERR_INVALID_ARG;
    if (flags & ~(unsigned)GEMM_OFFSETS_I32) return GEMM_ERR_INVALID_ARG;
    if (!X || (!offsets && groups != 1)) return GEMM_ERR_INVALID_ARG;
    // (31-bit offsets in a k-tile of 64 rows)
    if (K > 0 && (ldy < std::max<int64_t>(1, N) || ldy > WGRAD8_LD_MAX)) return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0 || groups == 0) return GEMM_OK;
    if (!extent_ok(groups, M, ldc, N)) return GEMM_ERR_INVALID_ARG;
    if (offsets && !offsets_ok(offsets, flags)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!extent_ok(1, K, ldy, N) || !q8_operand_ok(*X, M, 1, K, K) || !Y || (uintptr_t)Y % 2))
        return GEMM_ERR_INVALID_ARG;
    return check_outputs(C, D, ep);
}

// The large tiles read X's factors by 31-bit offsets inside a k-tile.
inline bool wgrad8_narrow(const gemm_q8_t &X) { return X.scale_row < (1ll << 22) && X.scale_k < (1ll << 26); }

}  // namespace plan
}  // namespace dmp
