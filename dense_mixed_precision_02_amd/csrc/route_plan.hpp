// route_plan.hpp -- host-side argument checks and sizes of the experts' router (plain
// C++: no HIP types).
#pragma once
#include "ragged_plan.hpp"

namespace dmp {
namespace plan {

constexpr int ROUTE_E_MAX = 1024, ROUTE_K_MAX = 64;

// Tokens to a workgroup and workgroups.  Up to 32 tokens, two turns of its 16 waves,
// one workgroup does everything in one launch; beyond, as many workgroups as CUs.  (Kernel
// time of one / two launches, the second costing 1 to 4 us beside it, bf16, 8 of 64 experts and 6 of
// 160: 32 tokens 11.6 / 9.8 and 13.7 / 10.6 us, 64 tokens 15.2 / 10.3 and 19.2 / 11.6.)
inline void route_split(int64_t T, int num_cus, int &rows, int &blocks) {
    if (T <= 32) {
        rows = 32;
        blocks = 1;
        return;
    }
    rows = (int)(cdiv(cdiv(T, num_cus), 16) * 16);
    blocks = (int)cdiv(T, rows);
}

// Bytes of scratch: counts and sums of each workgroup.
inline int64_t route_work(int64_t T, int64_t E, int num_cus) {
    int rows, blocks;
    route_split(T, num_cus, rows, blocks);
    return (int64_t)blocks * (8 * E + 12);
}

inline bool route_sizes_ok(int64_t T, int64_t E, int64_t k, int64_t ld, int x_type) {
    if (T < 0 || E < 1 || E > ROUTE_E_MAX || k < 1 || k > E || k > ROUTE_K_MAX) return false;
    if (T > SIZE_MAX_1 || T * k > SIZE_MAX_1 || !float_out(x_type)) return false;
    return ld >= E && ld <= LD_MAX && (T == 0 || extent_ok(1, T, ld, E));
}

inline bool route_tables_ok(const gemm_route_t *r, int64_t T) {
    if (!r || !r->counts || !r->offsets || !r->loss) return false;
    if (T > 0 && (!r->experts || !r->weights || !r->lse || !r->order || !r->place)) return false;
    const uintptr_t all = (uintptr_t)r->experts | (uintptr_t)r->weights | (uintptr_t)r->lse | (uintptr_t)r->counts |
                          (uintptr_t)r->offsets | (uintptr_t)r->order | (uintptr_t)r->place | (uintptr_t)r->loss;
    return all % 4 == 0;
}

inline int validate_route(gemm_handle_t h, const void *x, int x_type, int64_t T, int64_t E, int64_t ld, int64_t k,
                          unsigned flags, const gemm_route_t *r, const void *work) {
    if (!h || (flags & ~(unsigned)GEMM_ROUTE_NORMALIZE) || !route_sizes_ok(T, E, k, ld, x_type))
        return GEMM_ERR_INVALID_ARG;
    if (!route_tables_ok(r, T) || !work || (uintptr_t)work % 8) return GEMM_ERR_INVALID_ARG;
    if (T > 0 && (!x || (uintptr_t)x % (uintptr_t)out_bytes(x_type))) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

inline int validate_route_grad(gemm_handle_t h, const void *x, int x_type, int64_t T, int64_t E, int64_t ld, int64_t k,
                               unsigned flags, const gemm_route_t *r, const void *dw, const void *dx, int64_t ldd) {
    if (!h || (flags & ~(unsigned)GEMM_ROUTE_NORMALIZE) || !route_sizes_ok(T, E, k, ld, x_type))
        return GEMM_ERR_INVALID_ARG;
    if (ldd < E || ldd > LD_MAX || (T > 0 && !extent_ok(1, T, ldd, E))) return GEMM_ERR_INVALID_ARG;
    if (!route_tables_ok(r, T) || (uintptr_t)dw % 4) return GEMM_ERR_INVALID_ARG;
    const uintptr_t es = (uintptr_t)out_bytes(x_type);
    if (T > 0 && (!x || !dx || (uintptr_t)x % es || (uintptr_t)dx % es)) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

}  // namespace plan
}  // namespace dmp
