// wgrad8_api.hip -- the entry point of the weight gradients from 8-bit checkpoints
// (declared in include/dmp_gemm.h): argument checks, kernel choice and launches.
#include <hip/hip_runtime.h>

#include "../../include/dmp_gemm.h"
#include "handle.hpp"
#include "pack.hpp"
#include "wgrad8.hpp"
#include "wgrad8_plan.hpp"

using namespace dmp;
using namespace dmp::plan;

namespace {

template <class Args>
int launch(void (*kernel)(Args), int64_t workgroups, int threads, hipStream_t s, const Args &a) {
    GridShape g;
    if (!grid_shape(workgroups, g)) return GEMM_ERR_INVALID_ARG;  // beyond one launch's grid
    hipLaunchKernelGGL(kernel, dim3(g.x, g.y), dim3((unsigned)threads), 0, s, a);
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

// per_cu: workgroups that a CU holds
int launch_tile(gemm_handle_t h, void (*kernel)(Wgrad8Args), int BM, int BN, int threads, int per_cu, Wgrad8Args a, hipStream_t s) {
    RaggedArgs &r = a.r;
    r.tiles_m = (int)cdiv(r.M, BM);
    r.tiles_n = (int)cdiv(r.N, BN);
    const int64_t tiles = (int64_t)r.tiles_m * r.tiles_n;
    // runs of tiles on an XCD: as many as it works on at a time, but every XCD gets some
    r.run = (int)std::max<int64_t>(1, std::min<int64_t>(h->num_cus / 8 * per_cu, cdiv(r.groups * tiles, 8)));
    const int64_t units = cdiv(r.groups * cdiv(tiles, r.run), 8) * 8 * r.run;
    if (units > 0x7fffffff) return GEMM_ERR_INVALID_ARG;
    a.units = (int)units;
    return launch(kernel, units * a.splits, threads, s, a);
}

template <class DT, int FMT>
int launch_wgrad8(gemm_handle_t h, int edge, const Wgrad8Args &a, hipStream_t s) {
    if (edge == 256) return launch_tile(h, wgrad8_large_tile<DT, FMT>, 256, 256, 256, 1, a, s);
    if (edge == 128) return launch_tile(h, wgrad8_tile<DT, FMT, 128, 128, 2, 2>, 128, 128, 256, 2, a, s);
    return launch_tile(h, wgrad8_tile<DT, FMT, 64, 128, 2, 2>, 64, 128, 256, 2, a, s);
}

}  // namespace

extern "C" {

int64_t gemm_wgrad8_work(gemm_handle_t h, const void *Y, int64_t groups, int64_t M, int64_t N, int64_t K, int64_t ldy) {
    if (!h || !wgrad8_sizes_ok(groups, M, N, K) || (K > 0 && N > WGRAD8_LD_MAX)) return -1;
    if (groups > 0 && M > 0 && N > 0 && !extent_ok(groups, M, N, N)) return -1;
    return wgrad8_work(h->num_cus, Y, groups, M, N, K, ldy);
}

int gemm_run_wgrad8(gemm_handle_t h, const gemm_q8_t *X, const void *Y, const void *C, void *D, const void *offsets,
                    int64_t groups, int64_t M, int64_t N, int64_t K, int64_t ldy, int64_t ldc, int dtype, unsigned flags,
                    float alpha, float beta, int c_type, int d_type, void *work, void *stream) {
    EpiParams ep;
    ep.alpha = alpha; ep.beta = beta;
    ep.c_type = c_type; ep.d_type = d_type;
    ep.use_c = beta != 0.0f;
    const int rc = validate_wgrad8(h, X, Y, C, D, offsets, groups, M, N, K, ldy, ldc, dtype, flags, ep);
    if (rc != GEMM_OK || M == 0 || N == 0 || groups == 0) return rc;
    Wgrad8Args a{};
    Wgrad8Plan plan = wgrad8_plan(h->num_cus, groups, M, N, K);
    if (plan.edge == 256 && !wgrad8_narrow(*X)) plan.edge = 128;
    a.splits = plan.splits;
    const int64_t pack = wgrad8_pack(Y, N, K, ldy);
    if ((a.splits > 1 || pack > 0) && (!work || !aligned16(work))) return GEMM_ERR_INVALID_ARG;
    char *const part = (char *)work + pack;
    hipStream_t s = (hipStream_t)stream;
    RaggedArgs &r = a.r;
    r.A = X->q; r.sa = X->scale; r.sa_row = X->scale_row; r.sa_k = X->scale_k; r.lda = X->ld;
    r.B = Y; r.ldb = ldy; r.offsets = offsets;
    if (pack > 0) {
        PackArgs q{};
        q.src = Y; q.dst = work; q.rows = K; q.cols = N; q.ld = ldy;
        const int st = launch(pack_rows, cdiv(K * cdiv(N, 8), 256), 256, s, q);
        if (st != GEMM_OK) return st;
        r.B = work; r.ldb = cdiv(N, 8) * 8;
    }
    r.M = M; r.N = N; r.K = K;
    r.groups = (int)groups;
    r.off32 = (flags & GEMM_OFFSETS_I32) != 0;
    r.C = C; r.D = D; r.ldc = ldc; r.sC = M * ldc; r.ep = ep;
    if (a.splits > 1) {
        r.D = part; r.ldc = N; r.sC = M * N;
        r.ep.alpha = 1.0f; r.ep.use_c = 0; r.ep.d_type = OUT_F32;
        a.part = groups * M * N;
    }
    const bool e4 = X->type == GEMM_E4M3;
    int st;
    if (dtype == GEMM_F16) st = e4 ? launch_wgrad8<F16, 0>(h, plan.edge, a, s) : launch_wgrad8<F16, 1>(h, plan.edge, a, s);
    else st = e4 ? launch_wgrad8<BF16, 0>(h, plan.edge, a, s) : launch_wgrad8<BF16, 1>(h, plan.edge, a, s);
    if (st != GEMM_OK || a.splits == 1) return st;
    Wgrad8JoinArgs j{};
    j.part = (const float *)part; j.C = C; j.D = D;
    j.rows = groups * M; j.N = N; j.ldc = ldc; j.splits = a.splits; j.ep = ep;
    return launch(wgrad8_join, cdiv(j.rows * cdiv(N, 4), 256), 256, s, j);
}

}  // extern "C"
