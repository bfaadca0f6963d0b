// ragged_api.hip -- the entry points of the products over ragged groups, the
// 8-bit quantization and the 8-bit block-scaled products (declared in
// include/dmp_gemm.h): argument checks, kernel choice and launches.
#include <hip/hip_runtime.h>

#include "../../include/dmp_gemm.h"
#include "handle.hpp"
#include "quant8.hpp"
#include "ragged.hpp"
#include "ragged_plan.hpp"
#include "ragged_staged.hpp"
#include "ragged_tile.hpp"
#include "scaled_tile.hpp"
#include "skinny.hpp"

using namespace dmp;
using namespace dmp::plan;

namespace {

EpiParams out_stage(float alpha, float beta, int c_type, int d_type) {
    EpiParams ep;
    ep.alpha = alpha;
    ep.beta = beta;
    ep.c_type = c_type;
    ep.d_type = d_type;
    ep.use_c = beta != 0.0f;
    return ep;
}

template <class Args>
int launch(void (*kernel)(Args), int64_t workgroups, int threads, hipStream_t s, const Args &a) {
    GridShape g;
    if (!grid_shape(workgroups, g)) return GEMM_ERR_INVALID_ARG;  // beyond one launch's grid
    hipLaunchKernelGGL(kernel, dim3(g.x, g.y), dim3((unsigned)threads), 0, s, a);
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

// One workgroup to each tile there can be.  ROWS, SCALED: row tiles, at most one
// more for each group than the rows fill.  WGRAD: runs of tiles (my_tile), the
// tiles that an XCD works on at a time, but few enough that every XCD gets some.
int64_t tile_grid(gemm_handle_t h, RaggedArgs &a, int mode, int bm, int bn, int per_cu) {
    a.tiles_n = (int)cdiv(a.N, bn);
    if (mode != RAGGED_WGRAD) return (cdiv(a.M, bm) + a.groups) * a.tiles_n;
    a.tiles_m = (int)cdiv(a.M, bm);
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
    a.run = (int)std::max<int64_t>(1, std::min<int64_t>(h->num_cus / 8 * per_cu, cdiv(a.groups * tiles, 8)));
    return cdiv(a.groups * cdiv(tiles, a.run), 8) * 8 * a.run;
}

template <class DT, bool AK, bool BKC, int MODE>
int launch_tile(gemm_handle_t h, RaggedArgs a, hipStream_t s) {
    a.cut = h->num_cus;  // 256 x 256 tiles: one workgroup to a CU
    const int64_t grid = tile_grid(h, a, MODE, 256, 256, 1) + (MODE == RAGGED_ROWS ? 2 * a.cut : 0);
    return launch(ragged_tile<DT, 256, 256, AK, BKC, MODE>, grid, 256, s, a);
}

template <class DT, int BM, int BN, int WM, int WN, bool AK, bool BKC, int MODE, bool FAST>
int launch_staged(gemm_handle_t h, RaggedArgs a, hipStream_t s) {
    const int64_t grid = tile_grid(h, a, MODE, BM, BN, 8 / (WM * WN));
    return launch(ragged_staged<DT, BM, BN, WM, WN, AK, BKC, MODE, FAST>, grid, WM * WN * 64, s, a);
}

// 16-bit operands: FA, FB unused.
template <class DT, int MODE, int TN, int NW, int FA, int FB>
int launch_skinny(RaggedArgs a, hipStream_t s) {
    a.tiles_n = (int)cdiv(a.N, 16 * TN);
    return launch(skinny<DT, MODE, TN, NW, FA, FB>, (int64_t)a.groups * a.tiles_n, NW * 64, s, a);
}

// N-contiguous B, 16-bit operands.
template <class DT, int NW>
int launch_skinny_n(RaggedArgs a, hipStream_t s) {
    a.tiles_n = (int)cdiv(a.N, 128);
    return launch(skinny_n<DT, NW>, (int64_t)a.groups * a.tiles_n, NW * 64, s, a);
}

template <class DT, bool AK, bool BKC, int MODE>
int launch_cfg(gemm_handle_t h, int cfg, const RaggedArgs &a, hipStream_t s) {
    if (cfg == CFG_L) return launch_tile<DT, AK, BKC, MODE>(h, a, s);
    if constexpr (MODE == RAGGED_ROWS) {
        if (cfg == CFG_M) return launch_staged<DT, 128, 128, 2, 2, AK, BKC, MODE, true>(h, a, s);
    } else {
        if (cfg == CFG_S) return launch_staged<DT, 64, 128, 1, 4, AK, BKC, MODE, true>(h, a, s);
    }
    if constexpr (MODE == RAGGED_ROWS && BKC) {
        if (cfg == CFG_SKINNY1) return launch_skinny<DT, MODE, 1, 4, 0, 0>(a, s);
        if (cfg == CFG_SKINNY2) return launch_skinny<DT, MODE, 2, 4, 0, 0>(a, s);
    }
    if constexpr (MODE == RAGGED_ROWS && !BKC) {
        if (cfg == CFG_SKINNY_N) return launch_skinny_n<DT, 4>(a, s);
    }
    return launch_staged<DT, 64, 128, 1, 4, AK, BKC, MODE, false>(h, a, s);
}

template <int FA, int FB, int BM, int BN, int WM, int WN, bool EXACT>
int launch_scaled_tile(gemm_handle_t h, RaggedArgs a, hipStream_t s) {
    const int64_t grid = tile_grid(h, a, RAGGED_SCALED, BM, BN, 1);
    return launch(scaled_tile<FA, FB, BM, BN, WM, WN, EXACT>, grid, WM * WN * 64, s, a);
}

template <int FA, int FB>
int launch_scaled(gemm_handle_t h, int cfg, const RaggedArgs &a, hipStream_t s) {
    if (cfg == CFG_SKINNY1) return launch_skinny<F8<FA, FB>, RAGGED_SCALED, 1, 4, FA, FB>(a, s);
    if (cfg == CFG_SKINNY2) return launch_skinny<F8<FA, FB>, RAGGED_SCALED, 2, 4, FA, FB>(a, s);
    if (cfg == CFG_SKINNY4) return launch_skinny<F8<FA, FB>, RAGGED_SCALED, 4, 4, FA, FB>(a, s);
    const bool exact = a.ep.d_type == OUT_F32;
    if (cfg == CFG_L)
        return exact ? launch_scaled_tile<FA, FB, 256, 128, 4, 2, true>(h, a, s)
                     : launch_scaled_tile<FA, FB, 256, 256, 2, 4, false>(h, a, s);
    return exact ? launch_scaled_tile<FA, FB, 128, 128, 2, 2, true>(h, a, s)
                 : launch_scaled_tile<FA, FB, 128, 128, 2, 2, false>(h, a, s);
}

template <int XT, int FMT>
int launch_quant8(const Quant8Args &a, bool col, int block, int64_t grid, hipStream_t s) {
    if (!col && block == 1) return launch(quant8_rows<XT, FMT>, grid, 256, s, a);
    if (!col) return launch(quant8_tile<XT, FMT, false, true>, grid, 256, s, a);
    if (block == 1) return launch(quant8_tile<XT, FMT, true, false>, grid, 256, s, a);
    return launch(quant8_tile<XT, FMT, true, true>, grid, 256, s, a);
}

}  // namespace

extern "C" {

int gemm_run_grouped(gemm_handle_t h, const void *A, const void *B, const void *C, void *D,
                     const void *offsets, int64_t groups, int64_t M, int64_t N, int64_t K, int64_t lda,
                     int64_t ldb, int64_t ldc, int dtype, unsigned flags, float alpha, float beta,
                     int c_type, int d_type, void *stream) {
    const EpiParams ep = out_stage(alpha, beta, c_type, d_type);
    const int rc = validate_grouped(h, A, B, C, D, offsets, groups, M, N, K, lda, ldb, ldc, dtype, flags, ep);
    if (rc != GEMM_OK || M == 0 || N == 0 || groups == 0) return rc;
    const bool bc = flags & GEMM_B_COLMAJOR;
    RaggedArgs a{};
    a.A = A; a.B = B; a.C = C; a.D = D; a.offsets = offsets;
    a.M = M; a.N = N; a.K = K; a.lda = lda; a.ldb = ldb; a.ldc = ldc;
    a.sB = K == 0 ? 0 : (bc ? N : K) * ldb;
    a.groups = (int)groups;
    a.off32 = (flags & GEMM_OFFSETS_I32) != 0;
    a.ep = ep;
    hipStream_t s = (hipStream_t)stream;
    const int cfg = grouped_cfg(h->num_cus, A, B, groups, M, N, K, lda, ldb, bc);
    if (dtype == GEMM_F16)
        return bc ? launch_cfg<F16, true, true, RAGGED_ROWS>(h, cfg, a, s)
                  : launch_cfg<F16, true, false, RAGGED_ROWS>(h, cfg, a, s);
    return bc ? launch_cfg<BF16, true, true, RAGGED_ROWS>(h, cfg, a, s)
              : launch_cfg<BF16, true, false, RAGGED_ROWS>(h, cfg, a, s);
}

int gemm_run_grouped_wgrad(gemm_handle_t h, const void *X, const void *Y, const void *C, void *D,
                           const void *offsets, int64_t groups, int64_t M, int64_t N, int64_t K,
                           int64_t ldx, int64_t ldy, int64_t ldc, int dtype, unsigned flags, float alpha,
                           float beta, int c_type, int d_type, void *stream) {
    const EpiParams ep = out_stage(alpha, beta, c_type, d_type);
    const int rc = validate_wgrad(h, X, Y, C, D, offsets, groups, M, N, K, ldx, ldy, ldc, dtype, flags, ep);
    if (rc != GEMM_OK || M == 0 || N == 0 || groups == 0) return rc;
    RaggedArgs a{};
    a.A = X; a.B = Y; a.C = C; a.D = D; a.offsets = offsets;
    a.M = M; a.N = N; a.K = K; a.lda = ldx; a.ldb = ldy; a.ldc = ldc;
    a.sC = M * ldc;
    a.groups = (int)groups;
    a.off32 = (flags & GEMM_OFFSETS_I32) != 0;
    a.ep = ep;
    hipStream_t s = (hipStream_t)stream;
    const int cfg = wgrad_cfg(h->num_cus, X, Y, groups, M, N, K, ldx, ldy);
    return dtype == GEMM_F16 ? launch_cfg<F16, false, false, RAGGED_WGRAD>(h, cfg, a, s)
                             : launch_cfg<BF16, false, false, RAGGED_WGRAD>(h, cfg, a, s);
}

int gemm_quant8(gemm_handle_t h, const void *X, int64_t M, int64_t K, int64_t ldx, int x_type,
                unsigned flags, int64_t batch, int block, int q_type, void *Q, float *scale, void *stream) {
    const int rc = validate_quant8(h, X, M, K, ldx, x_type, flags, batch, block, q_type, Q, scale);
    if (rc != GEMM_OK || M == 0 || K == 0 || batch == 0) return rc;
    const bool col = flags & GEMM_A_COLMAJOR;
    Quant8Args a{};
    a.X = X; a.Q = (uint8_t *)Q; a.scale = scale;
    a.M = M; a.K = K; a.ldx = ldx; a.Kp = k16(K); a.sX = (col ? K : M) * ldx;
    a.KB = (int)cdiv(K, 128);
    a.MB = cdiv(M, block);
    const bool rows = !col && block == 1;
    a.tiles_m = cdiv(M, rows ? QUANT_ROWS : 128);
    a.batch = (int)batch;
    const __int128 g = (__int128)batch * a.tiles_m * (rows ? cdiv(a.KB, 8) : a.KB);
    if (g > 0x7fffffff) return GEMM_ERR_INVALID_ARG;
    const int64_t grid = (int64_t)g;
    hipStream_t s = (hipStream_t)stream;
    const bool e4 = q_type == GEMM_E4M3;
    if (x_type == GEMM_OUT_F32)
        return e4 ? launch_quant8<OUT_F32, 0>(a, col, block, grid, s) : launch_quant8<OUT_F32, 1>(a, col, block, grid, s);
    if (x_type == GEMM_OUT_F16)
        return e4 ? launch_quant8<OUT_F16, 0>(a, col, block, grid, s) : launch_quant8<OUT_F16, 1>(a, col, block, grid, s);
    return e4 ? launch_quant8<OUT_BF16, 0>(a, col, block, grid, s) : launch_quant8<OUT_BF16, 1>(a, col, block, grid, s);
}

int gemm_run_scaled8(gemm_handle_t h, const gemm_q8_t *A, const gemm_q8_t *B, const void *C, void *D,
                     const void *offsets, int64_t groups, int64_t M, int64_t N, int64_t K, int64_t ldc,
                     unsigned flags, float alpha, float beta, int c_type, int d_type, void *stream) {
    const EpiParams ep = out_stage(alpha, beta, c_type, d_type);
    const int rc = validate_scaled8(h, A, B, C, D, offsets, groups, M, N, K, ldc, flags, ep);
    if (rc != GEMM_OK || M == 0 || N == 0 || groups == 0) return rc;
    RaggedArgs a{};
    a.A = A->q; a.B = B->q; a.C = C; a.D = D; a.offsets = offsets;
    a.sa = A->scale; a.sb = B->scale;
    a.M = M; a.N = N; a.K = k16(K);
    a.lda = A->ld; a.ldb = B->ld; a.ldc = ldc;
    a.sB = groups > 1 ? B->group : 0;
    a.sa_row = A->scale_row; a.sa_k = A->scale_k;
    a.sb_col = B->scale_row; a.sb_k = B->scale_k; a.sb_group = groups > 1 ? B->scale_group : 0;
    a.groups = (int)groups;
    a.off32 = (flags & GEMM_OFFSETS_I32) != 0;
    a.ep = ep;
    hipStream_t s = (hipStream_t)stream;
    const int cfg = scaled_cfg(h->num_cus, groups, M, N);
    const bool a4 = A->type == GEMM_E4M3, b4 = B->type == GEMM_E4M3;
    if (a4) return b4 ? launch_scaled<0, 0>(h, cfg, a, s) : launch_scaled<0, 1>(h, cfg, a, s);
    return b4 ? launch_scaled<1, 0>(h, cfg, a, s) : launch_scaled<1, 1>(h, cfg, a, s);
}

}  // extern "C"
