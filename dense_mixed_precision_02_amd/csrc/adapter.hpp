// adapter.hpp -- low-rank adapters of many requests beside a shared projection:
//
//   D[i] = alpha * (X[i] W + s_a (X[i] A_a) B_a) + beta * C[i]
//
// for the rows i of every request, a its adapter (or none).  X: M x K, W: K x N, A_a: K x r,
// B_a: r x N, with r of 8 to a few hundred.  Two launches:
//
//   hidden   H[i] = s_a (X[i] A_a): r columns over a long K, bound by reading X once (and,
//            with few rows, A_a).  A workgroup takes 16 or 64 rows of one request and up to 64
//            of the columns; its eight waves split K, each streams its part of X and A_a
//            straight into matrix-instruction operands, and their sums meet in LDS.
//   product  [X | H] [W; B_a]: the projection's K loop runs on, over r more for each request
//            that has rows in the tile, with the rows of H outside that request as zeros.  So
//            D is written once; adding H B_a in a pass of its own would read and write it again.
//
// H is rounded to the inputs' type, as an input of the matrix instructions; its error
// relative to H B_a is that of rounding X.  Where D has 32 bits H is kept as the sum of two
// such numbers (within 2^-16 of it for bf16, 2^-22 for fp16), each multiplied by B_a.
//
// A tile finds its requests by scanning the offsets (ragged.hpp's GroupWalk), 64 at a time.
//
// Zeros times an infinity or a NaN are no zeros: an adapter that holds one would spoil the
// other requests' rows of the tile.  So the parts of B_a that a tile uses are looked at on
// their way (a few instructions for each request), and a tile that found one is
// computed again, one request at a time.
#pragma once
#include "ragged_staged.hpp"

namespace dmp {

struct AdapterArgs {
    RaggedArgs r;            // A: X; B: W; groups, offsets: the requests
    const void *A, *B;       // the adapters'
    const int32_t *ids;      // adapter of each request, or NULL: its number
    const float *scale;      // of each adapter, or NULL: 1
    int64_t lda, ldb;        // leading dimensions of A_a, B_a
    int64_t sA, sB;          // elements from one adapter's to the next
    int adapters, rank;
    char *H;                 // parts x M x rp 16-bit values, zeros from rank to rp
    int rp, parts;
    void *hidden;            // M x rank, ld_hidden apart, or NULL: H for the caller
    int64_t ld_hidden;
    int tiles_r;             // hidden: column tiles of A_a
};

// Request g's adapter; -1: none.
__device__ static inline int adapter_of(const AdapterArgs &p, int g) {
    const int a = p.ids ? p.ids[g] : g;
    return (uint32_t)a < (uint32_t)p.adapters ? a : -1;
}

// Up to eight 16-bit values from e on, of which n exist (n <= 0: none is touched).
__device__ static inline intx4 load8(const uint16_t *e, int n) {
    intx4 v = {0, 0, 0, 0};
    if (n >= 8) {
        __builtin_memcpy(&v, e, 16);
    } else if (n > 0) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) v[i / 2] |= (int)((uint32_t)e[i] << (i % 2 * 16));
    }
    return v;
}

constexpr int HIDDEN_WAVES = 8;

// H of `rows` rows from row0 on (rows <= 16 TM), adapter a, columns c0 .. c0 + 16 TN - 1;
// A_a K-contiguous.
template <class DT, int TM, int TN, bool FAST>
__device__ static inline void hidden_sum(const AdapterArgs &p, int a, int64_t row0, int rows, int c0, float *lds) {
    constexpr int U = TM + TN <= 2 ? 4 : TM + TN <= 5 ? 2 : 1;  // k-tiles of 64 in a stage
    const int lane = lane_id(), wave = wave_id(), r16 = lane & 15, K = (int)p.r.K;
    const int nkt = (K + 63) / 64, per = (nkt + HIDDEN_WAVES - 1) / HIDDEN_WAVES;
    const int kt0 = min(wave * per, nkt), kt1 = min(kt0 + per, nkt);
    const int cols = p.rank - c0;
    const char *xb = (const char *)p.r.A + row0 * p.r.lda * 2, *ab = (const char *)p.A + (a * p.sA + c0 * p.lda) * 2;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(xb), ra = make_rsrc(ab);
    floatx4 acc[TM][TN] = {};
    intx4 fx[2][U][TM][2], fa[2][U][TN][2];
    auto one = [&](const __amdgpu_buffer_rsrc_t &rs, const char *base, int64_t ld, int row, bool there, int k) {
        if constexpr (FAST) {
            return __builtin_bit_cast(intx4, __builtin_amdgcn_raw_buffer_load_b128(
                                                 rs, there && k < K ? (row * (int)ld + k) * 2 : OOB_OFFSET, 0, 0));
        } else {
            return load8((const uint16_t *)base + row * ld + k, there ? K - k : 0);
        }
    };
    auto load = [&](int st, int kt) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (kt + u) * 64 + 32 * h + 8 * (lane >> 4);
                const bool in = kt + u < kt1;
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    fa[st][u][j][h] = one(ra, ab, p.lda, j * 16 + r16, in && j * 16 + r16 < cols, k);
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    fx[st][u][i][h] = one(rx, xb, p.r.lda, i * 16 + r16, in && i * 16 + r16 < rows, k);
            }
    };
    auto multiply = [&](int st) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[i][j] = mma16<DT>(fx[st][u][i][h], fa[st][u][j][h], acc[i][j]);
    };
    if (kt0 < kt1) {
        load(0, kt0);
        for (int kt = kt0; kt < kt1; kt += 2 * U) {
            load(1, kt + U);
            multiply(0);
            load(0, kt + 2 * U);
            multiply(1);
        }
    }
    constexpr int CW = 16 * TN, SZ = 16 * TM * CW;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                lds[wave * SZ + (i * 16 + 4 * (lane >> 4) + q) * CW + j * 16 + r16] = acc[i][j][q];
}

// The same with r-contiguous A_a, on 16 rows and 128 columns: as skinny_n (skinny.hpp),
// a lane turns 8 x 8 blocks in registers, and the t-th instruction computes the
// columns t, 8 + t, ..., 120 + t.
template <class DT, bool FAST>
__device__ static inline void hidden_sum_n(const AdapterArgs &p, int a, int64_t row0, int rows, int c0, float *lds) {
    const int lane = lane_id(), wave = wave_id(), r16 = lane & 15, K = (int)p.r.K;
    const int ns = (K + 31) / 32, per = (ns + HIDDEN_WAVES - 1) / HIDDEN_WAVES;
    const int s0 = min(wave * per, ns), s1 = min(s0 + per, ns);
    const int cols = p.rank - c0, k8 = 8 * (lane >> 4), c8 = 8 * r16;
    const uint16_t *ab = (const uint16_t *)p.A + a * p.sA + c0;
    const uint16_t *xr = (const uint16_t *)p.r.A + (row0 + r16) * p.r.lda;
    floatx4 acc[8] = {};
    for (int s = s0; s < s1; ++s) {
        const int k = s * 32 + k8;
        intx4 fb[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int n = k + r < K ? cols - c8 : 0;
            if constexpr (FAST) {
                // whole granules: the rank is a multiple of 8
                fb[r] = n > 0 ? *(const intx4 *)(ab + (int64_t)(k + r) * p.lda + c8) : intx4{0, 0, 0, 0};
            } else {
                fb[r] = load8(ab + (int64_t)(k + r) * p.lda + c8, n);
            }
        }
        const intx4 fx = load8(xr + k, r16 < rows ? K - k : 0);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            intx4 b;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                b[d] = (int)__builtin_amdgcn_perm((uint32_t)fb[2 * d + 1][t / 2], (uint32_t)fb[2 * d][t / 2],
                                                  t % 2 ? 0x07060302u : 0x05040100u);
            acc[t] = mma16<DT>(fx, b, acc[t]);
        }
    }
    constexpr int CW = 128, SZ = 16 * CW;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int t = 0; t < 8; ++t) lds[wave * SZ + (4 * (lane >> 4) + q) * CW + c8 + t] = acc[t][q];
}

// The waves' sums, added in their order, times the adapter's scale, rounded into H (and the
// caller's copy).
template <class DT, int CW, int SZ>
__device__ static inline void hidden_store(const AdapterArgs &p, int a, int64_t row0, int rows, int c0, const float *lds) {
    constexpr bool f16 = std::is_same_v<DT, F16>;
    __syncthreads();
    const float s = p.scale && a >= 0 ? p.scale[a] : 1.0f;
    const int cols = min(CW, p.rp - c0);
    for (int e = threadIdx.x; e < rows * CW; e += HIDDEN_WAVES * 64) {
        const int r = e / CW, c = e % CW;
        if (c >= cols) continue;
        float v = 0.0f;
        if (a >= 0 && c0 + c < p.rank) {
            v = lds[e];
            for (int w = 1; w < HIDDEN_WAVES; ++w) v += lds[w * SZ + e];
            v *= s;
        }
        const uint16_t hi = encode16(v, f16);
        const int64_t at = (row0 + r) * p.rp + c0 + c;
        ((uint16_t *)p.H)[at] = hi;
        if (p.parts > 1) {
            // (an infinity's rest would be no number)
            const float left = v - decode16(hi, f16);
            ((uint16_t *)p.H)[p.r.M * p.rp + at] = encode16(__builtin_isfinite(left) ? left : 0.0f, f16);
        }
        if (p.hidden && c0 + c < p.rank) ((uint16_t *)p.hidden)[(row0 + r) * p.ld_hidden + c0 + c] = hi;
    }
}

// H.  TM, TN: 16 TM rows by 16 TN columns to a workgroup (K-contiguous A_a); TN == 0:
// r-contiguous A_a, 16 rows by 128 columns.
template <class DT, int TM, int TN, bool FAST>
__global__ __launch_bounds__(HIDDEN_WAVES * 64, 2) void adapter_hidden(const AdapterArgs p) {
    constexpr int BM = 16 * TM, CW = TN ? 16 * TN : 128, SZ = BM * CW;
    __shared__ float lds[HIDDEN_WAVES * SZ];
    const int id = workgroup_id(), lane = lane_id(), total = (int)p.r.M;
    const int tile = id / p.tiles_r, c0 = (id - tile * p.tiles_r) * CW;
    GroupWalk<BM> walk;
    walk.load(p.r, total, lane);
    int g, r0, r1, tile0;
    if (!walk.find(p.r, total, lane, tile, g, r0, r1, tile0)) return;
    const int a = __builtin_amdgcn_readfirstlane(adapter_of(p, g));
    if (a < 0 && !p.hidden) return;
    const int64_t row0 = r0 + (int64_t)(tile - tile0) * BM;
    const int rows = (int)min((int64_t)BM, r1 - row0);
    if (a >= 0) {
        if constexpr (TN > 0) hidden_sum<DT, TM, TN, FAST>(p, a, row0, rows, c0, lds);
        else hidden_sum_n<DT, FAST>(p, a, row0, rows, c0, lds);
    }
    hidden_store<DT, CW, SZ>(p, a, row0, rows, c0, lds);
}

// A tile's requests that have an adapter: rows lo .. hi - 1 of the tile, in ascending order.
struct AdapterEntry {
    int rows;      // lo | hi << 16
    int adapter;
};

// By one wave; returns their number (at most BM: no two share a row).
template <int BM>
__device__ static inline int adapter_entries(const AdapterArgs &p, int row0, int rows, DMP_LDS AdapterEntry *list) {
    const int lane = lane_id(), total = (int)p.r.M;
    GroupWalk<BM> walk;
    walk.load(p.r, total, lane);
    int n = 0;
    do {
        const int lo = max(walk.lo, row0) - row0, hi = min(walk.hi, row0 + rows) - row0;
        int a = -1;
        if (lo < hi) a = adapter_of(p, walk.chunk + lane);  // (an empty request is none past the last)
        const uint64_t has = __ballot(a >= 0);
        if (a >= 0) {
            const int at = n + __popcll(has & ((1ull << lane) - 1));
            list[at].rows = lo | hi << 16;
            list[at].adapter = a;
        }
        n += __popcll(has);
    } while (__builtin_amdgcn_readlane(walk.hi, 63) < row0 + rows && walk.next(p.r, total, lane));
    return n;
}

// This workgroup's tile of the rows that the requests own; false: it has none.
template <int BM, int BN, class DT, bool BKC>
__device__ static inline bool adapter_tile_at(const AdapterArgs &p, TileAt &at) {
    const int total = (int)p.r.M;
    const int first = __builtin_amdgcn_readfirstlane(load_offset(p.r, 0, total));
    const int last = __builtin_amdgcn_readfirstlane(load_offset(p.r, p.r.groups, total));
    if (last <= first) return false;
    const int tiles_m = (last - first - 1) / BM + 1, id = workgroup_id();
    const int64_t tiles = (int64_t)tiles_m * p.r.tiles_n;
    if (id >= tiles) return false;
    int tm, tn;
    grouped_order(xcd_remap(id, (int)tiles), tiles_m, p.r.tiles_n, tm, tn);
    at.group = 0;
    at.row0 = first + (int64_t)tm * BM;
    at.rows = min(BM, last - (int)at.row0);
    at.col0 = (int64_t)tn * BN;
    at.cols = (int)p.r.N - tn * BN;
    at.k = (int)p.r.K;
    at.A = (const char *)p.r.A + at.row0 * p.r.lda * DT::ESZ;
    at.B = (const char *)p.r.B + (BKC ? at.col0 * p.r.ldb : at.col0) * DT::ESZ;
    return true;
}

// Does a granule hold an infinity or a NaN?
template <class DT>
__device__ static inline bool not_finite(const intx4 &v) {
    constexpr uint32_t E = std::is_same_v<DT, F16> ? 0x7c00u : 0x7f80u;
    bool bad = false;
#pragma unroll
    for (int w = 0; w < 4; ++w) bad |= ((uint32_t)v[w] & E) == E || ((uint32_t)v[w] & E << 16) == E << 16;
    return bad;
}

// The rows and entries of a pass over a tile: all of them first (pass < 0); where that found
// a B_a with an infinity or a NaN, one pass to each entry (odd passes) and to the rows before,
// between and behind them (even ones).
struct AdapterPass {
    int first, entries;  // entries of the list
    int lo, hi;          // rows of the tile that are stored
};
__device__ static inline AdapterPass adapter_pass(const DMP_LDS AdapterEntry *list, int entries, int rows, int pass) {
    if (pass < 0) return {0, entries, 0, rows};
    const int e = pass / 2;
    if (pass % 2) return {e, 1, list[e].rows & 0xffff, (int)((uint32_t)list[e].rows >> 16)};
    return {e, 0, e > 0 ? (int)((uint32_t)list[e - 1].rows >> 16) : 0, e < entries ? list[e].rows & 0xffff : rows};
}

// What a k-tile is read from.
struct AdapterSource {
    const char *A, *B;   // first element of the tile's rows and columns at the k-tile's first k
    int left;            // k that are left
    int lo, hi;          // rows of the tile that are not zeros
    bool more;           // past the projection's K: H and B_a
};

// K-tile kt of a tile: the projection's first, then for each request ceil(rank / 64) of its
// adapter, times parts.
template <class DT, bool BKC>
__device__ static inline AdapterSource adapter_source(const AdapterArgs &p, const TileAt &at, const DMP_LDS AdapterEntry *list,
                                                      int entries, int nkt, int kt) {
    AdapterSource s;
    s.more = kt >= nkt;
    if (!s.more) {
        s.A = at.A + (int64_t)kt * 128;
        s.B = at.B + (BKC ? (int64_t)kt * 128 : (int64_t)kt * 128 * p.r.ldb);
        s.left = at.k - kt * 64;
        s.lo = 0;
        s.hi = at.rows;
        return s;
    }
    const int nr = (p.rank + 63) / 64, e = (kt - nkt) / (nr * p.parts), j = (kt - nkt) - e * nr * p.parts;
    const int part = j / nr, k = 64 * (j - part * nr);
    const bool there = e < entries;
    const int rows = there ? list[e].rows : 0, a = there ? list[e].adapter : 0;
    s.lo = __builtin_amdgcn_readfirstlane(rows & 0xffff);
    s.hi = __builtin_amdgcn_readfirstlane((uint32_t)rows >> 16);
    s.left = there ? p.rank - k : 0;
    s.A = p.H + (part * p.r.M * p.rp + at.row0 * p.rp + k) * 2;
    const int64_t b = (int64_t)__builtin_amdgcn_readfirstlane(a) * p.sB;
    s.B = (const char *)p.B + (b + (BKC ? at.col0 * p.ldb + k : k * p.ldb + at.col0)) * 2;
    return s;
}

// The product, operands staged through registers as in ragged_staged.hpp.  FAST: all
// operands' 16-byte granules are aligned and whole.
template <class DT, int BM, int BN, int WM, int WN, bool BKC, bool FAST>
__global__ __launch_bounds__(WM *WN * 64, 2) void adapter_staged(const AdapterArgs p) {
    constexpr int NW = WM * WN, WTM = BM / WM, WTN = BN / WN, TM = WTM / 16, TN = WTN / 16;
    constexpr int DEPTH = 2;
    using OpA = Operand<DT, BM, NW, true>;
    using OpB = Operand<DT, BN, NW, BKC>;
    __shared__ __attribute__((aligned(1024))) char lds_a[2][OpA::BYTES];
    __shared__ __attribute__((aligned(1024))) char lds_b[2][OpB::BYTES];
    __shared__ AdapterEntry list[BM];
    __shared__ int count;
    const int lane = lane_id(), wave = wave_id();
    const int wm = wave / WN, wn = wave % WN;
    TileAt at;
    if (!adapter_tile_at<BM, BN, DT, BKC>(p, at)) return;
    if (wave == 0) {
        const int n = at.k > 0 ? adapter_entries<BM>(p, (int)at.row0, at.rows, (DMP_LDS AdapterEntry *)list) : 0;
        if (lane == 0) count = n;
    }
    __syncthreads();
    const int all = __builtin_amdgcn_readfirstlane(count), nkt0 = at.k / 64 + (at.k % 64 != 0);
    OpA opa, oph;
    OpB opb, opr;
    opa.init(wave, lane, p.r.lda, 0, BM);
    oph.init(wave, lane, p.rp, 0, BM);
    opb.init(wave, lane, p.r.ldb, 0, BN);
    opr.init(wave, lane, p.ldb, 0, BN);

    floatx4 acc[TM][TN];
    intx4 ra[DEPTH][OpA::CPW], rb[DEPTH][OpB::CPW];
    const DMP_LDS AdapterEntry *entry = (const DMP_LDS AdapterEntry *)list;
    int entries = all, nkt = 0;
    bool odd = false;
    auto fetch = [&](int kt, int slot) {
        const AdapterSource s = adapter_source<DT, BKC>(p, at, entry, entries, nkt0, kt);
        const __amdgpu_buffer_rsrc_t rsa = make_rsrc(s.A), rsb = make_rsrc(s.B);
        const int a0 = s.more ? oph.off0 : opa.off0, as = s.more ? oph.step : opa.step;
#pragma unroll
        for (int j = 0; j < OpA::CPW; ++j) {
            const int row = opa.row_or_k + 8 * NW * j;
            if (FAST || s.more) {  // (H is laid out in whole granules)
                const bool ok = row >= s.lo && row < s.hi && opa.fixed < s.left;
                ra[slot][j] = __builtin_bit_cast(
                    intx4, __builtin_amdgcn_raw_buffer_load_b128(rsa, ok ? a0 + j * as : OOB_OFFSET, 0, 0));
            } else {
                ra[slot][j] = load8((const uint16_t *)s.A + row * p.r.lda + opa.fixed, row < s.hi ? s.left - opa.fixed : 0);
            }
        }
        const int64_t ldb = s.more ? p.ldb : p.r.ldb;
        const int b0 = s.more ? opr.off0 : opb.off0, bs = s.more ? opr.step : opb.step;
#pragma unroll
        for (int j = 0; j < OpB::CPW; ++j) {
            const int r = BKC ? opb.row_or_k + 8 * NW * j : opb.fixed;
            const int k = BKC ? opb.fixed : opb.row_or_k + OpB::KSTEP * j;
            const bool ok = r < at.cols && k < s.left;
            if constexpr (FAST) {
                rb[slot][j] = __builtin_bit_cast(
                    intx4, __builtin_amdgcn_raw_buffer_load_b128(rsb, ok ? b0 + j * bs : OOB_OFFSET, 0, 0));
            } else {
                rb[slot][j] = load8((const uint16_t *)s.B + (BKC ? r * ldb + k : k * ldb + r),
                                    ok ? (BKC ? s.left - k : at.cols - r) : 0);
            }
        }
    };
    auto put = [&](int kt, int slot, int buf) {
        if (kt >= nkt0) {
#pragma unroll
            for (int j = 0; j < OpB::CPW; ++j) odd |= not_finite<DT>(rb[slot][j]);
        }
#pragma unroll
        for (int j = 0; j < OpA::CPW; ++j)
            *(DMP_LDS intx4 *)((DMP_LDS char *)lds_a[buf] + OpA::chunk_offset(j * NW + wave) + lane * 16) = ra[slot][j];
#pragma unroll
        for (int j = 0; j < OpB::CPW; ++j)
            *(DMP_LDS intx4 *)((DMP_LDS char *)lds_b[buf] + OpB::chunk_offset(j * NW + wave) + lane * 16) = rb[slot][j];
    };
    auto multiply = [&](int buf) {
        const DMP_LDS char *la = (const DMP_LDS char *)lds_a[buf], *lb = (const DMP_LDS char *)lds_b[buf];
        intx4 fa[2][TM], fb[2][TN];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[s][i] = frag16<DT, OpA, BM, true>(la, wm * WTM + i * 16, s, lane);
#pragma unroll
            for (int j = 0; j < TN; ++j) fb[s][j] = frag16<DT, OpB, BN, BKC>(lb, wn * WTN + j * 16, s, lane);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mma16<DT>(fa[s][i], fb[s][j], acc[i][j]);
    };
    constexpr int SLAB = 32 * (WTN + 4) * 4, INA = 2 * OpA::BYTES / SLAB;
    static_assert(NW <= INA || (NW - INA) * SLAB <= 2 * OpB::BYTES, "slabs must fit");
    DMP_LDS char *slab = wave < INA ? (DMP_LDS char *)&lds_a[0][0] + wave * SLAB
                                    : (DMP_LDS char *)&lds_b[0][0] + (wave - INA) * SLAB;
    const EpiParams &ep = p.r.ep;
    const int64_t first = at.row0 * p.r.ldc + at.col0;
    for (int pass = -1; pass <= 2 * all; ++pass) {
        const AdapterPass q = adapter_pass((const DMP_LDS AdapterEntry *)list, all, at.rows, pass);
        if (q.lo >= q.hi) continue;
        entry = (const DMP_LDS AdapterEntry *)list + q.first;
        entries = __builtin_amdgcn_readfirstlane(q.entries);
        nkt = nkt0 + entries * ((p.rank + 63) / 64) * p.parts;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = floatx4{0, 0, 0, 0};
        if (nkt > 0) {
#pragma unroll
            for (int s = 0; s < DEPTH; ++s) fetch(s, s);
            put(0, 0, 0);
            barrier_vmcnt<63>();
            bool done = nkt == 1;
            for (int kt = 0; !done; kt += DEPTH) {
#pragma unroll
                for (int s = 0; s < DEPTH; ++s) {
                    // k-tile kt + s is in LDS buffer s % 2, the next DEPTH - 1 are on their way
                    fetch(kt + s + DEPTH, s);
                    asm volatile("" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                    step_sync();
                    multiply(s % 2);
                    put(kt + s + 1, (s + 1) % DEPTH, (s + 1) % 2);
                    step_sync();
                    barrier_vmcnt<63>();
                    if (kt + s + 2 >= nkt) {
                        done = true;
                        break;
                    }
                }
            }
            multiply((nkt - 1) % 2);
        }
        if (pass < 0 && all > 0 && __syncthreads_or(odd)) continue;
        __syncthreads();
        store_wave_tile<WTM, WTN, true>((DMP_LDS float *)slab, ep, (const char *)p.r.C + first * out_size(ep.c_type),
                                        (char *)p.r.D + first * out_size(ep.d_type), p.r.ldc, q.hi, at.cols, wm * WTM,
                                        wn * WTN, lane, [&](int i, int j) { return acc[i][j]; }, q.lo);
        if (pass < 0) break;
        __syncthreads();
    }
}

}  // namespace dmp
