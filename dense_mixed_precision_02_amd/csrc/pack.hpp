// pack.hpp -- a 16-bit matrix whose rows begin anywhere, copied to rows of whole 16-byte
// granules (zeros past a row's end).
//
// The products' kernels copy and transpose granules.  Reading such rows piece by piece inside a
// tile costs a multiple of what the copy does, which is a read and a write of the matrix (4096
// rows by 1500 x 1500, 8-bit gradients: 200 us without, 52 with the copy; adapters beside 4099 x
// 2051 x 2051, row-major: 210 us of product without, 91 and two copies of 4 to 9 with them).
#pragma once
#include "common.hpp"
#include "ragged.hpp"

namespace dmp {

struct PackArgs {
    const void *src;
    void *dst;
    int64_t rows, cols, ld;  // ld: the source's, in elements; the copy's is cols, rounded up to 8
};

// A granule to a thread.
static __global__ __launch_bounds__(256) void pack_rows(const PackArgs p) {
    const int64_t per = (p.cols + 7) / 8, i = (int64_t)workgroup_id() * 256 + threadIdx.x;
    const int64_t row = i / per, col = (i - row * per) * 8;
    if (row >= p.rows) return;
    const uint16_t *q = (const uint16_t *)p.src + row * p.ld + col;
    const int n = (int)min((int64_t)8, p.cols - col);
    intx4 v = {0, 0, 0, 0};
    if (n == 8) {
        __builtin_memcpy(&v, q, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) v[e / 2] |= (int)((uint32_t)q[e] << (e % 2 * 16));
    }
    *(intx4 *)((uint16_t *)p.dst + i * 8) = v;
}

}  // namespace dmp
