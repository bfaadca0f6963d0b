// Host-side check of the grids of the grouped and 8-bit kernels
// (csrc/ragged_plan.hpp: grid_shape), built with the address and
// undefined-behaviour sanitizers by tests/test_ragged_grid.py: every workgroup
// that is asked for has one place, no axis passes what a launch takes with 512
// threads to a workgroup, and what is left over is less than a row.
// Exit status 0: all checks held.
#include <cstdint>
#include <cstdio>

#include "../../dense_mixed_precision_02_amd/csrc/ragged_plan.hpp"

using namespace dmp::plan;

static int failures = 0;
#define CHECK(cond)                                                        \
    do {                                                                   \
        if (!(cond)) {                                                     \
            std::fprintf(stderr, "FAILED line %d: %s\n", __LINE__, #cond); \
            ++failures;                                                    \
        }                                                                  \
    } while (0)

int main() {
    const int64_t row = 1ll << GRID_ROW_BITS;
    for (int64_t n : {(int64_t)1, (int64_t)7, row - 1, row, row + 1, 2 * row, (int64_t)1 << 23, ((int64_t)1 << 24) - 1,
                      (int64_t)1 << 24, ((int64_t)1 << 24) + 1, (int64_t)17 << 20, (int64_t)1 << 30, (int64_t)0x7fffffff}) {
        GridShape g{};
        CHECK(grid_shape(n, g));
        const int64_t all = (int64_t)g.x * g.y;
        CHECK(all >= n && all - n < row);
        CHECK((int64_t)g.x * 512 < (1ll << 32) && g.y <= 65535);
        CHECK(g.y == 1 || g.x == (uint64_t)row);  // the number is y * 2^22 + x
        CHECK(all - 1 <= 0x7fffffff);             // and fits an int, past the count too
        CHECK(row % 8 == 0);                      // consecutive numbers go round the XCDs
    }
    GridShape g{};
    CHECK(!grid_shape(0, g) && !grid_shape(-1, g) && !grid_shape(1ll << 31, g) && !grid_shape(INT64_MAX, g));
    std::printf("%d failures\n", failures);
    return failures != 0;
}
