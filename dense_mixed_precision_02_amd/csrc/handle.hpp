// handle.hpp -- what a gemm_handle_t points to (host code only).
#pragma once
#include <stddef.h>

struct gemm_handle {
    int device = 0;
    int num_cus = 0;
    void *ws = nullptr;   // split-K partials or the transposed int8 B, grown on demand
    size_t ws_bytes = 0;
};
