// int8.cuh -- the int8 matrix format with one scale a row (include/moe.h) as its kernels address it (sm_103a).
#pragma once

#include "common.cuh"

namespace moe {

// A matrix [rows, cols]: the fp32 scale of every row, rounded up to 16 bytes, then panels of 32 columns, each the 32
// codes of every row.
__host__ __device__ inline int64_t i8_scale_bytes(int64_t rows) { return (4 * rows + 15) / 16 * 16; }
__host__ __device__ inline int64_t i8_bytes(int64_t rows, int64_t cols) { return i8_scale_bytes(rows) + rows * cols; }

// The sorted rows [first, last) of expert e.  Offsets are the caller's device data: whatever they hold, the range stays
// inside [0, P] (an expert whose range is reversed has no rows).
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int P, int* first, int* last) {
    if (!offsets) {   // one matrix, every row
        *first = 0;
        *last = P;
        return;
    }
    const int a = min(max(__ldg(offsets + e), 0), P), b = min(max(__ldg(offsets + e + 1), 0), P);
    *first = a;
    *last = max(a, b);
}

}  // namespace moe
