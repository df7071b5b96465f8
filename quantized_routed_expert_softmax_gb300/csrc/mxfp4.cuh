// mxfp4.cuh -- the MXFP4 matrix format (include/moe.h) as its kernels address it (sm_103a).
#pragma once

#include "common.cuh"

// The kernels of the MXFP4 operators and of the balance loss wait for the kernel before them (pdl_wait), and
// let the next one start as their CTAs end: allowed in earlier, its CTAs fill what room the SMs have left,
// unevenly, and a grid of one wave with equal shares then runs at the pace of the fullest SM (45056 x 2816 fp32,
// quantise and decode in turn: 205 us, 190 without).
namespace moe {

// A matrix [rows, cols]: codes row-major (cols / 2 bytes a row), then panels of 128 columns, each
// the 4 scale bytes (blocks 4q .. 4q+3) of every row.
__host__ __device__ inline int64_t mx_panels(int64_t cols) { return (cols + 127) / 128; }
__host__ __device__ inline int64_t mx_code_bytes(int64_t rows, int64_t cols) { return rows * (cols / 2); }
__host__ __device__ inline int64_t mx_bytes(int64_t rows, int64_t cols) {
    return (mx_code_bytes(rows, cols) + 4 * rows * mx_panels(cols) + 15) / 16 * 16;
}

constexpr uint32_t kMxScaleNaN = 255;   // a block that held a NaN or an infinity
constexpr uint32_t kMxScalePad = 127;   // 2^0: the blocks of the last panel past the end

// Scale byte -> 2^(b - 127), NaN for 255.  2^-127 is subnormal in fp32.
__device__ __forceinline__ float mx_scale(uint32_t b) {
    if (b == kMxScaleNaN) return __uint_as_float(0x7fffffffu);
    return __uint_as_float(b ? b << 23 : 0x00400000u);
}

// The sorted rows [first, last) of expert e.  Offsets are the caller's device data: whatever they
// hold, the range stays inside [0, P] (an expert whose range is reversed has no rows).
__device__ __forceinline__ void mx_expert_rows(const int32_t* offsets, int e, int P, int* first, int* last) {
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
