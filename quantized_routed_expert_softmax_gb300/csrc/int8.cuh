// int8.cuh -- the int8 matrix format with one scale a row (include/moe.h) as its kernels address it (sm_103a).
#pragma once

#include "common.cuh"

namespace moe {

// A matrix [rows, cols]: the fp32 scale of every row, rounded up to 16 bytes, then panels of 32 columns, each the 32
// codes of every row.
__host__ __device__ inline int64_t i8_scale_bytes(int64_t rows) { return (4 * rows + 15) / 16 * 16; }
__host__ __device__ inline int64_t i8_bytes(int64_t rows, int64_t cols) { return i8_scale_bytes(rows) + rows * cols; }

// max(z, 0), a NaN stays.  (As a choice by comparisons it becomes branches on the data.)
__device__ __forceinline__ float relu_nan(float z) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(z));
    return r;
}

// Four codes -> two pairs of f16, exactly: 0x64 in front of the byte c + 128 is the f16 value 1152 + c, and subtracting 1152
// leaves c; two values an instruction.
__device__ __forceinline__ void i8_f16(uint32_t w, uint32_t* h) {
    const uint32_t u = w ^ 0x80808080u, k1152 = 0x64806480u;
    asm("{\n\t.reg .b32 a, b;\n\tprmt.b32 a, %2, %4, 0x4140;\n\tprmt.b32 b, %2, %4, 0x4342;\n\t"
        "sub.rn.f16x2 %0, a, %3;\n\tsub.rn.f16x2 %1, b, %3;\n\t}"
        : "=r"(h[0]), "=r"(h[1])
        : "r"(u), "r"(k1152), "r"(0x64646464u));
}
// A sum of codes meets its two scales one after the other: their product alone may be too small or too large for fp32 where the
// result is not.  A sum is 0 or 1 to 2^30 in magnitude, so it loses nothing to a scale however small (whole numbers of a subnormal
// step), and a scale of up to kI8LargeScale takes it to 2^127 at most.  The channel's scale comes first, or, where it is larger,
// the row's: if that overflows, the result does.  (Scales are not negative.)
constexpr float kI8LargeScale = 0x1p97f;
__device__ __forceinline__ float i8_scaled(float z, float row, float channel) {
    return channel > kI8LargeScale ? z * row * channel : z * channel * row;
}
// SiLU to a few units in the last place at any gate: exp(-|g|) is at most 1, so that the divisor of the fast division lies
// in [1, 2], where it is good to 2 units.
__device__ __forceinline__ float silu_fast(float g) {
    const float e = expf(-fabsf(g));
    return __fdividef(g < 0.0f ? g * e : g, 1.0f + e);
}

// Whether a call's rows are few enough to stream the weights through mma.sync (stream.cu).  us, streamed / by CTA pairs:
//   int8 gate.up (2816 -> 2 x 704): 8 rows of 8 experts 9.3 / 14.9, 16 of 16 18 / 24, 24 of 24 32 / 25, 64 of 48 48 / 41
//   int8, one matrix (2816 -> 2 x 2112): 1 row 5.2 / 14.5, 8 rows 6.2 / 14.4, 16 rows 11.0 / 15.7, 24 rows 16.0 / 15.9
//   bf16 block (2816, 2112): 1 row 8.8 / 19.7, 16 rows 17.5 / 20.9, 24 rows 23.8 / 20.9; (2816, 704), 16 rows of 16 experts
//   33 / 46, 24 of 24 55 / 52
inline bool stream_rows(int64_t P) { return P <= 16; }

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
