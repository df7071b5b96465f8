// grid.cuh -- grids over more blocks of tokens than one dimension holds.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// A grid of x by n blocks of tokens, n up to 2^20: dimension y ends at 65535, the rest goes to z.  Blocks past n
// are the kernel's to leave out.
constexpr int64_t kMaxGridY = 65535;
inline dim3 token_grid(int64_t x, int64_t n) {
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>(n < kMaxGridY ? n : kMaxGridY),
                static_cast<unsigned>((n + kMaxGridY - 1) / kMaxGridY));
}
__device__ __forceinline__ int token_block() { return static_cast<int>(blockIdx.z * gridDim.y + blockIdx.y); }

}  // namespace moe
