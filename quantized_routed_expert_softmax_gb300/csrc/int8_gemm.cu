// int8_gemm.cu -- the expert-indexed product of int8 rows with per-channel int8 weights:
//   z[r][n] = sx[r] sw[n] * sum_i qx[r][i] qw[n][i]
// with the sum of code products in integers, exact.
#include <algorithm>

#include "int8.cuh"

namespace moe {

// A thread has one result (SwiGLU: a gate and an up sum); a block 32 columns of 8 rows of one expert.
__global__ void __launch_bounds__(256) int8_product_kernel(const uint8_t* __restrict__ xq, int P, const uint8_t* __restrict__ wq,
                                                           int E, int N, int K, const int32_t* __restrict__ offsets, int act,
                                                           void* __restrict__ out, int ot) {
    pdl_wait();
    const int width = act == MOE_ACT_SWIGLU ? N / 2 : N;
    const float* sx = reinterpret_cast<const float*>(xq);
    for (int e = blockIdx.y; e < E; e += gridDim.y) {
        int first, last;
        expert_rows(offsets, e, P, &first, &last);
        const uint8_t* w = wq + e * i8_bytes(N, K);
        const float* sw = reinterpret_cast<const float*>(w);
        for (int n0 = blockIdx.x * 32; n0 < width; n0 += gridDim.x * 32) {
            const int n = n0 + (threadIdx.x & 31);
            if (n >= width) continue;
            for (int r = first + (threadIdx.x >> 5); r < last; r += 8) {
                int a = 0, b = 0;
                for (int p = 0; p < K / 32; ++p) {
                    const int* xp = reinterpret_cast<const int*>(xq + i8_scale_bytes(P) + (static_cast<int64_t>(p) * P + r) * 32);
                    const uint8_t* wp = w + i8_scale_bytes(N) + (static_cast<int64_t>(p) * N + n) * 32;
                    for (int i = 0; i < 8; ++i) {
                        a = __dp4a(xp[i], reinterpret_cast<const int*>(wp)[i], a);
                        if (act == MOE_ACT_SWIGLU) b = __dp4a(xp[i], reinterpret_cast<const int*>(wp + 32ll * width)[i], b);
                    }
                }
                float y = static_cast<float>(a) * (sx[r] * sw[n]);
                if (act == MOE_ACT_SWIGLU) y = silu(y) * (static_cast<float>(b) * (sx[r] * sw[width + n]));
                else if (act == MOE_ACT_RELU2) y = y > 0.0f ? y * y : (y <= 0.0f ? 0.0f : y);
                const int64_t o = static_cast<int64_t>(r) * width + n;
                if (ot == MOE_F32) static_cast<float*>(out)[o] = y;
                else static_cast<__nv_bfloat16*>(out)[o] = __float2bfloat16_rn(y);
            }
        }
    }
}

cudaError_t launch_int8_matmul(const void* xq, int64_t P, const void* wq, int64_t E, int64_t N, int64_t K, const int32_t* offsets,
                               int act, void* out, int ot, int32_t*, int, cudaStream_t s) {
    const int64_t width = act == MOE_ACT_SWIGLU ? N / 2 : N;
    return launch_pdl(int8_product_kernel, dim3(static_cast<unsigned>((width + 31) / 32), static_cast<unsigned>(E)), dim3(256), 0, s,
                      static_cast<const uint8_t*>(xq), static_cast<int>(P), static_cast<const uint8_t*>(wq), static_cast<int>(E),
                      static_cast<int>(N), static_cast<int>(K), offsets, act, out, ot);
}

}  // namespace moe
