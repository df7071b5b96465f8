// int8.cu -- rows coded in 8-bit integers with one fp32 scale each: the quantiser of expert inputs (and of weights with
// any number of rows), and its inverse.
//
// Per row: s = amax / 127, q = round-half-away(x / s), both divisions correctly rounded in fp32, as the per-channel
// weight packer has them.
#include <algorithm>

#include "int8.cuh"

namespace moe {

template <bool F32>
__global__ void __launch_bounds__(256) int8_quantize_kernel(const void* __restrict__ x, int64_t x_rows,
                                                            const int32_t* __restrict__ src_rows, int src_div, int64_t n_mat,
                                                            int64_t rows, int cols, uint8_t* __restrict__ dst) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < n_mat * rows; row += warps) {
        const int64_t m = row / rows, r = row - m * rows;
        int64_t sr = row;
        if (src_rows) {
            const int32_t i = __ldg(src_rows + r);
            sr = i < 0 || i / src_div >= x_rows ? -1 : i / src_div;
        }
        uint32_t amax = 0;   // as bits: non-negative floats order like their bit patterns, NaN above Inf
        if (sr >= 0)
            for (int c = lane; c < cols; c += 32)
                amax = max(amax, __float_as_uint(load_x(x, F32 ? MOE_F32 : MOE_BF16, sr * cols + c)) & 0x7fffffffu);
        amax = __reduce_max_sync(0xffffffffu, amax);
        const bool bad = amax >= 0x7f800000u;
        const float s = __fdiv_rn(__uint_as_float(amax), 127.0f);
        uint8_t* out = dst + m * i8_bytes(rows, cols);
        for (int c = lane; c < cols; c += 32) {
            int q = 0;
            if (!bad && s > 0.0f) {
                const float v = load_x(x, F32 ? MOE_F32 : MOE_BF16, sr * cols + c);
                q = static_cast<int>(fminf(fmaxf(roundf(__fdiv_rn(v, s)), -127.0f), 127.0f));
            }
            out[i8_scale_bytes(rows) + (static_cast<int64_t>(c >> 5) * rows + r) * 32 + (c & 31)] = static_cast<uint8_t>(q);
        }
        if (lane == 0) reinterpret_cast<float*>(out)[r] = bad ? __uint_as_float(0x7fffffffu) : s;
    }
}

template <bool F32>
__global__ void __launch_bounds__(256) int8_dequantize_kernel(const uint8_t* __restrict__ src, int64_t n_mat, int64_t rows,
                                                              int cols, void* __restrict__ out) {
    pdl_wait();
    const int64_t n = n_mat * rows * cols;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = i / cols, m = row / rows, r = row - m * rows;
        const int c = static_cast<int>(i - row * cols);
        const uint8_t* in = src + m * i8_bytes(rows, cols);
        const int8_t q = static_cast<int8_t>(in[i8_scale_bytes(rows) + (static_cast<int64_t>(c >> 5) * rows + r) * 32 + (c & 31)]);
        const float v = static_cast<float>(q) * reinterpret_cast<const float*>(in)[r];
        if (F32) static_cast<float*>(out)[i] = v;
        else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
    }
}

cudaError_t launch_int8_quantize(const void* x, int xt, int64_t x_rows, const int32_t* src_rows, int src_div, int64_t n_mat,
                                 int64_t rows, int64_t cols, void* dst, int num_sms, cudaStream_t s) {
    const int64_t ctas = std::min<int64_t>((n_mat * rows + 7) / 8, static_cast<int64_t>(num_sms) * 8);
    return launch_pdl(xt == MOE_F32 ? int8_quantize_kernel<true> : int8_quantize_kernel<false>, dim3(static_cast<unsigned>(ctas)),
                      dim3(256), 0, s, x, x_rows, src_rows, src_div, n_mat, rows, static_cast<int>(cols),
                      static_cast<uint8_t*>(dst));
}

cudaError_t launch_int8_dequantize(const void* src, int64_t n_mat, int64_t rows, int64_t cols, void* out, int ot, int num_sms,
                                   cudaStream_t s) {
    const int64_t ctas = std::min<int64_t>((n_mat * rows * cols + 255) / 256, static_cast<int64_t>(num_sms) * 8);
    return launch_pdl(ot == MOE_F32 ? int8_dequantize_kernel<true> : int8_dequantize_kernel<false>,
                      dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s, static_cast<const uint8_t*>(src), n_mat, rows,
                      static_cast<int>(cols), out);
}

}  // namespace moe
