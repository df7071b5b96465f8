// mxfp4.cu -- MXFP4 (OCP microscaling: E2M1 codes, one E8M0 scale per 32 consecutive values of a
// row): the quantiser of weights and expert inputs, and its inverse.
//
// Per block of 32: X = max(floor(log2 amax) - 2, -127), scale byte X + 127, codes E2M1(x * 2^-X)
// rounded to nearest even and saturated at 6 (2 is E2M1's largest exponent, so amax lands in
// [4, 8)).  Every step is exact up to the one rounding into the code: the exponent is read off the
// fp32 bits and 2^-X is a power of two in fp32's normal range (-X is in [-125, 127]).
#include <algorithm>

#include "mxfp4.cuh"

namespace moe {

// Eight values -> eight E2M1 codes, the first in the low nibble; a zero magnitude is coded +0.
__device__ __forceinline__ uint32_t e2m1x8(const float v[8], float mul) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t b;
        asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
            : "=r"(b)
            : "f"(v[2 * i + 1] * mul), "f"(v[2 * i] * mul));
        w |= b << (8 * i);
    }
    const uint32_t mag = w & 0x77777777u;
    return mag | (w & (mag + 0x77777777u) & 0x88888888u);   // the sign of a nibble with a magnitude
}

__device__ __forceinline__ void load8(const void* x, int xt, int64_t off, float v[8]) {
    if (xt == MOE_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + off);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + off));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

// 16 lanes per (row, panel of 128 columns): a lane codes 8 consecutive values, four lanes share a
// block, and the first lane of the 16 writes the panel's scale word.  grid-stride over the items.
__global__ void __launch_bounds__(256) mxfp4_quantize_kernel(const void* __restrict__ x, int xt, int64_t x_rows,
                                                              const int32_t* __restrict__ src_rows, int src_div,
                                                              int64_t items, int64_t rows, int64_t cols,
                                                              uint8_t* __restrict__ dst) {
    pdl_wait();
    pdl_trigger();
    const int64_t npan = mx_panels(cols), mat = mx_bytes(rows, cols), code_bytes = mx_code_bytes(rows, cols);
    const int lane16 = threadIdx.x & 15;
    const int64_t step = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 4;
    // (items is even or the last pair's second item repeats nothing: a warp's two halves may differ
    // in whether they have an item, so every lane stays in the loop while its warp's first half does)
    const int64_t it0 = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 4;
    for (int64_t it = it0; (it & ~int64_t(1)) < items; it += step) {
        const bool live = it < items;
        const int64_t rr = live ? it / npan : 0, q = live ? it - rr * npan : 0;   // matrix * rows + row, panel
        const int64_t m = rr / rows, r = rr - m * rows;
        const int64_t c = q * 128 + lane16 * 8;
        const bool in = live && c < cols;
        int64_t sr = rr;
        if (src_rows) {
            const int32_t s = live ? __ldg(src_rows + r) : -1;
            sr = s < 0 ? -1 : s / src_div;
        }
        float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (in && sr >= 0 && (!src_rows || sr < x_rows)) load8(x, xt, sr * cols + c, v);
        uint32_t amax = 0;   // as bits: non-negative floats order like their bit patterns, NaN above Inf
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const bool bad = amax >= 0x7f800000u;
        const int e = max(static_cast<int>(amax >> 23) - 2, 0);   // X + 127
        const uint32_t codes = bad ? 0u : e2m1x8(v, __uint_as_float(static_cast<uint32_t>(254 - e) << 23));
        uint32_t sb = bad ? kMxScaleNaN : static_cast<uint32_t>(e);
        if (!in) sb = kMxScalePad;
        uint32_t word = sb << (8 * (lane16 >> 2));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        uint8_t* out = dst + m * mat;
        if (in) *reinterpret_cast<uint32_t*>(out + r * (cols / 2) + c / 2) = codes;
        if (live && lane16 == 0) *reinterpret_cast<uint32_t*>(out + code_bytes + 4 * (q * rows + r)) = word;
    }
}

// One thread per 8 values.
__global__ void __launch_bounds__(256) mxfp4_dequantize_kernel(const uint8_t* __restrict__ src, int64_t items,
                                                                int64_t rows, int64_t cols, void* __restrict__ out,
                                                                int ot) {
    pdl_wait();
    pdl_trigger();
    const int64_t code_bytes = mx_code_bytes(rows, cols), mat = mx_bytes(rows, cols), per_row = cols / 8;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; it < items;
         it += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t rr = it / per_row, c = it - rr * per_row;
        const int64_t m = rr / rows, r = rr - m * rows;
        const uint8_t* p = src + m * mat;
        const uint32_t codes = __ldg(reinterpret_cast<const uint32_t*>(p + r * (cols / 2)) + c);
        const int64_t b = c / 4;   // block along the row
        const float s = mx_scale(__ldg(p + code_bytes + 4 * ((b / 4) * rows + r) + b % 4));
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = e2m1x2_to_f32x2((codes >> (8 * i)) & 0xffu);
            v[2 * i] = f.x * s;
            v[2 * i + 1] = f.y * s;
        }
        if (ot == MOE_F32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + 8 * it);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {   // exact: a code has 2 significant bits, and bf16 has fp32's exponents
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            reinterpret_cast<uint4*>(out)[it] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ------------------------------------------------------------------------------- launchers
namespace {
unsigned grid_for(int64_t threads, int num_sms) {   // CTAs of 256, grid-stride beyond 8 per SM
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((threads + 255) / 256, 8ll * num_sms)));
}
}  // namespace

cudaError_t launch_mxfp4_quantize(const void* x, int xt, int64_t x_rows, const int32_t* src_rows, int src_div,
                                  int64_t n_mat, int64_t rows, int64_t cols, void* dst, int num_sms, cudaStream_t s) {
    const int64_t items = n_mat * rows * mx_panels(cols);
    return launch_pdl(mxfp4_quantize_kernel, dim3(grid_for(items * 16, num_sms)), dim3(256), 0, s, x, xt, x_rows,
                      src_rows, src_div, items, rows, cols, static_cast<uint8_t*>(dst));
}

cudaError_t launch_mxfp4_dequantize(const void* src, int64_t n_mat, int64_t rows, int64_t cols, void* out, int ot,
                                    int num_sms, cudaStream_t s) {
    const int64_t items = n_mat * rows * (cols / 8);
    return launch_pdl(mxfp4_dequantize_kernel, dim3(grid_for(items, num_sms)), dim3(256), 0, s,
                      static_cast<const uint8_t*>(src), items, rows, cols, out, ot);
}

}  // namespace moe
