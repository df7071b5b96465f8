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

// Eight consecutive values.  fp32: one 32-byte access where the base is 32-byte aligned (every offset is
// a multiple of 8 values); two 16-byte ones of a warp would each touch every sector it covers.
template <bool F32>
__device__ __forceinline__ void load8(const void* x, int64_t off, bool wide, float v[8]) {
    if (F32 && wide) {
        asm("ld.global.nc.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
            : "l"(static_cast<const float*>(x) + off));
    } else if (F32) {
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

// Both kernels work on items of (row, panel of 128 columns), 16 lanes an item and 8 consecutive values a
// lane, so that a panel's loads and stores are whole 128-byte lines and its scale word has one writer.  Items
// go by tiles of 16 rows: the 16 items of a CTA's pass are one panel of 16 rows (their scale words lie side
// by side), and the next CTA's are the panel beside it.  A thread has two items' reads in flight.
// grid: x items of a slab (grid-stride), y slabs of rows (their items fit 30 bits), z matrices.
struct MxItems {
    uint32_t div_mul, div_shift;   // tile number / npan by a multiplication (0: npan is 1)
    uint32_t npan, row_bits;       // rows of a tile: 16, or 1 below 16 rows
    uint32_t items;                // of a slab, tiles filled up
    int64_t slab_rows;             // a multiple of the tile's

    __device__ __forceinline__ void at(uint32_t it, uint32_t* row, uint32_t* panel) const {
        const uint32_t t = it >> row_bits, tile = div_mul ? __umulhi(t, div_mul) >> div_shift : t;
        *panel = t - tile * npan;
        *row = (tile << row_bits) + (it & ((1u << row_bits) - 1u));
    }
};

constexpr int kMxCtas = 6;   // CTAs of 256 threads per SM (40 registers)

template <bool F32>
__global__ void __launch_bounds__(256, kMxCtas) mxfp4_quantize_kernel(const void* __restrict__ x, int64_t x_rows,
                                                              const int32_t* __restrict__ src_rows, int src_div,
                                                              MxItems items, int64_t rows, int64_t cols, bool wide,
                                                              uint8_t* __restrict__ dst) {
    pdl_wait();
    pdl_trigger();
    const int lane16 = threadIdx.x & 15;
    const int64_t r0 = blockIdx.y * items.slab_rows, code_bytes = mx_code_bytes(rows, cols);
    const int64_t src0 = blockIdx.z * rows;
    uint8_t* out = dst + blockIdx.z * mx_bytes(rows, cols);
    const uint32_t step = gridDim.x * 16;   // items of a pass of the grid
    // (the lanes of a warp differ in their item's lowest bit only, so all of them stay in the loop together)
    for (uint32_t it = blockIdx.x * 16 + (threadIdx.x >> 4); (it & ~1u) < items.items; it += 2 * step) {
        float v[2][8];
        int64_t r[2];
        uint32_t q[2];
        bool live[2], in[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t row;
            items.at(it + u * step, &row, &q[u]);
            r[u] = r0 + row;
            live[u] = it + u * step < items.items && row < items.slab_rows && r[u] < rows;
            const int64_t c = q[u] * 128ll + lane16 * 8;
            in[u] = live[u] && c < cols;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
            int64_t sr = src0 + r[u];
            if (src_rows) {
                int32_t i = live[u] ? __ldg(src_rows + r[u]) : -1;
                if (src_div != 1) i = i < 0 ? -1 : i / src_div;
                sr = i >= x_rows ? -1 : i;
            }
            if (in[u] && sr >= 0) load8<F32>(x, sr * cols + c, wide, v[u]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t amax = 0;   // as bits: non-negative floats order like their bit patterns, NaN above Inf
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[u][i]) & 0x7fffffffu);
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const bool bad = amax >= 0x7f800000u;
            const int e = max(static_cast<int>(amax >> 23) - 2, 0);   // X + 127
            const uint32_t codes = bad ? 0u : e2m1x8(v[u], __uint_as_float(static_cast<uint32_t>(254 - e) << 23));
            const uint32_t sb = !in[u] ? kMxScalePad : (bad ? kMxScaleNaN : static_cast<uint32_t>(e));
            uint32_t word = sb << (8 * (lane16 >> 2));
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
            word |= __shfl_xor_sync(0xffffffffu, word, 8);
            if (in[u]) *reinterpret_cast<uint32_t*>(out + r[u] * (cols / 2) + q[u] * 64 + lane16 * 4) = codes;
            if (live[u] && lane16 == 0) *reinterpret_cast<uint32_t*>(out + code_bytes + 4 * (q[u] * rows + r[u])) = word;
        }
    }
}

template <bool F32>
__global__ void __launch_bounds__(256, kMxCtas) mxfp4_dequantize_kernel(const uint8_t* __restrict__ src, MxItems items,
                                                                int64_t rows, int64_t cols, bool wide,
                                                                void* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    const int lane16 = threadIdx.x & 15;
    const int64_t r0 = blockIdx.y * items.slab_rows, code_bytes = mx_code_bytes(rows, cols);
    const uint8_t* p = src + blockIdx.z * mx_bytes(rows, cols);
    const uint32_t step = gridDim.x * 16;
    for (uint32_t it = blockIdx.x * 16 + (threadIdx.x >> 4); it < items.items; it += 2 * step) {
        uint32_t codes[2], word[2];
        int64_t o[2];
        bool in[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t row, q;
            items.at(it + u * step, &row, &q);
            const int64_t r = r0 + row, c = q * 128ll + lane16 * 8;
            in[u] = it + u * step < items.items && row < items.slab_rows && r < rows && c < cols;
            o[u] = (blockIdx.z * rows + r) * cols + c;
            codes[u] = in[u] ? __ldg(reinterpret_cast<const uint32_t*>(p + r * (cols / 2) + c / 2)) : 0;
            word[u] = in[u] ? __ldg(reinterpret_cast<const uint32_t*>(p + code_bytes + 4 * (q * rows + r))) : 0;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (!in[u]) continue;
            const float s = mx_scale((word[u] >> (8 * (lane16 >> 2))) & 0xffu);
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = e2m1x2_to_f32x2((codes[u] >> (8 * i)) & 0xffu);
                v[2 * i] = f.x * s;
                v[2 * i + 1] = f.y * s;
            }
            if (F32 && wide) {
                asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(static_cast<float*>(out) + o[u]),
                             "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                             : "memory");
            } else if (F32) {
                float4* d = reinterpret_cast<float4*>(static_cast<float*>(out) + o[u]);
                d[0] = make_float4(v[0], v[1], v[2], v[3]);
                d[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {   // exact: a code has 2 significant bits, and bf16 has fp32's exponents
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o[u]) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// ------------------------------------------------------------------------------- launchers
namespace {

MxItems mx_items(int64_t rows, int64_t cols) {
    MxItems m{};
    m.npan = static_cast<uint32_t>(mx_panels(cols));
    m.row_bits = rows >= 16 ? 4 : 0;
    const int64_t tile = 1ll << m.row_bits;
    m.slab_rows = std::min<int64_t>((rows + tile - 1) / tile * tile, (1ll << 30) / m.npan / tile * tile);
    m.items = static_cast<uint32_t>(m.slab_rows * m.npan);
    // t / npan for t < 2^30 as t * mul / 2^(30 + bits), mul = ceil(2^(30 + bits) / npan): mul npan is at most
    // npan - 1 < 2^bits too large, which t makes less than 2^(30 + bits), so the quotient is off by less than
    // 1 / npan
    if (m.npan > 1) {
        int bits = 2;
        while ((1u << bits) < m.npan) ++bits;
        m.div_mul = static_cast<uint32_t>(((uint64_t(1) << (30 + bits)) + m.npan - 1) / m.npan);
        m.div_shift = static_cast<uint32_t>(bits - 2);   // behind __umulhi's 32
    }
    return m;
}

// Two items a half warp at a time; one wave of CTAs, grid-stride.
dim3 mx_grid(const MxItems& m, int64_t n_mat, int64_t rows, int num_sms) {
    const int64_t want = (static_cast<int64_t>(m.items) + 31) / 32;
    return dim3(static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(kMxCtas) * num_sms)),
                static_cast<unsigned>((rows + m.slab_rows - 1) / m.slab_rows), static_cast<unsigned>(n_mat));
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const void* x, int xt, int64_t x_rows, const int32_t* src_rows, int src_div,
                                  int64_t n_mat, int64_t rows, int64_t cols, void* dst, int num_sms, cudaStream_t s) {
    const MxItems m = mx_items(rows, cols);
    return launch_pdl(xt == MOE_F32 ? mxfp4_quantize_kernel<true> : mxfp4_quantize_kernel<false>,
                      mx_grid(m, n_mat, rows, num_sms), dim3(256), 0, s, x, x_rows, src_rows, src_div, m, rows, cols,
                      (reinterpret_cast<uintptr_t>(x) & 31u) == 0, static_cast<uint8_t*>(dst));
}

cudaError_t launch_mxfp4_dequantize(const void* src, int64_t n_mat, int64_t rows, int64_t cols, void* out, int ot,
                                    int num_sms, cudaStream_t s) {
    const MxItems m = mx_items(rows, cols);
    return launch_pdl(ot == MOE_F32 ? mxfp4_dequantize_kernel<true> : mxfp4_dequantize_kernel<false>,
                      mx_grid(m, n_mat, rows, num_sms), dim3(256), 0, s, static_cast<const uint8_t*>(src), m, rows, cols,
                      (reinterpret_cast<uintptr_t>(out) & 31u) == 0, out);
}

}  // namespace moe
