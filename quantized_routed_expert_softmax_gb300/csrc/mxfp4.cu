// mxfp4.cu -- MXFP4 (OCP microscaling: E2M1 codes, one E8M0 scale per 32 consecutive values of a
// row): the quantiser of weights and expert inputs, and its inverse.
//
// Per block of 32: X = max(floor(log2 amax) - 2, -127), scale byte X + 127, codes E2M1(x * 2^-X)
// rounded to nearest even and saturated at 6 (2 is E2M1's largest exponent, so amax lands in
// [4, 8)).  Every step is exact up to the one rounding into the code: the exponent is read off the
// fp32 bits and 2^-X is a power of two in fp32's normal range (-X is in [-125, 127]).
//
// Measured (GB300): quantising 45056 x 2816 fp32 85.8 us, 6.7 TB/s read and written, the rate of a copy; 4096
// rows x 2816 bf16 from L2 8.2 us (gathered 8.7), bound by instructions; 45056 x 2816 bf16 64.0 us, 5.0 TB/s.  The
// decode of the same to fp32 92 us, 6.2 TB/s, seven eighths of it stores, to bf16 58.8 us, 5.5 TB/s.
#include <algorithm>

#include "mxfp4.cuh"

namespace moe {

// Eight values -> eight E2M1 codes, the first in the low nibble; a zero magnitude is coded +0.
__device__ __forceinline__ uint32_t e2m1x8(const float v[8], float mul) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(v[0] * mul), "f"(v[1] * mul), "f"(v[2] * mul), "f"(v[3] * mul), "f"(v[4] * mul), "f"(v[5] * mul),
          "f"(v[6] * mul), "f"(v[7] * mul));
    const uint32_t mag = w & 0x77777777u;
    return mag | (w & (mag + 0x77777777u) & 0x88888888u);   // the sign of a nibble with a magnitude
}
// Eight codes -> their values as four f16 pairs (exact).
__device__ __forceinline__ void e2m1x8_values(uint32_t w, uint32_t h[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Eight consecutive values.  fp32: one 32-byte access where the base is 32-byte aligned (every offset is
// a multiple of 8 values); two 16-byte ones of a warp would each touch every sector it covers.
template <bool F32>
__device__ __forceinline__ void load8(const char* p, bool wide, float v[8]) {
    if (F32 && wide) {
        asm("ld.global.nc.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
            : "l"(p));
    } else if (F32) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

// Both kernels: 16 lanes have a row and 8 consecutive values each, a panel of 128 columns, so that a panel's
// loads and stores are whole 128-byte lines and its scale word has one writer.  The quantiser's pass of a CTA
// is 16 rows (their scale words lie side by side) by `run` panels, two at a time; addresses advance by
// constants within it, as the kernel is bound by issuing instructions where the data is in L2.
// grid: x passes (grid-stride), y matrices (grid-stride).
struct MxRuns {
    uint32_t chunks, passes;   // runs of a row tile; of a matrix
    int run, npan;
};

constexpr int kMxCtas = 6;   // CTAs of 256 threads per SM (40 registers)

template <bool F32>
__global__ void __launch_bounds__(256, kMxCtas) mxfp4_quantize_kernel(const char* __restrict__ x, int64_t x_rows,
                                                                       const int32_t* __restrict__ src_rows, int src_div,
                                                                       MxRuns runs, int64_t n_mat, int64_t rows, int cols,
                                                                       bool wide, uint8_t* __restrict__ dst) {
    pdl_wait();
    constexpr int kElem = F32 ? 4 : 2;
    const int lane16 = threadIdx.x & 15;
    for (int64_t m = blockIdx.y; m < n_mat; m += gridDim.y) {
        uint8_t* out = dst + m * mx_bytes(rows, cols);
        for (uint32_t pass = blockIdx.x; pass < runs.passes; pass += gridDim.x) {
            const uint32_t tile = pass / runs.chunks;
            const int q0 = static_cast<int>(pass - tile * runs.chunks) * runs.run, q1 = min(runs.npan, q0 + runs.run);
            const int64_t r = static_cast<int64_t>(tile) * 16 + (threadIdx.x >> 4);
            const bool live = r < rows;
            int64_t sr = m * rows + r;
            if (src_rows) {
                int32_t i = live ? __ldg(src_rows + r) : -1;
                if (src_div != 1) i = i < 0 ? -1 : i / src_div;
                sr = i >= x_rows ? -1 : i;
            }
            int c = q0 * 128 + lane16 * 8;
            const bool has = live && sr >= 0;
            const char* src = x + (sr * cols + c) * kElem;
            uint8_t* o = out + r * (cols / 2) + c / 2;
            uint32_t* so = reinterpret_cast<uint32_t*>(out + mx_code_bytes(rows, cols)) + q0 * rows + r;
            for (int q = q0; q < q1; q += 2) {   // (the warp's lanes together)
                float v[2][8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
                    if (has && q + u < q1 && c + u * 128 < cols) load8<F32>(src + u * 128 * kElem, wide, v[u]);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t amax = 0;   // as bits: non-negative floats order like their bit patterns, NaN above Inf
#pragma unroll
                    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[u][i]) & 0x7fffffffu);
                    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                    const bool bad = amax >= 0x7f800000u, in = live && q + u < q1 && c + u * 128 < cols;
                    const int e = max(static_cast<int>(amax >> 23) - 2, 0);   // X + 127
                    const uint32_t codes = bad ? 0u : e2m1x8(v[u], __uint_as_float(static_cast<uint32_t>(254 - e) << 23));
                    const uint32_t sb = c + u * 128 >= cols ? kMxScalePad : (bad ? kMxScaleNaN : static_cast<uint32_t>(e));
                    uint32_t word = sb << (8 * (lane16 >> 2));
                    word |= __shfl_xor_sync(0xffffffffu, word, 4);
                    word |= __shfl_xor_sync(0xffffffffu, word, 8);
                    if (in) *reinterpret_cast<uint32_t*>(o + u * 64) = codes;
                    if (live && q + u < q1 && lane16 == 0) so[u * rows] = word;
                }
                c += 256;
                src += 256 * kElem;
                o += 128;
                so += 2 * rows;
            }
        }
    }
}

// The decode writes most: the half warps go along the rows, so that a CTA's pass writes one run of memory
// (by tiles of 16 rows 45056 x 2816 fp32 took 108 us).  Items (row, panel) are numbered within slabs of rows,
// whose items fit 30 bits; the division by the panels of a row is a multiplication.
struct MxItems {
    uint32_t npan, div_mul, div_shift;   // div_mul 0: npan is 1
    uint32_t items;                      // of a slab
    int64_t slab_rows;
};

// CTAs per SM.  fp32: with 4 (up to 64 registers) 45056 x 2816 took 95 us, with 6 (40) 102; bf16: 4096 x 2816 from
// L2 8.7 and 7.3.
constexpr int mx_decode_ctas(bool f32) { return f32 ? 4 : 6; }

template <bool F32>
__global__ void __launch_bounds__(256, mx_decode_ctas(F32)) mxfp4_dequantize_kernel(const uint8_t* __restrict__ src, MxItems n,
                                                                         int64_t n_mat, int64_t rows, int cols, bool wide,
                                                                         char* __restrict__ out) {
    pdl_wait();
    constexpr int kElem = F32 ? 4 : 2;
    const int lane16 = threadIdx.x & 15;
    const int64_t r0 = blockIdx.z * n.slab_rows;
    const uint32_t items = static_cast<uint32_t>(min(static_cast<int64_t>(n.items), (rows - r0) * n.npan)), step = gridDim.x * 16;
    for (int64_t m = blockIdx.y; m < n_mat; m += gridDim.y) {
        const uint8_t* in = src + m * mx_bytes(rows, cols);
        const uint32_t* scales = reinterpret_cast<const uint32_t*>(in + mx_code_bytes(rows, cols));
        for (uint32_t it = blockIdx.x * 16 + (threadIdx.x >> 4); it < items; it += 2 * step) {
            uint32_t codes[2], word[2];
            char* d[2];
            bool has[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t i = it + u * step, row = n.div_mul ? __umulhi(i, n.div_mul) >> n.div_shift : i;
                const uint32_t q = i - row * n.npan;
                const int c = static_cast<int>(q * 128 + lane16 * 8);
                const int64_t r = r0 + row;
                has[u] = i < items && c < cols;
                codes[u] = has[u] ? __ldg(reinterpret_cast<const uint32_t*>(in + r * (cols / 2) + c / 2)) : 0;
                word[u] = has[u] ? __ldg(scales + (q * rows + r)) : 0;
                d[u] = out + ((m * rows + r) * cols + c) * kElem;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (!has[u]) continue;
                const float s = mx_scale((word[u] >> (8 * (lane16 >> 2))) & 0xffu);
                uint32_t h[4];
                e2m1x8_values(codes[u], h);
                float v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
                    v[2 * i] = f.x * s;
                    v[2 * i + 1] = f.y * s;
                }
                if (F32 && wide) {
                    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(d[u]), "f"(v[0]), "f"(v[1]),
                                 "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                                 : "memory");
                } else if (F32) {
                    reinterpret_cast<float4*>(d[u])[0] = make_float4(v[0], v[1], v[2], v[3]);
                    reinterpret_cast<float4*>(d[u])[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else {   // exact: a code has 2 significant bits, and bf16 has fp32's exponents
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                        w[i] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                    *reinterpret_cast<uint4*>(d[u]) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
    }
}

// ------------------------------------------------------------------------------- launchers
namespace {

// Passes of two panels where that leaves at most four to a CTA, else longer ones.
MxRuns mx_runs(int64_t n_mat, int64_t rows, int64_t cols, int num_sms) {
    MxRuns m{};
    const int64_t tiles = (rows + 15) / 16, npan = mx_panels(cols), ctas = static_cast<int64_t>(kMxCtas) * num_sms;
    m.npan = static_cast<int>(npan);
    const int64_t run = n_mat * tiles * npan / (4 * ctas) / 2 * 2;
    m.run = static_cast<int>(std::max<int64_t>(2, std::min<int64_t>(run, 8)));
    m.chunks = static_cast<uint32_t>((npan + m.run - 1) / m.run);
    m.passes = static_cast<uint32_t>(tiles * m.chunks);   // (at most 2^21 * 256)
    return m;
}

// One wave of CTAs over the passes of all matrices.
dim3 mx_grid(const MxRuns& m, int64_t n_mat, int num_sms) {
    const int64_t ctas = static_cast<int64_t>(kMxCtas) * num_sms;
    const int64_t gx = std::min<int64_t>(m.passes, ctas);
    return dim3(static_cast<unsigned>(gx), static_cast<unsigned>(std::min<int64_t>(n_mat, std::max<int64_t>(1, ctas / gx))));
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const void* x, int xt, int64_t x_rows, const int32_t* src_rows, int src_div,
                                  int64_t n_mat, int64_t rows, int64_t cols, void* dst, int num_sms, cudaStream_t s) {
    const MxRuns m = mx_runs(n_mat, rows, cols, num_sms);
    return launch_pdl(xt == MOE_F32 ? mxfp4_quantize_kernel<true> : mxfp4_quantize_kernel<false>,
                      mx_grid(m, n_mat, num_sms), dim3(256), 0, s, static_cast<const char*>(x), x_rows, src_rows, src_div, m,
                      n_mat, rows, static_cast<int>(cols), (reinterpret_cast<uintptr_t>(x) & 31u) == 0,
                      static_cast<uint8_t*>(dst));
}

cudaError_t launch_mxfp4_dequantize(const void* src, int64_t n_mat, int64_t rows, int64_t cols, void* out, int ot,
                                    int num_sms, cudaStream_t s) {
    MxItems m{};
    m.npan = static_cast<uint32_t>(mx_panels(cols));
    m.slab_rows = std::min<int64_t>(rows, (1ll << 30) / m.npan);
    m.items = static_cast<uint32_t>(m.slab_rows * m.npan);
    // i / npan for i < 2^30 as i * mul / 2^(30 + bits), mul = ceil(2^(30 + bits) / npan): mul npan is at most
    // npan - 1 < 2^bits too large, which i makes less than 2^(30 + bits), so the quotient is off by less than
    // 1 / npan
    if (m.npan > 1) {
        int bits = 2;
        while ((1u << bits) < m.npan) ++bits;
        m.div_mul = static_cast<uint32_t>(((uint64_t(1) << (30 + bits)) + m.npan - 1) / m.npan);
        m.div_shift = static_cast<uint32_t>(bits - 2);   // behind __umulhi's 32
    }
    const int64_t ctas = static_cast<int64_t>(mx_decode_ctas(ot == MOE_F32)) * num_sms;
    const int64_t gx = std::min<int64_t>((static_cast<int64_t>(m.items) + 31) / 32, ctas);
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(std::min<int64_t>(n_mat, std::max<int64_t>(1, ctas / gx))),
                    static_cast<unsigned>((rows + m.slab_rows - 1) / m.slab_rows));
    return launch_pdl(ot == MOE_F32 ? mxfp4_dequantize_kernel<true> : mxfp4_dequantize_kernel<false>, grid, dim3(256), 0, s,
                      static_cast<const uint8_t*>(src), m, n_mat, rows, static_cast<int>(cols),
                      (reinterpret_cast<uintptr_t>(out) & 31u) == 0, static_cast<char*>(out));
}

}  // namespace moe
