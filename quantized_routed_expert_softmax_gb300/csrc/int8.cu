// int8.cu -- rows coded in 8-bit integers with one fp32 scale each: the quantiser of expert inputs (and of weights with
// any number of rows), and its inverse.
//
// Per row: s = amax / 127, q = round-half-away(x / s), both divisions correctly rounded in fp32, as the per-channel
// weight packer has them.  A division a value would bound the kernel by instructions, so the quotient is taken as x * (1 / s).
// For bf16 rows the factor is chosen so that this always gives the same code (i8_factor); for fp32 an exact comparison decides
// where the quotient lies close to the middle between two codes (i8_codes).
//
// Measured: quantising 45056 x 2816 fp32 96 us, 6.6 TB/s read and written; 32768 x 2816 bf16 45 us, 6.1 TB/s, gathered from
// 4097 rows in L2 34 us, 32764 rows 44 and 38; one row 2.5 us.  Bound by HBM; the gathered rows, at half its
// rate, by a row's copy, search and coding one after the other or by their stores, which of these has not been measured.
// What it took, us for 32764 gathered bf16 rows: rows in registers 82; read again from L1 58; held in shared memory 52; one
// decision a row for values close to a middle, in place of one a value, 39 (a quarter of a warp's steps had such a value).  Not
// gathered 82, 69 by then, and 44 by panels.
// The decode to fp32 113 us, 5.6 TB/s, of 32764 x 2816 to bf16 46 us, 6.0 TB/s.
#include <algorithm>

#include "int8.cuh"

namespace moe {

// Eight consecutive values as fp32.  fp32: one 32-byte access where the base is 32-byte aligned.
template <bool F32>
__device__ __forceinline__ void i8_load8(const char* p, bool wide, uint32_t* raw) {
    if (F32 && wide) {
        asm("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
            : "=r"(raw[0]), "=r"(raw[1]), "=r"(raw[2]), "=r"(raw[3]), "=r"(raw[4]), "=r"(raw[5]), "=r"(raw[6]), "=r"(raw[7])
            : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
            raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
        }
    }
}
template <bool F32>
__device__ __forceinline__ void i8_values(const uint32_t* raw, float* v) {
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) {
        if (F32) {
            v[i] = __uint_as_float(raw[i]);
        } else {
            v[2 * i] = __uint_as_float(raw[i] << 16);
            v[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
        }
    }
}
// The larger of m and the magnitudes of eight values, as bits (non-negative floats order like their bit patterns, NaN above
// Inf); bf16: of both halves of a word at once, a NaN stays, the signs mean nothing.
template <bool F32>
__device__ __forceinline__ uint32_t i8_amax(uint32_t m, const uint32_t* raw) {
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) {
        if (F32) m = max(m, raw[i] & 0x7fffffffu);
        else asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(raw[i]));
    }
    return m;
}
template <bool F32>
__device__ __forceinline__ uint32_t i8_amax_bits(uint32_t m) { return F32 ? m : max((m & 0x7fffu) << 16, m & 0x7fff0000u); }

constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: added, it rounds to an integer and leaves its two's complement in the low byte

// The factor for a row's codes, about 1 / s, or 0 where s is so small that they are divided.
// bf16: the codes are x * inv rounded to the nearest integer, so inv has to be such that no product falls on the other side of
// the middle m between two codes than the rounded quotient.  s comes from a bf16 maximum, one of 128 mantissas: but for
// two cases no bf16 number lies within 2^-16 of a middle m s, relatively (all of them were gone through).  One is amax / 2, whose
// m is 63.5: inv is moved by three steps, if need be, to the side that the exact comparison (i8_codes) asks for.  The other is s = a
// power of two, where x / s meets middles exactly and they go away from zero: inv is the number above 1 / s.
template <bool F32>
__device__ __forceinline__ float i8_factor(float amax, float s) {
    if (!(s >= 1e-27f)) return 0.0f;
    const float inv = __frcp_rn(s);   // (s is 2.7e36 at most)
    if (F32) return inv;
    const float half = 0.5f * amax, want = fmaf(-63.5f, s, half) >= -0x1p-19f * s ? 64.0f : 63.0f;
    int steps = 0;
    if ((__float_as_uint(s) & 0x7fffffu) == 0) steps = 1;
    else if (fmaf(half, inv, kMagic) - kMagic != want) steps = want == 64.0f ? 3 : -3;
    return __uint_as_float(__float_as_uint(inv) + steps);
}

// Eight codes of a row with scale s and that factor.  fp32: what the rounding took off tells how near the quotient is to a
// middle m.  There the rounded quotient decides: it is at least m if |v| / s is at least m less half of fp32's step below m,
// and |v| - m s, a small difference of numbers of 24 and 32 bits, is exact.
constexpr float kNearTie = 0.49997f;   // (the roundings of v inv and inv: 2^-23 of 127 at most, 1.6e-5)
template <bool F32>
__device__ __forceinline__ uint2 i8_codes(const uint32_t* raw, float s, float inv) {
    float v[8];
    i8_values<F32>(raw, v);
    uint32_t b[8];
    float d[8], worst = 0.0f;
    const uint64_t up = pack_f32x2(inv, inv), minus = pack_f32x2(-kMagic, -kMagic), magic = pack_f32x2(kMagic, kMagic);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {   // two values at a time; fp32: the rounded quotients negative, the same low bytes
        const uint64_t w = pack_f32x2(v[i], v[i + 1]);
        uint64_t r = F32 ? minus : magic;
        fma_f32x2(r, w, F32 ? pack_f32x2(-inv, -inv) : up);
        const float2 rf = unpack_f32x2(r);
        b[i] = __float_as_uint(rf.x), b[i + 1] = __float_as_uint(rf.y);
        if (F32) {
            uint64_t t = add_f32x2(r, magic);
            fma_f32x2(t, w, up);
            const float2 df = unpack_f32x2(t);
            d[i] = fabsf(df.x), d[i + 1] = fabsf(df.y);
            asm("max.f32 %0, %0, %1, %2;" : "+f"(worst) : "f"(d[i]), "f"(d[i + 1]));
        }
    }
    uint2 out = make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                           __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
    if (worst >= kNearTie || inv == 0.0f) {
        // value by value, so that lanes whose values are at different places go through this together
        uint32_t left = 0xff;
        if (F32 && inv != 0.0f) {
            left = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) left |= d[i] >= kNearTie ? 1u << i : 0u;
        }
        while (left) {
            const int i = __ffs(left) - 1;
            left &= left - 1;
            const float lo = i & 2 ? (i & 1 ? v[3] : v[2]) : (i & 1 ? v[1] : v[0]);
            const float hi = i & 2 ? (i & 1 ? v[7] : v[6]) : (i & 1 ? v[5] : v[4]);
            const float x = i & 4 ? hi : lo;
            float code;
            if (F32 && inv != 0.0f) {
                const float n = fmaf(x, inv, kMagic) - kMagic;
                const float m = fabsf(n + copysignf(0.5f, fmaf(x, inv, -n)));
                const float step = m == 0.5f ? 0x1p-26f : __uint_as_float((__float_as_uint(m) & 0x7f800000u) - (24u << 23));
                code = copysignf(fmaf(-m, s, fabsf(x)) >= -step * s ? m + 0.5f : m - 0.5f, x);
            } else {
                code = fminf(fmaxf(roundf(__fdiv_rn(x, s)), -127.0f), 127.0f);
            }
            const uint32_t byte = (__float_as_uint(code + kMagic) & 0xffu) << (8 * (i & 3)), keep = ~(0xffu << (8 * (i & 3)));
            if (i & 4) out.y = (out.y & keep) | byte;
            else out.x = (out.x & keep) | byte;
        }
    }
    return out;
}

constexpr int kQRow = 256;   // columns that a warp covers at a time, eight a lane

__device__ __forceinline__ void i8_copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// `split` warps a row, 8 / split consecutive rows a CTA, so that a panel's codes of a CTA's rows lie side by side.  Between
// the search for the largest and the coding a lane holds its part of the row, eight values each time: ITERS times in
// registers (fp32), or in shared memory (bf16); 0: it reads the row again.  kHeldPanels: the codes go through shared memory too,
// and 16 bytes a lane to their panels.
constexpr int kHeld = -1, kHeldPanels = -2, kMaxIters = 12;
__host__ __device__ constexpr int held_row(int iters) { return iters * 512 + 32; }   // (32: the rows of a panel lie in different banks)
template <bool F32, int ITERS>
__global__ void __launch_bounds__(256, F32 ? 2 : 4) int8_quantize_kernel(const char* __restrict__ x, int64_t x_rows,
                                                            const int32_t* __restrict__ src_rows, int src_div, int64_t n_mat,
                                                            int64_t rows, int cols, int split, bool wide,
                                                            uint8_t* __restrict__ dst) {
    constexpr int kElem = F32 ? 4 : 2, kRaw = F32 ? 8 : 4;
    __shared__ uint32_t largest[8];
    extern __shared__ __align__(16) unsigned char held[];
    pdl_wait();   // (no early trigger: with the next kernel's blocks among its own, quantising and decoding 32764 rows takes 104 us, not 87)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp & (split - 1), lead = warp - sub;
    const int per = 8 / split, split_log = __ffs(split) - 1, per_log = 3 - split_log, step = split * kQRow, c0 = sub * kQRow + lane * 8;
    const int64_t groups = (rows + per - 1) / per;
    for (int64_t m = blockIdx.y; m < n_mat; m += gridDim.y) {
        uint8_t* out = dst + m * i8_bytes(rows, cols);
        for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x) {
            const int64_t r = grp * per + warp / split;
            const bool live = r < rows;
            int64_t sr = m * rows + r;
            if (src_rows) {
                int32_t i = live ? __ldg(src_rows + r) : -1;
                if (src_div != 1) i = i < 0 ? -1 : i / src_div;
                sr = i >= x_rows ? -1 : i;
            }
            const bool has = live && sr >= 0;
            const char* src = x + (sr * cols + c0) * kElem;
            uint32_t raw[ITERS > 0 ? ITERS : 1][kRaw];
            uint32_t amax = 0;
            const int times = (cols - c0 + step - 1) / step;   // that this lane has eight values
            const int iters = (cols + step - 1) / step;
            unsigned char* mine = held + warp * held_row(iters);
            if constexpr (ITERS < 0) {
                if (has) {
                    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(mine)) + lane * 16;
                    const char* from = src;
                    for (int u = 0; u < times; ++u, from += step * kElem) i8_copy16(to + u * 512, from);
                    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 4
                    for (int u = 0; u < times; ++u) amax = i8_amax<F32>(amax, reinterpret_cast<const uint32_t*>(mine + u * 512 + lane * 16));
                }
            } else if constexpr (ITERS > 0) {
#pragma unroll
                for (int u = 0; u < ITERS; ++u) {
#pragma unroll
                    for (int i = 0; i < kRaw; ++i) raw[u][i] = 0;
                    if (has && c0 + u * step < cols) i8_load8<F32>(src + static_cast<int64_t>(u) * step * kElem, wide, raw[u]);
                }
#pragma unroll
                for (int u = 0; u < ITERS; ++u) amax = i8_amax<F32>(amax, raw[u]);
            } else if (has) {
                for (int c = c0; c < cols; c += 4 * step) {
                    uint32_t w[4][kRaw];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
#pragma unroll
                        for (int i = 0; i < kRaw; ++i) w[u][i] = 0;
                        if (c + u * step < cols) i8_load8<F32>(src + static_cast<int64_t>(c - c0 + u * step) * kElem, false, w[u]);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) amax = i8_amax<F32>(amax, w[u]);
                }
            }
            amax = __reduce_max_sync(0xffffffffu, i8_amax_bits<F32>(amax));
            if (split > 1) {
                if (lane == 0) largest[warp] = amax;
                __syncthreads();
                for (int i = 0; i < split; ++i) amax = max(amax, largest[lead + i]);
                __syncthreads();
            }
            if (ITERS != kHeldPanels && !live) continue;
            const bool bad = amax >= 0x7f800000u;
            const float s = __fdiv_rn(__uint_as_float(amax), 127.0f);
            const float inv = i8_factor<F32>(__uint_as_float(amax), s);
            const bool code = has && !bad && s > 0.0f;
            uint8_t* o = out + i8_scale_bytes(rows) + (static_cast<int64_t>(c0 >> 5) * rows + r) * 32 + (c0 & 31);
            const int64_t o_step = static_cast<int64_t>(step >> 5) * rows * 32;
            if constexpr (ITERS == kHeld) {
#pragma unroll 2
                for (int u = 0; u < times; ++u, o += o_step) {
                    const uint4 w = *reinterpret_cast<const uint4*>(mine + u * 512 + lane * 16);
                    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
                    *reinterpret_cast<uint2*>(o) = code ? i8_codes<F32>(v, s, inv) : make_uint2(0, 0);
                }
            } else if constexpr (ITERS == kHeldPanels) {
                // the codes over the values, which all lanes have read by then
#pragma unroll 2
                for (int u = 0; u < iters; ++u) {
                    uint2 c = make_uint2(0, 0);
                    if (code && u < times) {
                        const uint4 w = *reinterpret_cast<const uint4*>(mine + u * 512 + lane * 16);
                        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
                        c = i8_codes<F32>(v, s, inv);
                    }
                    __syncwarp();
                    *reinterpret_cast<uint2*>(mine + u * 256 + lane * 8) = c;
                }
            } else if constexpr (ITERS > 0) {
#pragma unroll
                for (int u = 0; u < ITERS; ++u)
                    if (c0 + u * step < cols)
                        *reinterpret_cast<uint2*>(o + u * o_step) = code ? i8_codes<F32>(raw[u], s, inv) : make_uint2(0, 0);
            } else {
                for (int c = c0; c < cols; c += step, o += o_step) {
                    if (code) i8_load8<F32>(src + static_cast<int64_t>(c - c0) * kElem, false, raw[0]);
                    *reinterpret_cast<uint2*>(o) = code ? i8_codes<F32>(raw[0], s, inv) : make_uint2(0, 0);
                }
            }
            if (live && sub == 0 && lane == 0) reinterpret_cast<float*>(out)[r] = bad ? __uint_as_float(0x7fffffffu) : s;
            if constexpr (ITERS == kHeldPanels) {   // a panel's codes of the CTA's rows, 16 bytes a lane
                const int64_t r0 = grp * per;
                const int pieces = 2 * static_cast<int>(min(static_cast<int64_t>(per), rows - r0));
                uint8_t* to = out + i8_scale_bytes(rows) + r0 * 32;
                __syncthreads();
                for (int i = threadIdx.x; i < (cols >> 5) * 2 * per; i += 256) {
                    const int panel = i >> (per_log + 1), j = i & (2 * per - 1), set = panel >> 3;
                    if (j >= pieces) continue;
                    const unsigned char* from = held + ((j >> 1) * split + (set & (split - 1))) * held_row(iters);
                    from += (set >> split_log) * 256 + (panel & 7) * 32 + (j & 1) * 16;
                    *reinterpret_cast<uint4*>(to + static_cast<int64_t>(panel) * rows * 32 + j * 16) = *reinterpret_cast<const uint4*>(from);
                }
                __syncthreads();
            }
        }
    }
}

// A warp a row, eight consecutive rows a CTA; grid.y takes parts of the columns where there are few rows.
template <bool F32>
__global__ void __launch_bounds__(256) int8_dequantize_kernel(const uint8_t* __restrict__ src, int64_t n_mat, int64_t rows,
                                                              int cols, bool wide, char* __restrict__ out) {
    constexpr int kElem = F32 ? 4 : 2;
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int step = gridDim.y * kQRow, c0 = blockIdx.y * kQRow + lane * 8;
    const int64_t groups = (rows + 7) / 8;
    for (int64_t m = blockIdx.z; m < n_mat; m += gridDim.z) {
        const uint8_t* in = src + m * i8_bytes(rows, cols);
        for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x) {
            const int64_t r = grp * 8 + warp;
            if (r >= rows) continue;
            const float s = __ldg(reinterpret_cast<const float*>(in) + r);
            const uint8_t* p = in + i8_scale_bytes(rows) + (static_cast<int64_t>(c0 >> 5) * rows + r) * 32 + (c0 & 31);
            const int64_t p_step = static_cast<int64_t>(step >> 5) * rows * 32;
            char* d = out + ((m * rows + r) * cols + c0) * kElem;
#pragma unroll 4
            for (int c = c0; c < cols; c += step, p += p_step, d += static_cast<int64_t>(step) * kElem) {
                const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {   // 2^23 in front of the byte c + 128: 2^23 + 128 + c
                    const uint32_t w = (i < 4 ? q.x : q.y) ^ 0x80808080u;
                    v[i] = (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7650 + (i & 3))) - 8388736.0f) * s;
                }
                if (F32 && wide) {
                    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(d), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                                 : "memory");
                } else if (F32) {
                    reinterpret_cast<float4*>(d)[0] = make_float4(v[0], v[1], v[2], v[3]);
                    reinterpret_cast<float4*>(d)[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                        w[i] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
    }
}

namespace {

using QuantizeKernel = void (*)(const char*, int64_t, const int32_t*, int, int64_t, int64_t, int, int, bool, uint8_t*);

// bf16 by panels: where these start 16 bytes off a sector each store of a lane's codes would meet two (32764 rows of 2816: 68 us,
// by panels 44); where they do not, the barriers of the panels cost more (32768 rows 43 against 45, gathered 38 against 34,
// 100000 rows of 704 52 against 46).  Rows longer than shared memory has room for are read again.
QuantizeKernel quantize_kernel(bool f32, int iters, bool panels) {
    if (!f32 && iters > kMaxIters) return int8_quantize_kernel<false, 0>;
    if (!f32) return panels ? int8_quantize_kernel<false, kHeldPanels> : int8_quantize_kernel<false, kHeld>;
    if (iters <= 3) return int8_quantize_kernel<true, 3>;
    if (iters <= 6) return int8_quantize_kernel<true, 6>;
    return iters <= kMaxIters ? int8_quantize_kernel<true, kMaxIters> : int8_quantize_kernel<true, 0>;
}

}  // namespace

cudaError_t configure_int8_codec() {
    cudaError_t e = cudaSuccess;
    for (bool panels : {false, true}) {
        const void* fn = reinterpret_cast<const void*>(quantize_kernel(false, 1, panels));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 8 * held_row(kMaxIters));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    }
    return e;
}

cudaError_t launch_int8_quantize(const void* x, int xt, int64_t x_rows, const int32_t* src_rows, int src_div, int64_t n_mat,
                                 int64_t rows, int64_t cols, void* dst, int num_sms, cudaStream_t s) {
    // Warps a row: more while a lane would hold more than 12 times eight values, or while half the SMs would have no CTA
    // and a warp more than 256 columns.
    int split = 1;
    auto iters = [&] { return static_cast<int>((cols + split * kQRow - 1) / (split * kQRow)); };
    while (split < 8 && (iters() > kMaxIters || (iters() > 1 && n_mat * rows * split < 4ll * num_sms))) split *= 2;
    const bool in_shared = xt != MOE_F32 && iters() <= kMaxIters, panels = in_shared && i8_scale_bytes(rows) % 32 != 0;
    const int64_t groups = (rows * split + 7) / 8;
    // (by panels: a CTA for about kMaxIters steps, so that its barriers meet other CTAs' work: 32764 rows 47 -> 44 us)
    const int64_t ctas = std::max<int64_t>(8ll * num_sms, panels ? groups / (kMaxIters / iters()) : 0);
    const int64_t gx = std::min<int64_t>(groups, ctas);
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(std::min<int64_t>(n_mat, std::max<int64_t>(1, ctas / gx))));
    const size_t held = in_shared ? 8 * static_cast<size_t>(held_row(iters())) : 0;
    return launch_pdl(quantize_kernel(xt == MOE_F32, iters(), panels), grid, dim3(256), held, s,
                      static_cast<const char*>(x), x_rows, src_rows, src_div, n_mat, rows, static_cast<int>(cols), split,
                      (reinterpret_cast<uintptr_t>(x) & 31u) == 0, static_cast<uint8_t*>(dst));
}

cudaError_t launch_int8_dequantize(const void* src, int64_t n_mat, int64_t rows, int64_t cols, void* out, int ot, int num_sms,
                                   cudaStream_t s) {
    const int64_t groups = (rows + 7) / 8, ctas = 8ll * num_sms;
    const int64_t gx = std::min<int64_t>(groups, ctas), chunks = (cols + kQRow - 1) / kQRow;
    const int64_t gz = std::min<int64_t>(n_mat, std::max<int64_t>(1, ctas / gx));
    const int64_t gy = std::min<int64_t>(chunks, std::max<int64_t>(1, ctas / (gx * gz)));
    return launch_pdl(ot == MOE_F32 ? int8_dequantize_kernel<true> : int8_dequantize_kernel<false>,
                      dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy), static_cast<unsigned>(gz)), dim3(256), 0, s,
                      static_cast<const uint8_t*>(src), n_mat, rows, static_cast<int>(cols), (reinterpret_cast<uintptr_t>(out) & 31u) == 0,
                      static_cast<char*>(out));
}

}  // namespace moe
