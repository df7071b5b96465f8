// ffn.cu -- the gated feed-forward block over bf16 weights, rows sorted by expert, forward and backward.
#include <algorithm>

#include "int8.cuh"

namespace moe {

// One kernel for the block's six products: out[e][n][m] = sum_k A(m, k) B(n, k), a thread a result.
//   rows:  n is a row of the expert, k a column; A a weight of expert e.
//   grad:  k runs over the expert's rows, m and n are columns.
struct FfnProduct {
    const uint16_t *a, *b;
    int64_t a_mat, a_m, a_k;   // strides of A: expert, m, k
    int64_t b_n, b_k;
    int M, N, K;
    bool grad;
};

enum { kFfnPlain = 0, kFfnAct = 1, kFfnActGrad = 2 };

struct FfnSimple {
    FfnProduct p;
    const int32_t* offsets;
    int P, E, f, act, epi;
    const uint16_t* z_in;
    uint16_t *z_out, *h_out;
    void* out;
    int ot;
};

__device__ __forceinline__ uint16_t ffn_bf16(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

__global__ void __launch_bounds__(256) ffn_simple_kernel(FfnSimple g) {
    pdl_wait();
    const FfnProduct& p = g.p;
    const int m = blockIdx.x * 32 + (threadIdx.x & 31);
    for (int e = blockIdx.y; e < g.E; e += gridDim.y) {
        int first, last;
        expert_rows(g.offsets, e, g.P, &first, &last);
        const int n0 = p.grad ? 0 : first, n1 = p.grad ? p.N : last;
        const int k0 = p.grad ? first : 0, k1 = p.grad ? last : p.K;
        if (m >= p.M) continue;
        const uint16_t* a = p.a + e * p.a_mat + m * p.a_m;
        for (int n = n0 + (threadIdx.x >> 5) + 8 * blockIdx.z; n < n1; n += 8 * gridDim.z) {
            const uint16_t* b = p.b + n * p.b_n;
            float s = 0.0f, s2 = 0.0f;
            for (int64_t k = k0; k < k1; ++k) {
                const float bv = bf16_bits_to_f32(b[k * p.b_k]);
                s = fmaf(bf16_bits_to_f32(a[k * p.a_k]), bv, s);
                if (g.epi == kFfnAct && g.act == MOE_ACT_SWIGLU) s2 = fmaf(bf16_bits_to_f32(a[g.f * p.a_m + k * p.a_k]), bv, s2);
            }
            const int64_t row = static_cast<int64_t>(n);
            if (g.epi == kFfnPlain) {
                const int64_t o = (p.grad ? (static_cast<int64_t>(e) * p.N + n) : row) * p.M + m;
                if (g.ot == MOE_F32) static_cast<float*>(g.out)[o] = s;
                else static_cast<uint16_t*>(g.out)[o] = ffn_bf16(s);
            } else if (g.epi == kFfnAct) {
                const bool gated = g.act == MOE_ACT_SWIGLU;
                const int64_t zo = row * (gated ? 2 * g.f : g.f) + m;
                if (g.z_out) {
                    g.z_out[zo] = ffn_bf16(s);
                    if (gated) g.z_out[zo + g.f] = ffn_bf16(s2);
                }
                g.h_out[row * g.f + m] = ffn_bf16(gated ? silu(s) * s2 : (s > 0.0f ? s * s : (s <= 0.0f ? 0.0f : s)));
            } else {
                const bool gated = g.act == MOE_ACT_SWIGLU;
                const int64_t zo = row * (gated ? 2 * g.f : g.f) + m;
                const float zg = bf16_bits_to_f32(g.z_in[zo]);
                if (gated) {
                    const float zu = bf16_bits_to_f32(g.z_in[zo + g.f]), sg = 1.0f / (1.0f + expf(-zg));
                    g.z_out[zo] = ffn_bf16(s * zu * (sg * (1.0f + zg * (1.0f - sg))));
                    g.z_out[zo + g.f] = ffn_bf16(s * (zg * sg));
                } else {
                    g.z_out[zo] = ffn_bf16(s * (2.0f * (zg > 0.0f ? zg : (zg <= 0.0f ? 0.0f : zg))));
                }
            }
        }
    }
}

static cudaError_t ffn_simple(const FfnSimple& g, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((g.p.M + 31) / 32), static_cast<unsigned>(g.E), g.p.grad ? 8u : (g.E == 1 ? 64u : 4u));
    return launch_pdl(ffn_simple_kernel, grid, dim3(256), 0, s, g);
}

cudaError_t launch_ffn_forward(const uint16_t* x, int64_t P, const uint16_t* wgu, const uint16_t* wd, int64_t E, int64_t d, int64_t f,
                               const int32_t* offsets, int act, uint16_t* y, uint16_t* z, uint16_t* h, int32_t*, int, cudaStream_t s) {
    const int64_t nz = act == MOE_ACT_SWIGLU ? 2 * f : f;
    FfnSimple g{};
    g.offsets = offsets, g.P = static_cast<int>(P), g.E = static_cast<int>(E), g.f = static_cast<int>(f), g.act = act;
    g.p = {wgu, x, nz * d, d, 1, d, 1, static_cast<int>(f), 0, static_cast<int>(d), false};
    g.epi = kFfnAct, g.z_out = z, g.h_out = h;
    cudaError_t e = ffn_simple(g, s);
    if (e != cudaSuccess) return e;
    g.p = {wd, h, d * f, f, 1, f, 1, static_cast<int>(d), 0, static_cast<int>(f), false};
    g.epi = kFfnPlain, g.out = y, g.ot = MOE_BF16;
    return ffn_simple(g, s);
}

cudaError_t launch_ffn_backward(const uint16_t* dy, const uint16_t* x, int64_t P, const uint16_t* wgu, const uint16_t* wd, int64_t E,
                                int64_t d, int64_t f, const int32_t* offsets, int act, const uint16_t* z, const uint16_t* h,
                                uint16_t* dz, uint16_t* dx, void* dwgu, void* dwd, int gt, int32_t*, int, cudaStream_t s) {
    const int64_t nz = act == MOE_ACT_SWIGLU ? 2 * f : f;
    const int id = static_cast<int>(d), jf = static_cast<int>(f), jz = static_cast<int>(nz);
    FfnSimple g{};
    g.offsets = offsets, g.P = static_cast<int>(P), g.E = static_cast<int>(E), g.f = jf, g.act = act;
    cudaError_t e = cudaSuccess;
    if (dx || dwgu) {
        g.p = {wd, dy, d * f, 1, f, d, 1, jf, 0, id, false};
        g.epi = kFfnActGrad, g.z_in = z, g.z_out = dz;
        e = ffn_simple(g, s);
    }
    g.epi = kFfnPlain;
    if (dx && e == cudaSuccess) {
        g.p = {wgu, dz, nz * d, 1, d, nz, 1, id, 0, jz, false};
        g.out = dx, g.ot = MOE_BF16;
        e = ffn_simple(g, s);
    }
    g.ot = gt;
    if (dwgu && e == cudaSuccess) {
        g.p = {x, dz, 0, 1, d, 1, nz, id, jz, 0, true};
        g.out = dwgu;
        e = ffn_simple(g, s);
    }
    if (dwd && e == cudaSuccess) {
        g.p = {h, dy, 0, 1, f, 1, d, jf, id, 0, true};
        g.out = dwd;
        e = ffn_simple(g, s);
    }
    return e;
}

}  // namespace moe
