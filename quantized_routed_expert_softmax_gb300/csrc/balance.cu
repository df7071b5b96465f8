// balance.cu -- the router's load-balance loss over a batch of sequences, its per-expert counts,
// and the gradient of the logits.
//
// Per sequence s with n_s counted tokens (mask != 0):
//   p[t] = softmax(logits[t]),  f_e = counts_e / (k n_s),  P_e = (1 / n_s) sum_t p[t][e],
//   L_s = E sum_e f_e P_e;   loss = mean of L_s over the S' sequences with n_s > 0.
// The counts have no gradient, so
//   dloss/dlogit[t][e] = E / (S' n_s) p_e (f_e - sum_j f_j p_j).
// In a balanced router every f_e is near 1/E and the bracket is a small difference of nearly equal
// numbers.  As sum p = 1 a constant may be taken off f first: with f_e - 1/E, which is formed from
// the integer counts, (E counts_e - k n_s) / (E k n_s), nothing cancels.
//
// No floating-point atomics: every chunk of a sequence's tokens writes its own partial sums, and
// they are added in chunk order.
#include <algorithm>

#include "common.cuh"

namespace moe {

constexpr int kBalThreads = 256, kBalWarps = kBalThreads / 32;

__device__ __forceinline__ float bal_logit(const void* x, int lt, int64_t off) {
    return lt == MOE_F32 ? __ldg(static_cast<const float*>(x) + off)
                         : bf16_bits_to_f32(__ldg(static_cast<const uint16_t*>(x) + off));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The softmax of one row by a warp: lane holds experts lane + 32 i.  A row of -inf has no
// probability at all (p = 0); a NaN or +inf logit makes the row NaN.
template <int NE>
__device__ __forceinline__ void row_softmax(const void* logits, int lt, int64_t t, int E, int lane, float p[NE]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 32 * i;
        p[i] = e < E ? bal_logit(logits, lt, t * E + e) : -INFINITY;
        m = fmaxf(m, p[i]);
    }
    m = warp_max(m);
    if (m == -INFINITY) m = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        p[i] = expf(p[i] - m);
        s += p[i];
    }
    s = warp_sum(s);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < NE; ++i) p[i] *= inv;
}

// One CTA per (sequence, chunk of tokens): part[s][chunk][E] sums of p, cnt[s][chunk][E + 1] counts
// and, last, the chunk's counted tokens.
template <int NE>
__global__ void __launch_bounds__(kBalThreads) balance_partial_kernel(
    const void* __restrict__ logits, int lt, const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
    int64_t L, int chunks, int chunk_tokens, int E, int k, float* __restrict__ part, int32_t* __restrict__ cnt) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ float red[];                                  // [kBalWarps][E]
    int32_t* hist = reinterpret_cast<int32_t*>(red + kBalWarps * E);   // [E + 1]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t s = blockIdx.x / chunks, c = blockIdx.x - s * chunks;
    const int64_t t0 = s * L + c * chunk_tokens, t1 = s * L + min(L, (c + 1) * chunk_tokens);
    for (int e = threadIdx.x; e <= E; e += kBalThreads) hist[e] = 0;
    __syncthreads();
    for (int64_t i = t0 * k + threadIdx.x; i < t1 * k; i += kBalThreads) {
        const int e = __ldg(idx + i);
        if (e >= 0 && e < E && (!mask || __ldg(mask + i / k))) atomicAdd(hist + e, 1);
    }
    float acc[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) acc[i] = 0.0f;
    int n = 0;
    for (int64_t t = t0 + warp; t < t1; t += kBalWarps) {
        if (mask && !__ldg(mask + t)) continue;
        float p[NE];
        row_softmax<NE>(logits, lt, t, E, lane, p);
#pragma unroll
        for (int i = 0; i < NE; ++i) acc[i] += p[i];
        ++n;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i)
        if (lane + 32 * i < E) red[warp * E + lane + 32 * i] = acc[i];
    if (lane == 0) atomicAdd(hist + E, n);
    __syncthreads();
    float* po = part + static_cast<int64_t>(blockIdx.x) * E;
    int32_t* co = cnt + static_cast<int64_t>(blockIdx.x) * (E + 1);
    for (int e = threadIdx.x; e < E; e += kBalThreads) {
        float v = 0.0f;
        for (int w = 0; w < kBalWarps; ++w) v += red[w * E + e];
        po[e] = v;
    }
    for (int e = threadIdx.x; e <= E; e += kBalThreads) co[e] = hist[e];
}

// One CTA per sequence: the chunks in order; counts, tokens, prob and the sequence's loss.
__global__ void __launch_bounds__(kBalThreads) balance_sequence_kernel(const float* __restrict__ part,
                                                                        const int32_t* __restrict__ cnt, int chunks,
                                                                        int E, int k, int32_t* __restrict__ counts,
                                                                        float* __restrict__ prob,
                                                                        int32_t* __restrict__ tokens,
                                                                        double* __restrict__ seq_loss) {
    pdl_wait();
    pdl_trigger();
    const int64_t s = blockIdx.x;
    __shared__ double red[kBalWarps];
    int n = 0;
    for (int c = 0; c < chunks; ++c) n += cnt[(s * chunks + c) * (E + 1) + E];
    const double rn = n > 0 ? 1.0 / n : 0.0;
    double dot = 0.0;
    for (int e = threadIdx.x; e < E; e += kBalThreads) {
        double p = 0.0;
        int count = 0;
        for (int c = 0; c < chunks; ++c) {
            p += part[(s * chunks + c) * E + e];
            count += cnt[(s * chunks + c) * (E + 1) + e];
        }
        p *= rn;
        counts[s * E + e] = count;
        prob[s * E + e] = static_cast<float>(p);
        dot += p * count;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        double v = 0.0;
        for (int w = 0; w < kBalWarps; ++w) v += red[w];
        tokens[s] = n;
        seq_loss[s] = v * rn * E / k;
    }
}

// Sum over threads of one CTA, the same on every thread; `red` holds kBalWarps values.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    T t = 0;
    for (int w = 0; w < kBalWarps; ++w) t += red[w];
    return t;
}

__global__ void __launch_bounds__(kBalThreads) balance_loss_kernel(const double* __restrict__ seq_loss,
                                                                    const int32_t* __restrict__ tokens, int64_t S,
                                                                    float* __restrict__ loss) {
    pdl_wait();
    pdl_trigger();
    __shared__ double rd[kBalWarps];
    __shared__ int ri[kBalWarps];
    double v = 0.0;
    int live = 0;
    for (int64_t s = threadIdx.x; s < S; s += kBalThreads) {
        if (tokens[s] > 0) {   // a sequence without a counted token is not part of the mean
            v += seq_loss[s];
            ++live;
        }
    }
    v = block_sum(v, rd);
    live = block_sum(live, ri);
    if (threadIdx.x == 0) *loss = live > 0 ? static_cast<float>(v / live) : 0.0f;
}

// A persistent grid over (sequence, chunk): the chunk's f_e - 1/E times E / (S' n_s) times the
// incoming gradient in shared memory, then one warp per token.
template <int NE>
__global__ void __launch_bounds__(kBalThreads) balance_backward_kernel(
    const void* __restrict__ logits, int lt, const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const uint8_t* __restrict__ mask, const float* __restrict__ grad_loss, int64_t S, int64_t L, int chunks,
    int chunk_tokens, int E, int k, void* __restrict__ grad) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ float sf[];   // [E]
    __shared__ int ri[kBalWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int live = 0;
    for (int64_t s = threadIdx.x; s < S; s += kBalThreads) live += tokens[s] > 0;
    live = block_sum(live, ri);
    const double g = __ldg(grad_loss);
    for (int64_t b = blockIdx.x; b < S * chunks; b += gridDim.x) {
        const int64_t s = b / chunks, c = b - s * chunks;
        const int n = tokens[s];
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += kBalThreads) {
            // (E counts - k n) / (E k n) * g E / (S' n)
            const int64_t num = static_cast<int64_t>(E) * counts[s * E + e] - static_cast<int64_t>(k) * n;
            sf[e] = n > 0 ? static_cast<float>(g * static_cast<double>(num) /
                                               (static_cast<double>(k) * n * (static_cast<double>(live) * n)))
                          : 0.0f;
        }
        __syncthreads();
        float f[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) f[i] = lane + 32 * i < E ? sf[lane + 32 * i] : 0.0f;
        const int64_t t0 = s * L + c * chunk_tokens, t1 = s * L + min(L, (c + 1) * chunk_tokens);
        for (int64_t t = t0 + warp; t < t1; t += kBalWarps) {
            float p[NE];
            if (mask && !__ldg(mask + t)) {
#pragma unroll
                for (int i = 0; i < NE; ++i) p[i] = 0.0f;
            } else {
                row_softmax<NE>(logits, lt, t, E, lane, p);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < NE; ++i) dot += p[i] * f[i];
                dot = warp_sum(dot);
#pragma unroll
                for (int i = 0; i < NE; ++i) p[i] *= f[i] - dot;
            }
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 32 * i;
                if (e >= E) continue;
                if (lt == MOE_F32) static_cast<float*>(grad)[t * E + e] = p[i];
                else static_cast<__nv_bfloat16*>(grad)[t * E + e] = __float2bfloat16_rn(p[i]);
            }
        }
    }
}

// ------------------------------------------------------------------------------- launchers
namespace {

struct BalPlan {
    int chunk_tokens, chunks;
};

// Chunks of whole warps' tokens, about 600 of them (4 CTAs per SM), none across two sequences.
BalPlan bal_plan(int64_t S, int64_t L) {
    int64_t per = (S * L + 607) / 608;
    per = std::max<int64_t>(kBalWarps, (per + kBalWarps - 1) / kBalWarps * kBalWarps);
    per = std::min<int64_t>(per, (L + kBalWarps - 1) / kBalWarps * kBalWarps);
    return {static_cast<int>(per), static_cast<int>((L + per - 1) / per)};
}

template <typename F>
cudaError_t with_ne(int64_t E, F f) {
    if (E <= 32) return f(std::integral_constant<int, 1>{});
    if (E <= 64) return f(std::integral_constant<int, 2>{});
    if (E <= 128) return f(std::integral_constant<int, 4>{});
    if (E <= 256) return f(std::integral_constant<int, 8>{});
    if (E <= 512) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t balance_workspace_bytes(int64_t S, int64_t L, int64_t E) {
    const int64_t n = S * bal_plan(S, L).chunks;
    return align256(sizeof(float) * n * E) + align256(sizeof(int32_t) * n * (E + 1)) + align256(sizeof(double) * S);
}

cudaError_t launch_balance_loss(const void* logits, int lt, const int32_t* idx, const uint8_t* mask, int64_t S,
                                int64_t L, int64_t E, int k, float* loss, int32_t* counts, float* prob, int32_t* tokens,
                                void* workspace, cudaStream_t st) {
    const BalPlan p = bal_plan(S, L);
    const int64_t n = S * p.chunks;
    char* w = static_cast<char*>(workspace);
    float* part = reinterpret_cast<float*>(w);
    w += align256(sizeof(float) * n * E);
    int32_t* cnt = reinterpret_cast<int32_t*>(w);
    w += align256(sizeof(int32_t) * n * (E + 1));
    double* seq_loss = reinterpret_cast<double*>(w);
    const int e32 = static_cast<int>(E);
    cudaError_t e = with_ne(E, [&](auto ne) {
        return launch_pdl(balance_partial_kernel<decltype(ne)::value>, dim3(static_cast<unsigned>(n)), dim3(kBalThreads),
                          sizeof(float) * kBalWarps * E + sizeof(int32_t) * (E + 1), st, logits, lt, idx, mask, L,
                          p.chunks, p.chunk_tokens, e32, k, part, cnt);
    });
    if (e == cudaSuccess)
        e = launch_pdl(balance_sequence_kernel, dim3(static_cast<unsigned>(S)), dim3(kBalThreads), 0, st,
                       static_cast<const float*>(part), static_cast<const int32_t*>(cnt), p.chunks, e32, k, counts, prob,
                       tokens, seq_loss);
    if (e == cudaSuccess)
        e = launch_pdl(balance_loss_kernel, dim3(1), dim3(kBalThreads), 0, st, static_cast<const double*>(seq_loss),
                       static_cast<const int32_t*>(tokens), S, loss);
    return e;
}

cudaError_t launch_balance_backward(const void* logits, int lt, const int32_t* counts, const int32_t* tokens,
                                    const uint8_t* mask, const float* grad_loss, int64_t S, int64_t L, int64_t E, int k,
                                    void* grad, int num_sms, cudaStream_t st) {
    const BalPlan p = bal_plan(S, L);
    const int64_t n = std::min<int64_t>(S * p.chunks, 4ll * num_sms);
    return with_ne(E, [&](auto ne) {
        return launch_pdl(balance_backward_kernel<decltype(ne)::value>, dim3(static_cast<unsigned>(n)),
                          dim3(kBalThreads), sizeof(float) * E, st, logits, lt, counts, tokens, mask, grad_loss, S, L,
                          p.chunks, p.chunk_tokens, static_cast<int>(E), k, grad);
    });
}

}  // namespace moe
