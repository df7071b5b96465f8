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
// One wave of CTAs (of the largest batches' forward pass several), each with an equal run of the batch's tokens,
// whatever the sequences' length (chunks of one sequence left up to a third of the SMs idle in the last wave: 16 x
// 4096 x 512 fp32 forward 43 us).
// No floating-point atomics: every part of a run that lies in one sequence writes a record of partial sums,
// and the records of a sequence are added in order.
//
// Both directions read the logits once and are bound by that (backward also by writing the gradient).
// A row is held by kLanes lanes, 4 consecutive experts at a time, so that loads are 16 (bf16: 8) bytes
// a lane and a warp takes up to 16 rows of a small router at once.  The next row's logits and expert
// indices are read before this row's softmax, and the mask of the row after it, so that no read waits for
// another.
// Measured (GB300), 16 sequences of 4096 tokens, 512 experts, top-22, fp32: forward 35.0 us (134 MB read), backward
// 46.7 us (134 MB read and 134 MB written, 5.7 TB/s); 7 x 1021 tokens, 128 experts, bf16: 12.1 and 6.4 us, latency;
// 65536 x 128 bf16 17.4 and 16.5, 32768 x 256 fp32 17.4 and 15.9 us, much of the forward's in its reduction kernel.
#include <algorithm>

#include "common.cuh"

namespace moe {

constexpr int kBalThreads = 256, kBalWarps = kBalThreads / 32;

// The runs: CTA b of n has tokens [start(b), start(b + 1)), multiples of 8 up to the end.  Run b's part of
// sequence s is record b + s: both grow along the tokens, one at a time.  (T is at most 2^20 and n below 4096:
// 32 bits hold the products.)
struct BalRuns {
    int T, n;
    __host__ __device__ int start(int b) const {
        const int t = (T + 7) / 8 * b / n * 8;
        return t < T ? t : T;
    }
    // the last run that starts at or before token t < T
    __device__ int run_of(int t) const {
        int b = t / 8 * n / ((T + 7) / 8);   // start(b) <= t, and the answer is at most a step away
        while (b + 1 < n && start(b + 1) <= t) ++b;
        return b;
    }
};

// a, b -> exp(a - m), exp(b - m), m at least both.  With d = a - m and t = d log2 e rounded, exp(d) = 2^t exp(d - t ln 2),
// and q = d - t ln 2, exact up to 2^-24 of itself through ln 2 in two parts, is so small that exp(q) = 1 + q to 2^-33:
// the result is as good as the hardware's 2^t (2^-22 of it) at any distance, where 2^t alone is off by
// up to |d| 2^-24 more (at -80 by 20 times as much).  Below 2^-126 it is 0.  Pairs go in packed instructions:
// 16 x 4096 x 512 fp32 forward 35.1 us, with expf 38.1, with 2^t alone 33.9.
__device__ __forceinline__ void bal_exp(float& a, float& b, float m) {
    constexpr float kLog2e = 1.44269504f, kLn2Hi = 0.693145752f, kLn2Lo = 1.42860677e-6f;   // (hi has 16 bits)
    const uint64_t d = add_f32x2(pack_f32x2(a, b), pack_f32x2(-m, -m));
    uint64_t t, q = d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(d), "l"(pack_f32x2(kLog2e, kLog2e)));
    fma_f32x2(q, t, pack_f32x2(-kLn2Hi, -kLn2Hi));
    fma_f32x2(q, t, pack_f32x2(-kLn2Lo, -kLn2Lo));
    const float2 tf = unpack_f32x2(t), qf = unpack_f32x2(q);
    float ea, eb;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ea) : "f"(tf.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(eb) : "f"(tf.y));
    // (where t is -inf e is 0 and q +inf or, for d = -inf, NaN; a NaN logit is NaN in e)
    uint64_t e = pack_f32x2(ea, eb);
    fma_f32x2(e, pack_f32x2(ea, eb), pack_f32x2(fminf(qf.x, 1.0f), fminf(qf.y, 1.0f)));
    const float2 r = unpack_f32x2(e);
    a = r.x, b = r.y;
}

// How a warp holds rows of E logits.  Vector form (E a multiple of 4): element i of lane l of a group of
// LANES is expert 4 (l + LANES (i / 4)) + i % 4.  Scalar form: expert l + 32 i.
template <int LANES, int N, bool VEC>
struct BalRow {
    static constexpr int kLanes = LANES, kN = N, kGroups = 32 / LANES;
    static_assert(VEC ? N % 4 == 0 : LANES == 32, "forms");
    static __device__ __forceinline__ int expert(int l, int i) { return VEC ? 4 * (l + LANES * (i / 4)) + i % 4 : l + 32 * i; }

    // Logits of row t, -inf past E (E is a multiple of 4 in the vector form: a quad is in or out).
    static __device__ __forceinline__ void load(const void* x, int lt, int64_t t, int E, int l, float v[N]) {
        if (VEC) {
#pragma unroll
            for (int q = 0; q < N / 4; ++q) {
                const int e = expert(l, 4 * q);
                float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (e < E) {
                    if (lt == MOE_F32) {
                        f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(x) + t * E + e));
                    } else {
                        const uint2 b = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x) + t * E + e));
                        f = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                                        __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
                    }
                }
                v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = expert(l, i) < E ? load_x(x, lt, t * E + expert(l, i)) : -INFINITY;
        }
    }
    static __device__ __forceinline__ void store(void* g, int lt, int64_t t, int E, int l, const float v[N]) {
#pragma unroll
        for (int i = 0; i < N; i += VEC ? 4 : 1) {
            const int e = expert(l, i);
            if (e >= E) continue;
            if (lt == MOE_F32) {
                float* o = static_cast<float*>(g) + t * E + e;
                if (VEC) *reinterpret_cast<float4*>(o) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                else *o = v[i];
            } else {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(g) + t * E + e;
                if (VEC) {
                    const __nv_bfloat162 a = __floats2bfloat162_rn(v[i], v[i + 1]), b = __floats2bfloat162_rn(v[i + 2], v[i + 3]);
                    *reinterpret_cast<uint2*>(o) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
                } else {
                    *o = __float2bfloat16_rn(v[i]);
                }
            }
        }
    }
    // Over the group's lanes; every lane of the warp takes part.
    static __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int o = LANES / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    // Logits -> probabilities.  A row of -inf has no probability at all (p = 0); a NaN or +inf logit makes the row
    // NaN.
    static __device__ __forceinline__ void softmax(float v[N]) {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
#pragma unroll
        for (int o = LANES / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (m == -INFINITY) m = 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            bal_exp(v[i], v[i + 1], m);
            s += v[i];
            s += v[i + 1];
        }
        s = sum(s);
        const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= inv;
    }
};

// A running sum with the part that its additions rounded off beside it (two-sum: the rounding error of an
// addition, exact), so that it holds about 48 bits however many terms come.  (Not fp64: GB300 adds that at a
// small fraction of fp32's rate.)
struct BalSum {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)));
        hi = s;
    }
    __device__ __forceinline__ float value() const { return hi + lo; }
};

// Sum over threads of one CTA, the same on every thread; `red` holds kBalWarps values.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    T t = 0;
#pragma unroll
    for (int w = 0; w < kBalWarps; ++w) t += red[w];
    return t;
}

// CTAs that share an SM, by the registers that N logits of a lane take.
constexpr int bal_ctas_forward(int n) { return n <= 8 ? 4 : (n <= 16 ? 3 : 1); }
constexpr int bal_ctas_backward(int n) { return n <= 8 ? 4 : (n <= 16 ? 2 : 1); }

// What the forward pass writes.
struct BalOut {
    float* loss;
    int32_t* counts;
    float* prob;
    int32_t* tokens;
};

// 1 / n for a mean over n terms, 0 over none: formed before the sums that it meets are there.
__device__ __forceinline__ float bal_inverse(int n) { return n > 0 ? 1.0f / static_cast<float>(n) : 0.0f; }
// Pairwise sum of the warps' parts.
template <typename T>
__device__ __forceinline__ T warp_parts(T a[kBalWarps]) {
#pragma unroll
    for (int h = kBalWarps / 2; h >= 1; h >>= 1)
#pragma unroll
        for (int w = 0; w < h; ++w) a[w] += a[w + h];
    return a[0];
}

// One CTA per run.  A record is part[E], the sums of p, and cnt[E + 1], the experts' counts and, last, the
// counted tokens.  A single run has every sequence in one record, and its CTA writes the results itself (16
// tokens of 8 experts: one launch and no workspace, 2.3 us in place of 5.2).
template <typename Row>
__global__ void __launch_bounds__(kBalThreads, bal_ctas_forward(Row::kN)) balance_partial_kernel(
    const void* __restrict__ logits, int lt, const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
    int L, BalRuns runs, int E, int k, float* __restrict__ part, int32_t* __restrict__ cnt,
    uint32_t* __restrict__ done, BalOut out) {
    pdl_wait();
    constexpr int N = Row::kN;
    extern __shared__ float red[];                                     // [kBalWarps][E]
    int32_t* hist = reinterpret_cast<int32_t*>(red + kBalWarps * E);   // [E + 1]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % Row::kLanes, grp = lane / Row::kLanes;
    __shared__ float rd[kBalWarps];
    if (runs.n > 1 && blockIdx.x == 0 && threadIdx.x == 0) *done = 0;   // the next kernel's counter
    BalSum loss;
    int live_seq = 0;
    constexpr int kStep = kBalWarps * Row::kGroups;
    const int end = runs.start(blockIdx.x + 1);
    for (int t0 = runs.start(blockIdx.x); t0 < end;) {   // the run's part of one sequence
        const int s = t0 / L, t1 = min(end, (s + 1) * L);
        for (int e = threadIdx.x; e <= E; e += kBalThreads) hist[e] = 0;
        __syncthreads();
        float acc[N], v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = v[i] = 0.0f;
        int n = 0;
        int t = t0 + warp * Row::kGroups + grp;
        auto counted = [&](int u) -> bool { return u < t1 && (!mask || __ldg(mask + u)); };
        int e_next = -1;   // this lane's first index of the next row
        auto load = [&](int u) {
            Row::load(logits, lt, u, E, l, v);
            if (l < k) e_next = __ldg(idx + static_cast<int64_t>(u) * k + l);
        };
        bool live = counted(t), live2 = counted(t + kStep);
        if (live) load(t);
        for (int tw = t0 + warp * Row::kGroups; tw < t1; tw += kStep, t += kStep) {
            const bool now = live;
            const int e = e_next;
            float p[N];
#pragma unroll
            for (int i = 0; i < N; ++i) p[i] = v[i];
            live = live2;
            live2 = counted(t + 2 * kStep);
            if (live) load(t + kStep);
            if (now) {
                if (e >= 0 && e < E) atomicAdd(hist + e, 1);   // (-1 on lanes without an index)
                for (int j = l + Row::kLanes; j < k; j += Row::kLanes) {
                    const int e2 = __ldg(idx + static_cast<int64_t>(t) * k + j);
                    if (e2 >= 0 && e2 < E) atomicAdd(hist + e2, 1);
                }
                n += l == 0;
            }
            Row::softmax(p);
            if (now) {
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] += p[i];
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int o = Row::kLanes; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
            if (grp == 0 && Row::expert(l, i) < E) red[warp * E + Row::expert(l, i)] = acc[i];
        }
        if (n) atomicAdd(hist + E, n);
        __syncthreads();
        const int64_t rec = static_cast<int64_t>(blockIdx.x) + s;
        const bool only = runs.n == 1;
        const int tokens = hist[E];
        const float rn = bal_inverse(tokens), factor = rn * (static_cast<float>(E) / static_cast<float>(k));
        float dot = 0.0f;
        for (int e = threadIdx.x; e < E; e += kBalThreads) {
            float a[kBalWarps];
#pragma unroll
            for (int w = 0; w < kBalWarps; ++w) a[w] = red[w * E + e];
            const float total = warp_parts(a);
            if (only) {
                const float mean = total * rn;
                out.prob[rec * E + e] = mean;
                out.counts[rec * E + e] = hist[e];
                dot += mean * static_cast<float>(hist[e]);
            } else {
                part[rec * E + e] = total;
            }
        }
        if (only) {
            dot = block_sum(dot, rd);
            if (threadIdx.x == 0) out.tokens[s] = tokens;
            loss.add(dot * factor);
            live_seq += tokens > 0;
        } else {
            for (int e = threadIdx.x; e <= E; e += kBalThreads) cnt[rec * (E + 1) + e] = hist[e];
        }
        __syncthreads();
        t0 = t1;
    }
    if (runs.n == 1 && threadIdx.x == 0) *out.loss = live_seq > 0 ? loss.value() / static_cast<float>(live_seq) : 0.0f;
}

// One CTA per (sequence, 32 experts): warp w adds the sequence's records w, w + 8, ..; counts, tokens, prob and the
// block's part of the sequence's loss.  The last CTA adds those up, in order.
__global__ void __launch_bounds__(kBalThreads) balance_sequence_kernel(
    const float* __restrict__ part, const int32_t* __restrict__ cnt, int S, int L, BalRuns runs, int E, int k,
    int32_t* __restrict__ counts, float* __restrict__ prob, int32_t* tokens, float* seq_loss, uint32_t* done,
    float* __restrict__ loss) {
    pdl_wait();
    __shared__ float sp[kBalWarps][32], rd[kBalWarps];
    __shared__ int sc[kBalWarps][33], ri[kBalWarps];
    __shared__ bool last;
    const int blocks = (E + 31) / 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t s = blockIdx.x / blocks;
    const int e = (blockIdx.x % blocks) * 32 + lane;
    const int b0 = runs.run_of(static_cast<int>(s) * L);
    const int chunks = runs.run_of(static_cast<int>(s + 1) * L - 1) - b0 + 1;
    const float* ps = part + (b0 + s) * E + e;
    const int32_t* cs = cnt + (b0 + s) * (E + 1);
    BalSum sum;
    int count = 0, n = 0;
#pragma unroll 4
    for (int c = warp; c < chunks; c += kBalWarps) {
        if (e < E) {
            sum.add(__ldcg(ps + static_cast<int64_t>(c) * E));
            count += __ldcg(cs + static_cast<int64_t>(c) * (E + 1) + e);
        }
        n += lane == 0 ? __ldcg(cs + static_cast<int64_t>(c) * (E + 1) + E) : 0;
    }
    sp[warp][lane] = sum.value();
    sc[warp][lane] = count;
    if (lane == 0) sc[warp][32] = n;
    __syncthreads();
    if (warp == 0) {
        int ns[kBalWarps], cs8[kBalWarps];
        float ps8[kBalWarps];
#pragma unroll
        for (int w = 0; w < kBalWarps; ++w) ns[w] = sc[w][32], cs8[w] = sc[w][lane], ps8[w] = sp[w][lane];
        n = warp_parts(ns);
        count = warp_parts(cs8);
        const float rn = bal_inverse(n), p = warp_parts(ps8) * rn;
        float dot = e < E ? p * static_cast<float>(count) : 0.0f;
        if (e < E) {
            counts[s * E + e] = count;
            prob[s * E + e] = p;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) {
            if (e < 32) tokens[s] = n;
            seq_loss[blockIdx.x] = dot * (rn * (static_cast<float>(E) / static_cast<float>(k)));
            __threadfence();
            last = atomicAdd(done, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    BalSum v;   // (a thread adds 2^17 blocks at most)
    int live = 0;
    for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kBalThreads) v.add(__ldcg(seq_loss + i));   // 0 where n_s = 0
    for (int i = threadIdx.x; i < S; i += kBalThreads) live += __ldcg(tokens + i) > 0;
    const float total = block_sum(v.value(), rd);
    live = block_sum(live, ri);
    if (threadIdx.x == 0) *loss = live > 0 ? total / static_cast<float>(live) : 0.0f;
}

// One CTA per run: per sequence f_e - 1/E times E / (S' n_s) times the incoming gradient in registers, then
// the rows.
template <typename Row>
__global__ void __launch_bounds__(kBalThreads, bal_ctas_backward(Row::kN)) balance_backward_kernel(
    const void* __restrict__ logits, int lt, const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const uint8_t* __restrict__ mask, const float* __restrict__ grad_loss, int S, int L, BalRuns runs, int E,
    int k, void* __restrict__ grad) {
    pdl_wait();
    constexpr int N = Row::kN;
    __shared__ int ri[kBalWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % Row::kLanes, grp = lane / Row::kLanes;
    const float g = __ldg(grad_loss);
    constexpr int kStep = kBalWarps * Row::kGroups;
    const int64_t end = runs.start(blockIdx.x + 1);
    int live_seq = -1;
    for (int64_t t0 = runs.start(blockIdx.x); t0 < end;) {   // the run's part of one sequence
        const int64_t s = t0 / L, t1 = min(end, (s + 1) * L);
        float v[N], f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
        int t = t0 + warp * Row::kGroups + grp;
        auto counted = [&](int u) -> bool { return u < t1 && (!mask || __ldg(mask + u)); };
        bool live = counted(t), live2 = counted(t + kStep);
        if (live) Row::load(logits, lt, t, E, l, v);
        if (live_seq < 0) {   // (behind the first row's loads)
            int c = 0;
            for (int i = threadIdx.x; i < S; i += kBalThreads) c += __ldg(tokens + i) > 0;
            live_seq = block_sum(c, ri);
        }
        // (E counts - k n) / (E k n) * g E / (S' n), the difference and the divisor (2^45 at most) in integers: four
        // fp32 roundings in all
        const int n = __ldg(tokens + s);
        const int64_t kn = static_cast<int64_t>(k) * n;
        const float scale = n > 0 ? g / static_cast<float>(kn * (static_cast<int64_t>(live_seq) * n)) : 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = Row::expert(l, i);
            f[i] = e < E ? scale * static_cast<float>(static_cast<int64_t>(E) * __ldg(counts + static_cast<int64_t>(s) * E + e) - kn) : 0.0f;
        }
        for (int tw = t0 + warp * Row::kGroups; tw < t1; tw += kStep, t += kStep) {
            const bool now = live;
            float p[N];
#pragma unroll
            for (int i = 0; i < N; ++i) p[i] = v[i];
            live = live2;
            live2 = counted(t + 2 * kStep);
            if (live) Row::load(logits, lt, t + kStep, E, l, v);
            Row::softmax(p);
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) dot += p[i] * f[i];
            dot = Row::sum(dot);
#pragma unroll
            for (int i = 0; i < N; ++i) p[i] = now ? p[i] * (f[i] - dot) : 0.0f;
            if (t < t1) Row::store(grad, lt, t, E, l, p);
        }
        t0 = t1;
    }
}

// ------------------------------------------------------------------------------- launchers
namespace {

constexpr int64_t kBalSms = 152;   // the runs depend on the shapes alone, and so does the workspace

// At least `passes` of a CTA's passes (8 warps of `groups` rows) to a run: shorter runs are all latency, and each
// is a record that the next kernel has to add (65536 x 8 forward 12.9 us with one pass, 10.5 with 2, 8.6 with 4; 7147 x
// 128: 12.3, 10.7, 11.2; backward 6.4, 6.0, 7.0).
BalRuns bal_runs(int64_t T, int ctas_per_sm, int groups, int passes) {
    const int64_t rows = static_cast<int64_t>(passes) * kBalWarps * groups;
    return {static_cast<int>(T), static_cast<int>(std::min<int64_t>((T + rows - 1) / rows, kBalSms * ctas_per_sm))};
}

// Two rows a warp up to 256 experts: half the shuffles a row and two chains at once (65536 x 128 bf16, us: forward
// 23.6 -> 19.7, backward 16.6 -> 13.8; 32768 x 256 fp32: forward 20.1 -> 16.5).  Ten values a lane in place of 16 up to
// 320 experts: 32768 x 257 fp32 forward 26.4 -> 23.4, backward 20.0 -> 18.1; 65536 x 319 32.8 -> 27.6, 36.8 -> 35.3.
template <typename F>
cudaError_t with_row(int64_t E, F f) {
    if (E % 4 == 0) {
        if (E <= 8) return f(BalRow<2, 4, true>{});
        if (E <= 16) return f(BalRow<4, 4, true>{});
        if (E <= 32) return f(BalRow<8, 4, true>{});
        if (E <= 64) return f(BalRow<8, 8, true>{});
        if (E <= 128) return f(BalRow<16, 8, true>{});
        if (E <= 256) return f(BalRow<16, 16, true>{});
        if (E <= 512) return f(BalRow<32, 16, true>{});
        return f(BalRow<32, 32, true>{});
    }
    if (E <= 64) return f(BalRow<32, 2, false>{});
    if (E <= 128) return f(BalRow<32, 4, false>{});
    if (E <= 256) return f(BalRow<32, 8, false>{});
    if (E <= 320) return f(BalRow<32, 10, false>{});
    if (E <= 512) return f(BalRow<32, 16, false>{});
    return f(BalRow<32, 32, false>{});
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }
int64_t expert_blocks(int64_t E) { return (E + 31) / 32; }

}  // namespace

// The forward pass's runs.  A lane adds its rows of a run in turn, and a sequential fp32 sum of n like terms may be off
// by n / 2 units of 2^-24: a run has at most 64 passes, which takes more than one wave of them from 77824 tokens (E
// above 512; 233472 above 256) on.
constexpr int64_t kBalMaxPasses = 64;
static BalRuns bal_runs_forward(int64_t T, int64_t E) {
    BalRuns runs{};
    (void)with_row(E, [&](auto row) {
        using Row = decltype(row);
        runs = bal_runs(T, bal_ctas_forward(Row::kN), Row::kGroups, 4);
        const int64_t wave = kBalSms * bal_ctas_forward(Row::kN) * kBalMaxPasses * kBalWarps * Row::kGroups;
        if (T > wave) runs.n *= static_cast<int>((T + wave - 1) / wave);
        return cudaSuccess;
    });
    return runs;
}

size_t balance_workspace_bytes(int64_t S, int64_t L, int64_t E) {
    if (bal_runs_forward(S * L, E).n == 1) return 0;   // no records
    const int64_t n = bal_runs_forward(S * L, E).n + S;   // records, at most
    return 256 + align256(sizeof(float) * n * E) + align256(sizeof(int32_t) * n * (E + 1)) +
           align256(sizeof(float) * S * expert_blocks(E));
}

cudaError_t launch_balance_loss(const void* logits, int lt, const int32_t* idx, const uint8_t* mask, int64_t S,
                                int64_t L, int64_t E, int k, float* loss, int32_t* counts, float* prob, int32_t* tokens,
                                void* workspace, cudaStream_t st) {
    const BalRuns runs = bal_runs_forward(S * L, E);
    const int64_t n = runs.n + S;
    char* w = static_cast<char*>(workspace);
    uint32_t* done = reinterpret_cast<uint32_t*>(w);
    w += 256;
    float* part = reinterpret_cast<float*>(w);
    w += align256(sizeof(float) * n * E);
    int32_t* cnt = reinterpret_cast<int32_t*>(w);
    w += align256(sizeof(int32_t) * n * (E + 1));
    float* seq_loss = reinterpret_cast<float*>(w);
    const int e32 = static_cast<int>(E);
    cudaError_t e = with_row(E, [&](auto row) {
        return launch_pdl(balance_partial_kernel<decltype(row)>, dim3(static_cast<unsigned>(runs.n)), dim3(kBalThreads),
                          sizeof(float) * kBalWarps * E + sizeof(int32_t) * (E + 1), st, logits, lt, idx, mask,
                          static_cast<int>(L), runs, e32, k, part, cnt, done, BalOut{loss, counts, prob, tokens});
    });
    if (e != cudaSuccess || runs.n == 1) return e;
    return launch_pdl(balance_sequence_kernel, dim3(static_cast<unsigned>(S * expert_blocks(E))), dim3(kBalThreads), 0, st,
                      static_cast<const float*>(part), static_cast<const int32_t*>(cnt), static_cast<int>(S),
                      static_cast<int>(L), runs, e32, k, counts, prob,
                      tokens, seq_loss, done, loss);
}

cudaError_t launch_balance_backward(const void* logits, int lt, const int32_t* counts, const int32_t* tokens,
                                    const uint8_t* mask, const float* grad_loss, int64_t S, int64_t L, int64_t E, int k,
                                    void* grad, cudaStream_t st) {
    return with_row(E, [&](auto row) {
        const BalRuns runs = bal_runs(S * L, bal_ctas_backward(decltype(row)::kN), decltype(row)::kGroups, 2);
        return launch_pdl(balance_backward_kernel<decltype(row)>, dim3(static_cast<unsigned>(runs.n)), dim3(kBalThreads), 0,
                          st, logits, lt, counts, tokens, mask, grad_loss, static_cast<int>(S), static_cast<int>(L), runs,
                          static_cast<int>(E), k, grad);
    });
}

}  // namespace moe
