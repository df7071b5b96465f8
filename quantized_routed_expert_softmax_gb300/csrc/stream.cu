// stream.cu -- the experts' products for a few rows an expert (decoding): weights straight from memory into mma.sync
// fragments, for int8 rows and weights (moe_int8_matmul) and for bf16 (moe_ffn_forward).
//
// With a few rows the weights' bytes bound a product, and what counts is that every SM has enough loads on their way, from
// the first moment on.  An item is 16 weight rows (SwiGLU: 8 gate rows and the same neurons' 8 up rows, so that a lane's
// fragment holds both) by all of K, for up to 8 rows of one expert; one to sixteen warps share its K in slices of 32 columns,
// as many as it takes to fill the SMs.  A lane loads 8 consecutive columns of rows lane / 4 and + 8: as fragments of two
// m16n8k16 MMAs that is another order of the columns, the same for weights and rows, so nothing is moved between lanes, and
// the loads of a warp are whole sectors.
//
// int8: codes become f16 on the way (exact; see int8_gemm.cu).  Sums of up to 1024 columns are exact in the MMA's fp32; they
// go to 32-bit integers, which hold the whole sum exactly (127^2 * 65536 < 2^31).
#include <algorithm>

#include "int8.cuh"

namespace moe {

// What a product reads and writes (one of the two forms).
struct StreamArgs {
    const uint8_t *x, *w;       // codes or values of row 0 (of matrix 0)
    const float *sx, *sw;       // int8: scales of the rows, of matrix 0's channels
    int64_t w_mat;              // bytes between matrices
    const int32_t* offsets;
    int E, P, N, K;
    int split;                  // warps that share an item's K
    void* out;                  // [P][N], SwiGLU [P][N / 2]
    float* z_out;               // bf16: z [P][N], or null
    int f32;                    // out is fp32
};

template <bool I8>
__device__ __forceinline__ void stream_mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    if constexpr (I8)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 columns of a row: int8 8 bytes, bf16 16 bytes.  Weights pass L1 by, as nothing reads them again.
template <bool I8, bool STREAM>
__device__ __forceinline__ void stream_load(const uint8_t* p, bool in, uint32_t* v) {
#pragma unroll
    for (int i = 0; i < (I8 ? 2 : 4); ++i) v[i] = 0;
    if (!in) return;
    if constexpr (I8) {
        if constexpr (STREAM) asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p));
        else asm volatile("ld.global.nc.v2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p));
    } else {
        if constexpr (STREAM)
            asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "l"(p));
        else asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "l"(p));
    }
}

// 8 columns -> four pairs of 16-bit values.
template <bool I8>
__device__ __forceinline__ void stream_pairs(const uint32_t* v, uint32_t* h) {
    if constexpr (I8) {
        i8_f16(v[0], h);
        i8_f16(v[1], h + 2);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = v[i];
    }
}

// Blocks of four warps or of `split`; registers for 24 warps an SM.  (us, 8 rows of 8 experts, 2816 -> 2 x 704: six slices ahead
// 9.4, four of 64 registers 10.2, eight of 96 9.7, of 80 11.5.  bf16 block, 2816 and 704: three 19.5, four of 96 registers 22.7,
// six of 128 21.7, two of 64 21.2.)
template <bool I8, int ACT>
__global__ void __maxnreg__(80) stream_kernel(const StreamArgs g) {
    constexpr bool kGated = ACT == MOE_ACT_SWIGLU;
    constexpr int kWords = I8 ? 2 : 4, kElem = I8 ? 1 : 2;
    constexpr int kAhead = I8 ? 6 : 3;    // slices that a warp has on their way
    __shared__ uint32_t part[16][4][32];
    __shared__ int owner;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
    const int split = g.split, sub = warp & (split - 1), lead = warp - sub;   // this warp's share; the first warp of its item
    const int r0 = blockIdx.y;   // a block works if a group of 8 rows of an expert begins with its row
    if (tid == 0) owner = g.E;
    __syncthreads();
    pdl_wait();   // (no early trigger: the next kernel's blocks would take places unevenly, 8 rows of 8 experts 11.3 -> 12.1 us)
    for (int e = tid; e < g.E; e += blockDim.x) {
        int first, last;
        expert_rows(g.offsets, e, g.P, &first, &last);
        if (first <= r0 && r0 < last) atomicMin(&owner, e);
    }
    __syncthreads();
    const int e = owner;
    if (e >= g.E) return;
    int first, last;
    expert_rows(g.offsets, e, g.P, &first, &last);
    if ((r0 - first) % 8 != 0) return;
    const int rows = min(8, last - r0);
    const int width = kGated ? g.N / 2 : g.N, per = kGated ? 8 : 16;   // columns of the result an item
    const int items = (width + per - 1) / per, slices = (g.K + 31) / 32;
    const int64_t pitch = I8 ? 32 : static_cast<int64_t>(g.K) * 2;                // to the next row
    const int64_t step_w = I8 ? 32ll * g.N : 64, step_x = I8 ? 32ll * g.P : 64;   // to the next slice
    const uint8_t* w = g.w + e * g.w_mat + 8 * t * kElem;
    const uint8_t* x = g.x + (r0 + min(gr, rows - 1)) * pitch + 8 * t * kElem;
    const int abreast = (blockDim.x >> 5) / split;   // items that the block has at a time
    // (all warps of a block make the same rounds: those past the last item work on it again and store nothing)
    for (int item0 = blockIdx.x * abreast; item0 < items; item0 += gridDim.x * abreast) {
        const int item = item0 + lead / split, c0 = item * per;
        // this lane's two weight rows (past the end: the last one, not stored)
        const int ra = min(c0 + gr, width - 1), rb = kGated ? width + ra : min(c0 + gr + 8, width - 1);
        const uint8_t *wa = w + ra * pitch, *wb = w + rb * pitch;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        [[maybe_unused]] int tot[4] = {0, 0, 0, 0};
        int since = 0;   // slices since the sums went to integers
        for (int s0 = sub; s0 < slices; s0 += split * kAhead) {
            uint32_t a[kAhead][2][kWords], b[kAhead][kWords];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int s = s0 + u * split;
                const bool in = s < slices && (I8 || 32 * s + 8 * t < g.K);   // (bf16: K may end with half a slice)
                stream_load<I8, true>(wa + s * step_w, in, a[u][0]);
                stream_load<I8, true>(wb + s * step_w, in, a[u][1]);
                stream_load<I8, false>(x + s * step_x, in && gr < rows, b[u]);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                uint32_t ha[4], hb[4], hx[4];
                stream_pairs<I8>(a[u][0], ha);
                stream_pairs<I8>(a[u][1], hb);
                stream_pairs<I8>(b[u], hx);
                const uint32_t m0[4] = {ha[0], hb[0], ha[1], hb[1]}, m1[4] = {ha[2], hb[2], ha[3], hb[3]};
                stream_mma<I8>(acc, m0, hx[0], hx[1]);
                stream_mma<I8>(acc, m1, hx[2], hx[3]);
            }
            if constexpr (I8) {
                since += kAhead;
                if (since + kAhead > 32) {   // 32 slices are 1024 columns
#pragma unroll
                    for (int i = 0; i < 4; ++i) tot[i] += __float2int_rn(acc[i]), acc[i] = 0.0f;
                    since = 0;
                }
            }
        }
        float z[4];
        int zi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z[i] = acc[i];
            zi[i] = I8 ? tot[i] + __float2int_rn(acc[i]) : 0;
        }
        if (split > 1) {   // the item's first warp adds the others' parts, in order
            if (sub > 0)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[warp][i][lane] = I8 ? static_cast<uint32_t>(zi[i]) : __float_as_uint(z[i]);
            __syncthreads();
            if (sub == 0)
                for (int v = 1; v < split; ++v)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t p = part[warp + v][i][lane];
                        if (I8) zi[i] += static_cast<int>(p);
                        else z[i] += __uint_as_float(p);
                    }
            __syncthreads();   // (the parts are free again)
        }
        if (sub > 0 || item >= items) continue;
        if constexpr (I8) {
            const float* sw = reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(g.sw) + e * g.w_mat);
            const float swa = __ldg(sw + ra), swb = __ldg(sw + rb);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                z[i] = i8_scaled(static_cast<float>(zi[i]), __ldg(g.sx + r0 + min(2 * t + (i & 1), rows - 1)), i < 2 ? swa : swb);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // rows 2 t, 2 t + 1
            const int r = 2 * t + i;
            if (r >= rows) continue;
            const int64_t row = r0 + r;
            float v[2] = {z[i], z[2 + i]};   // columns c0 + gr and, SwiGLU: its up value, else: c0 + gr + 8
            const int c[2] = {c0 + gr, c0 + gr + 8};
            if (!I8 && ACT != MOE_ACT_NONE && g.z_out) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (c[kGated ? 0 : u] < width)
                        g.z_out[row * g.N + (kGated ? u * width + c[0] : c[u])] = v[u];
            }
            if (kGated) v[0] = silu_fast(v[0]) * v[1];
#pragma unroll
            for (int u = 0; u < (kGated ? 1 : 2); ++u) {
                if (ACT == MOE_ACT_RELU2) v[u] = relu_nan(v[u]) * relu_nan(v[u]);
                if (c[u] >= width) continue;
                if (g.f32) static_cast<float*>(g.out)[row * width + c[u]] = v[u];
                else static_cast<__nv_bfloat16*>(g.out)[row * width + c[u]] = __float2bfloat16_rn(v[u]);
            }
        }
    }
}

namespace {

template <bool I8, int ACT>
cudaError_t stream_launch(StreamArgs& g, int num_sms, cudaStream_t s) {
    const int width = ACT == MOE_ACT_SWIGLU ? g.N / 2 : g.N, per = ACT == MOE_ACT_SWIGLU ? 8 : 16;
    const int items = (width + per - 1) / per, slices = (g.K + 31) / 32;
    // Warps that share an item: as many as leave a warp four slices at least, until the SMs have 10 warps each (6: 12.0 us for 8 rows of 8 experts, 2816 -> 2 x 704, 40: 15.8, 10 to 28: 10.5 to 10.8).
    const int64_t groups = g.E == 1 ? (g.P + 7) / 8 : std::min(g.E, g.P);
    g.split = 1;
    // (half as many for bf16, whose warps take more registers: two blocks of the largest split have to fit an SM)
    while (g.split < (I8 ? 16 : 8) && items * groups * g.split < 10ll * num_sms && slices >= 8 * g.split) g.split *= 2;
    const int warps = std::max(4, g.split), abreast = warps / g.split;
    // Blocks enough for two waves at most, where the items need so many; longer rounds where they need more.
    const int64_t most = std::max<int64_t>(1, 48ll * num_sms / warps / std::max<int64_t>(1, groups));
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((items + abreast - 1) / abreast, most)), static_cast<unsigned>(g.P));
    return launch_pdl(stream_kernel<I8, ACT>, grid, dim3(32 * warps), 0, s, g);
}

template <bool I8>
cudaError_t stream_launch(StreamArgs& g, int act, int num_sms, cudaStream_t s) {
    if (act == MOE_ACT_SWIGLU) return stream_launch<I8, MOE_ACT_SWIGLU>(g, num_sms, s);
    if (act == MOE_ACT_RELU2) return stream_launch<I8, MOE_ACT_RELU2>(g, num_sms, s);
    return stream_launch<I8, MOE_ACT_NONE>(g, num_sms, s);
}

}  // namespace

cudaError_t launch_stream_int8(const void* xq, int64_t P, const void* wq, int64_t E, int64_t N, int64_t K, const int32_t* offsets,
                               int act, void* out, int ot, int num_sms, cudaStream_t s) {
    StreamArgs g{};
    g.sx = static_cast<const float*>(xq);
    g.sw = static_cast<const float*>(wq);
    g.x = static_cast<const uint8_t*>(xq) + i8_scale_bytes(P);
    g.w = static_cast<const uint8_t*>(wq) + i8_scale_bytes(N);
    g.w_mat = i8_bytes(N, K);
    g.offsets = offsets;
    g.E = static_cast<int>(E), g.P = static_cast<int>(P), g.N = static_cast<int>(N), g.K = static_cast<int>(K);
    g.out = out;
    g.f32 = ot == MOE_F32;
    return stream_launch<true>(g, act, num_sms, s);
}

cudaError_t launch_stream_bf16(const uint16_t* x, int64_t P, const uint16_t* w, int64_t E, int64_t N, int64_t K, const int32_t* offsets,
                               int act, uint16_t* out, float* z, int num_sms, cudaStream_t s) {
    StreamArgs g{};
    g.x = reinterpret_cast<const uint8_t*>(x);
    g.w = reinterpret_cast<const uint8_t*>(w);
    g.w_mat = 2 * N * K;
    g.offsets = offsets;
    g.E = static_cast<int>(E), g.P = static_cast<int>(P), g.N = static_cast<int>(N), g.K = static_cast<int>(K);
    g.out = out;
    g.z_out = z;
    return stream_launch<false>(g, act, num_sms, s);
}

}  // namespace moe
