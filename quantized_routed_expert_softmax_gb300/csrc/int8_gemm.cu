// int8_gemm.cu -- the expert-indexed product of int8 rows with per-channel int8 weights:
//   z[r][n] = sx[r] sw[n] * sum_i qx[r][i] qw[n][i]
//
// GB300's tensor cores take 8-bit integers at a small fraction of their f16 rate, so the codes, which f16 holds exactly, go
// through f16 MMAs (tcgen05 cta_group::2) with fp32 accumulators.  A product of two codes is at most 127^2, so the sum of
// 1024 columns is below 2^24 and exact; longer sums are cut into segments of 1024 whose exact sums are added in fp32, in the
// epilogue's registers.
//
// Weights are the MMA's M (256 a pair of CTAs), an expert's rows its N (32 .. 192), so that an expert with few rows does not
// pay for a full tile.  A persistent grid of CTA pairs; warps have fixed roles, linked by mbarriers:
//   warp 0       TMA: per K step of 128, the CTA's 128 weight rows and half of the tile's rows.  A panel of 32 columns holds
//                the codes of consecutive rows side by side, so a box takes a panel's 64 rows as one run of 2 KB;
//   warps 4-11   weight codes -> f16, straight into tensor memory as the MMA's A (row i in lane i), every other step by each
//                four;
//   warps 12-19  codes of the rows -> f16 into 128-byte-swizzled shared memory, as B, every other step by each four;
//   warp 1       of CTA 0: one thread issues the step's eight MMAs for both CTAs;
//   warps 20-27  epilogue: two groups of four warps that take 32 rows in turn.  Scales, activation, and through shared
//                memory in 16-byte pieces of whole rows to memory.
// Two accumulators alternate.
//
// Measured: 512 tokens' gate.up (32 rows an expert, 2816 -> 2 x 704) 95 us, 5.5 TB/s of weights, bound by HBM and by the
// chain load -> convert -> MMA of the stages; 65528 rows, 704 -> 2816, 221 us, 1,180 TFLOP/s (2817 columns, which no row
// begins aligned for, 345), gate.up 424 us, 1,230; 8192^3 659 us, 1,670.  Many rows are bound by no one part: the MMA issuer,
// the converters (five instructions a 4-code word, weights again for every row tile) and the epilogue are each at work for 60 to
// 85 % of the time, the issue slots 55 %.
// What it took, us for 65528 rows 704 -> 2816 / 8192^3: K steps of 64 by bulk copies 426 / 1382; TMA tiles of 128 columns,
// segment sums in registers 316 / 941; codes as fragments, without bank conflicts, read ahead 296 / 820; eight warps for the
// rows 259 / 746; blocks of weight tiles 252 / 695; row tiles of 192 232 / 695; addresses by xor, scales by shuffle and two
// staging buffers 229 / 693 (gate.up 452 -> 444); converted stages by halves 227 / 687 (gate.up 439); rows of any
// alignment in 16-byte pieces (65528 rows to 2817 columns 404 -> 345), which also freed registers of the other forms 227 / 659
// (gate.up 424); scales before the wait, groups in turn 221; ReLU^2 without branches on the data (relu_nan; 40040 rows of 512
// experts, 256 -> 520, 92 -> 44, 65528 rows 704 -> 2816 into fp32 436 -> 268).  Dropped: stores of A of 32 columns (848 against 820), commits one step later (no change).
#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>

#include "pair.cuh"

namespace moe {

constexpr int kI8Threads = 896;
constexpr int kI8ConvA0 = 4, kI8ConvB0 = 12, kI8Epi0 = 20;   // first warps of the roles
constexpr int kI8StepK = 128;
constexpr int kI8SegSteps = 1024 / kI8StepK;
constexpr int kI8RawA = 128 * kI8StepK, kI8MaxRawStages = 7;
// For tiles of up to nt rows, 32, 64, 128 or 192 (half of them in a CTA): bytes of a stage of codes and of converted rows, and how
// many of both.  Tensor memory has two accumulators of 128 columns (192) and A's stages of 64 behind them.
__host__ __device__ constexpr int i8_raw(int nt) { return kI8RawA + nt / 2 * kI8StepK; }
__host__ __device__ constexpr int i8_conv_b(int nt) { return nt / 2 * 2 * kI8StepK; }
__host__ __device__ constexpr int i8_raw_stages(int nt) { return nt > 64 ? 4 : 7; }
__host__ __device__ constexpr int i8_conv_stages(int nt) { return nt > 128 ? 2 : 4; }
constexpr int kI8EpiBytes = 16 * 1024;
constexpr uint32_t kI8TmemCols = 512;
constexpr int kI8LimitWord = 8;   // the waits' limit in ns (int64) in the workspace: 0 means a second
constexpr size_t i8_smem(int nt) { return 1024 + i8_conv_stages(nt) * i8_conv_b(nt) + i8_raw_stages(nt) * i8_raw(nt) + 2 * kI8EpiBytes; }
constexpr size_t i8_max(size_t a, size_t b) { return a > b ? a : b; }
constexpr size_t kI8Smem = i8_max(i8_smem(192), i8_max(i8_smem(128), i8_smem(64)));   // (tiles of 32 rows take less)
static_assert(2 * 128 + 64 * i8_conv_stages(128) <= kI8TmemCols && 2 * 192 + 64 * i8_conv_stages(192) <= kI8TmemCols, "tensor memory");
static_assert(kI8Smem + sizeof(RowTiles) + 512 <= 227 * 1024, "rings and staging fit beside the table");
static_assert((kI8Threads - 1) * 2 >= kMaxE, "the last thread has no offsets");
// Sums of more than 1024 columns: the epilogue's warps hold their segments' sums in registers, which the other warps give
// up (twenty warps of 48 and eight of 128 are less than the 28 of 72 that the block starts with).
constexpr int kI8RegsOther = 48, kI8RegsEpi = 128;
constexpr int kI8RegsLaunch = 72;   // of a thread as the block is launched; with fewer a kernel is not launched (i8_short)
static_assert(20 * kI8RegsOther + 8 * kI8RegsEpi <= 28 * kI8RegsLaunch, "registers of the block");

struct I8Args {
    CUtensorMap tw;      // codes of the weights {8 bytes, panel, matrix}, boxes of 64 rows by 4 panels
    CUtensorMap tx[3];   // codes of the rows {8 bytes, panel}, boxes of 16 << i rows by 4 panels (96 rows: 64 and 32)
    const uint8_t *xq, *wq;
    int64_t w_mat;   // bytes between weight matrices
    const int32_t* offsets;
    int E, P, N, K;
    int nt;      // rows of a tile at most: 32, 64, 128 or 192
    int block;   // weight tiles of a block
    void* out;
    int32_t* err;
};

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t* v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
// 16 lanes by 16 columns of tensor memory: v[0, 1] row lane / 4, columns 2 (lane % 4) and the next, v[2, 3] row + 8,
// v[4 .. 7] the same of columns 8 on.
__device__ __forceinline__ void tmem_st_frag16(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void i8_mma(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ void i8_fail(const I8Args& g, volatile tc::Waits* waits, uint32_t rank) {
    waits->fail = 1;
    tc::st_cluster(tc::peer_addr(tc::s_addr(const_cast<const int*>(&waits->fail)), rank ^ 1u), 1u);
    set_error(g.err, tc::kErrTimeout);
}

__device__ __forceinline__ uint32_t i8_pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// MULTI: sums of more than 1024 columns.  NT: 128 (also 64, by g.nt), or 192.
template <int ACT, bool F32, bool MULTI, int NT>
__global__ void __launch_bounds__(kI8Threads, 1) int8_gemm_kernel(const __grid_constant__ I8Args g) {
    constexpr bool kGated = ACT == MOE_ACT_SWIGLU;
    constexpr int kI8ConvStages = i8_conv_stages(NT);
    // The two halves of a converted stage, 64 columns each, are handed over one by one where each group of converting warps has
    // one stage alone, so that it converts a half while the MMAs of the other run.
    constexpr int kParts = kI8ConvStages > 2 ? 1 : 2;
    constexpr uint32_t kI8ACol = 2 * NT;
    static_assert(!MULTI || NT == 128, "the epilogue's registers hold two times 32 rows");
    static_assert(kI8ConvStages % 2 == 0, "the two groups of converting warps have stages of their own");
    extern __shared__ __align__(16) unsigned char dsm_raw[];
    unsigned char* convb = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t raw_bytes = i8_raw(g.nt), raw_stages = i8_raw_stages(g.nt), convb_bytes = i8_conv_b(g.nt);
    unsigned char* raw = convb + kI8ConvStages * convb_bytes;
    unsigned char* staging = raw + raw_stages * raw_bytes;
    __shared__ uint64_t raw_full[kI8MaxRawStages], raw_empty[kI8MaxRawStages], ready[kI8ConvStages * kParts], empty[kI8ConvStages * kParts];
    __shared__ uint64_t acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t issued, tmem_base;
    __shared__ volatile tc::Waits waits;
    __shared__ RowTiles tiles;
    // (through shuffles, so that the compiler takes the roles' branches as uniform)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = __shfl_sync(0xffffffffu, tc::cluster_rank(), 0);

    if (warp == 0 && lane == 0) {
        tc::prefetch_map(&g.tw);
        tc::prefetch_map(&g.tx[0]);
    }
    if (warp == 3) tc::pair_alloc(&tmem_base, kI8TmemCols);
    if (tid == 0) {
        for (int s = 0; s < kI8MaxRawStages; ++s) {
            tc::mbar_init(&raw_full[s], 1);
            tc::mbar_init(&raw_empty[s], 8);   // four warps for A, four for B
        }
        for (int s = 0; s < kI8ConvStages * kParts; ++s) {
            tc::mbar_init(&ready[s], 16);      // the same of both CTAs
            tc::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&acc_full[s], 1);
            tc::mbar_init(&acc_empty[s], 16);
        }
        tc::mbar_init(&drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        waits.fail = 0;
        issued = 0;
    }
    pdl_wait();   // (no early trigger: the layer's next kernels would begin unevenly, 8191 tokens 1280 -> 1309 us)
    if (tid == kI8Threads - 1) {
        const long long limit = *reinterpret_cast<const volatile long long*>(g.err + kI8LimitWord);
        waits.limit_ns = limit != 0 ? limit : tc::kWaitLimitNs;
    }
    build_row_tiles<kI8Threads>(tiles, g.offsets, g.E, g.P, [&](int n) { return (n + g.nt - 1) / g.nt; });
    tc::fence_before();
    tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = tmem_base;
    TileWalk walk(tiles, (g.N + 255) / 256, g.block, blockIdx.x >> 1, gridDim.x >> 1);
    const int ksteps = (g.K + kI8StepK - 1) / kI8StepK;
    const int width = kGated ? g.N / 2 : g.N;
    int e = 0, n0 = 0, n = 0;
    auto item = [&] {
        walk.at(&e, &n0, &n);
        e = __shfl_sync(0xffffffffu, e, 0);
        n0 = __shfl_sync(0xffffffffu, n0, 0);
        n = __shfl_sync(0xffffffffu, n, 0);
    };
    auto mma_n = [&] { return (n + 31) & ~31; };

    if (warp >= kI8Epi0) {
        if constexpr (MULTI) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kI8RegsEpi));
        // -------------------------------------------------------------------- epilogue
        constexpr int kRow = (kGated ? 64 : 128) * (F32 ? 4 : 2);   // bytes of a staged row
        const int q = warp & 3, grp = (warp - kI8Epi0) >> 2, t128 = tid & 127;
        const uint32_t sb = tc::s_addr(staging + grp * kI8EpiBytes);
        const uint32_t acc0 = tc::peer_addr(tc::s_addr(&acc_empty[0]), 0);
        const int mrow = lane >> 2, ncol = 2 * (lane & 3);   // this lane's place in a fragment
        const int r8 = lane & 7;
        const int piece = kGated ? q * 2 + ((lane >> 3) & 1) : q * 4 + (lane >> 3);   // stmatrix (bf16): this lane's 16 bytes
        const uint32_t at = sb + r8 * kRow + ((piece ^ r8) << 4) + (kGated ? (lane >> 4) * 8 * kRow : 0);
        // whole rows from shared memory to memory, 16 bytes a lane: this lane's piece of every kStep-th row.  (The rows' xor is the
        // same for all of them, but for fp32 rows of 512 bytes, where every other one has bit 2 of the piece turned.)
        constexpr int kElem = F32 ? 4 : 2, kPer = kRow / 16, kEach = 16 / kElem, kStep = 128 / kPer;
        constexpr bool kTwo = kRow * 32 * 2 <= kI8EpiBytes;   // two buffers, so that one barrier a chunk will do
        const int crow = t128 / kPer, cpiece = t128 % kPer;
        const uint32_t cfrom = sb + crow * kRow + ((F32 ? cpiece ^ (2 * ((crow >> 1) & 3)) : cpiece ^ (crow & 7)) << 4);
        const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const float* sx = reinterpret_cast<const float*>(g.xq);
        const bool wide = width % (F32 ? 4 : 8) == 0;
        const int segs = (ksteps + kI8SegSteps - 1) / kI8SegSteps;
        uint32_t n_acc = 0;
        [[maybe_unused]] uint32_t turns = 0;
        bool ok = true;
        uint32_t turn = 0;   // the buffer whose turn it is, bytes from the first
        for (; walk.more(); walk.next()) {
            item();
            const int col0 = walk.mtile() * (kGated ? 128 : 256) + static_cast<int>(rank) * (kGated ? 64 : 128);
            float sw[4];   // rows mrow, + 8, + 16, + 24 of the warp's (SwiGLU: gate, gate + 8, up, up + 8)
            {
                const float* ws = reinterpret_cast<const float*>(g.wq + e * g.w_mat);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = col0 + (kGated ? 16 * q + 8 * (i & 1) : 32 * q + 8 * i) + mrow;
                    sw[i] = __ldg(ws + (kGated && i >= 2 ? width : 0) + min(c, width - 1));
                }
            }
            // (the choice once a tile; in every product it cost 65528 rows 704 -> 2816 6 us of 221)
            const bool large = __any_sync(0xffffffffu, max(max(sw[0], sw[1]), max(sw[2], sw[3])) > kI8LargeScale);
            // Short sums are bound by the epilogue: the group that begins changes from tile to tile, as an odd number of chunks is more
            // for one of them, and the scales of the chunks' rows from + lane, + 64 .. are asked for at once, before the wait.
            const int from = 32 * (MULTI ? grp : grp ^ static_cast<int>(turns++ & 1));
            [[maybe_unused]] float scales[NT / 64];
            if constexpr (!MULTI)
#pragma unroll
                for (int ch = 0; ch < NT / 64; ++ch) scales[ch] = __ldg(sx + n0 + min(from + 64 * ch + lane, n - 1));
            float sums[MULTI ? 2 : 1][32];   // of 32 rows (two times, SwiGLU: gate and up rows): 16 lanes, the other 16
            for (int seg = 0; seg < segs; ++seg) {
                // (after a wait that ran out the group's warps go on, as they meet at barriers; the sums are not valid then)
                const uint32_t buf = n_acc & 1;
                if (ok) ok = tc::mbar_wait_warp(&acc_full[buf], n_acc >> 1, &waits);
                ++n_acc;
                tc::fence_after();
                const bool last = seg + 1 == segs;
#pragma unroll (MULTI ? 2 : 1)
                for (int ch = 0; ch < NT / 64; ++ch) {
                    const int c0 = from + 64 * ch;
                    if (c0 >= n) continue;
                    float* lo = sums[MULTI ? ch : 0];
                    float* hi = lo + 16;
                    if (!MULTI || seg == 0) {
                        tc::tmem_ld_frag(tq + buf * NT + c0, lo);
                        tc::tmem_ld_frag(tq + (16u << 16) + buf * NT + c0, hi);
                        tc::tmem_wait32(lo, hi);
                    } else {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float v[16];
                            tc::tmem_ld_frag(tq + (u ? 16u << 16 : 0u) + buf * NT + c0, v);
                            tc::tmem_ld_wait(v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) lo[16 * u + j] += v[j];
                        }
                    }
                    if (MULTI && !last) continue;
                    const float scale = MULTI     ? __ldg(sx + n0 + min(c0 + lane, n - 1))
                                        : ch == 0 ? scales[0]
                                        : ch == 1 ? scales[1]
                                                  : scales[NT / 64 - 1];
                    auto scaled = [&](auto slow) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 t = make_float2(__shfl_sync(0xffffffffu, scale, 8 * i + ncol), __shfl_sync(0xffffffffu, scale, 8 * i + ncol + 1));
#pragma unroll
                            for (int u = 0; u < 4; ++u) {   // rows mrow, + 8, + 16, + 24 of the warp's: two columns each
                                float* z = (u < 2 ? lo : hi) + 4 * i + 2 * (u & 1);
                                if constexpr (decltype(slow)::value) {
                                    z[0] = i8_scaled(z[0], t.x, sw[u]), z[1] = i8_scaled(z[1], t.y, sw[u]);
                                } else {   // i8_scaled, two at a time
                                    const float2 v = unpack_f32x2(mul_f32x2(mul_f32x2(pack_f32x2(z[0], z[1]), pack_f32x2(sw[u], sw[u])), pack_f32x2(t.x, t.y)));
                                    z[0] = v.x, z[1] = v.y;
                                }
                            }
                        }
                    };
                    if (large) scaled(std::true_type{});
                    else scaled(std::false_type{});
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (kGated) lo[j] = silu_fast(lo[j]) * hi[j];
                        if (ACT == MOE_ACT_RELU2) {
                            lo[j] = relu_nan(lo[j]), hi[j] = relu_nan(hi[j]);
                            lo[j] *= lo[j], hi[j] *= hi[j];
                        }
                    }
                    if constexpr (F32) {
#pragma unroll
                        for (int j = 0; j < (kGated ? 16 : 32); ++j) {   // (column ^ 8 * row / 2: the lanes of a store meet all banks)
                            const float v = j < 16 ? lo[j] : hi[j - 16];
                            const int r = 8 * ((j & 15) >> 2) + ncol + (j & 1);
                            const int c = q * (kGated ? 16 : 32) + (j >> 4) * 16 + ((j >> 1) & 1) * 8 + mrow;
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sb + turn + r * kRow + ((c ^ (8 * (lane & 3))) << 2)), "f"(v) : "memory");
                        }
                    } else if constexpr (kGated) {
#pragma unroll
                        for (int i = 0; i < 4; i += 2)
                            tc::stsm4_t(at + turn + i * 8 * kRow, i8_pack(lo[4 * i], lo[4 * i + 1]), i8_pack(lo[4 * i + 2], lo[4 * i + 3]),
                                        i8_pack(lo[4 * i + 4], lo[4 * i + 5]), i8_pack(lo[4 * i + 6], lo[4 * i + 7]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            tc::stsm4_t(at + turn + i * 8 * kRow, i8_pack(lo[4 * i], lo[4 * i + 1]), i8_pack(lo[4 * i + 2], lo[4 * i + 3]),
                                        i8_pack(hi[4 * i], hi[4 * i + 1]), i8_pack(hi[4 * i + 2], hi[4 * i + 3]));
                    }
                    tc::named_sync(1 + grp, 128);
                    const int left = n - c0, cols = width - col0;
                    const int64_t o0 = static_cast<int64_t>(n0 + c0) * width + col0;
                    if (wide) {
                        char* to = static_cast<char*>(g.out) + (o0 + static_cast<int64_t>(crow) * width + cpiece * kEach) * kElem;
                        const int64_t pitch = static_cast<int64_t>(kStep) * width * kElem;
                        const int rows = cpiece * kEach < cols ? left - crow : 0;
#pragma unroll
                        for (int j = 0; j < 32 / kStep; ++j, to += pitch)
                            if (j * kStep < rows) *reinterpret_cast<uint4*>(to) = lds128((cfrom ^ (F32 && !kGated && (j & 1) ? 64 : 0)) + turn + j * kStep * kRow);
                    } else {   // rows that start anywhere: memory's whole pieces of 16 bytes, then the columns before and behind them
                        const int w = min(cols, kPer * kEach);
                        auto row = [&](int r) { return static_cast<char*>(g.out) + (o0 + static_cast<int64_t>(r) * width) * kElem; };
                        auto head = [&](const char* to) { return static_cast<int>((0 - reinterpret_cast<uintptr_t>(to)) & 15) / kElem; };
                        auto place = [&](int r, int byte) {   // in shared memory
                            return sb + turn + r * kRow + (((byte >> 4) ^ (F32 ? 2 * ((r >> 1) & 3) : r & 7)) << 4) + (byte & 15);
                        };
                        for (int i = t128; i < 32 * kPer; i += 128) {
                            const int r = i / kPer;
                            if (r >= left) break;
                            char* to = row(r);
                            const int c = head(to) + i % kPer * kEach, at4 = c * kElem & ~3;
                            if (c + kEach > w) continue;
                            uint32_t v[5];
#pragma unroll
                            for (int j = 0; j < 4; ++j) v[j] = lds32(place(r, at4 + 4 * j));
                            if (!F32 && (c & 1)) {   // two bytes on
                                v[4] = lds32(place(r, at4 + 16));
#pragma unroll
                                for (int j = 0; j < 4; ++j) v[j] = __byte_perm(v[j], v[j + 1], 0x5432);
                            }
                            *reinterpret_cast<uint4*>(to + c * kElem) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                        for (int i = t128; i < 64 * kEach; i += 128) {
                            const int r = i / (2 * kEach), j = i % (2 * kEach);
                            if (r >= left) break;
                            char* to = row(r);
                            const int h = min(head(to), w), behind = h + (w - h) / kEach * kEach;
                            const int c = j < kEach ? j : behind + j - kEach;
                            if (c >= (j < kEach ? h : w)) continue;
                            const uint32_t v = lds32(place(r, c * kElem & ~3));
                            if (F32) *reinterpret_cast<uint32_t*>(to + c * kElem) = v;
                            else *reinterpret_cast<uint16_t*>(to + c * kElem) = static_cast<uint16_t>(c & 1 ? v >> 16 : v);
                        }
                    }
                    if constexpr (kTwo) {
                        turn ^= kI8EpiBytes / 2;
                    } else {
                        tc::named_sync(1 + grp, 128);   // the staging is free again
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0 && ok) tc::mbar_arrive_cluster(acc0 + buf * 8);
            }
        }
        if (!ok && lane == 0) i8_fail(g, &waits, rank);
    } else {
        if constexpr (MULTI) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kI8RegsOther));
        if (warp == 0) {
            // -------------------------------------------------------------------- copies
            const bool leader = tc::elect_one();
            const uint32_t raw0 = tc::s_addr(raw);
            uint32_t st = 0, use = 0;
            bool ok = true;
            for (; walk.more() && ok; walk.next()) {
                item();
                const int half = mma_n() >> 1, before = static_cast<int>(rank) * half;
                const int col = walk.mtile() * (kGated ? 128 : 256) + static_cast<int>(rank) * (kGated ? 64 : 128);   // of the result
                int bi = 0;
                while (bi < 2 && (16 << bi) < half) ++bi;   // the smallest box of rows; more than 64: and one of 32
                const bool more = NT > 128 && half > 64;
                for (int ks = 0; ks < ksteps; ++ks) {
                    if (use > 0 && !tc::mbar_wait_warp(&raw_empty[st], use - 1, &waits)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        // (rows and panels past a matrix's end arrive as zeros)
                        const uint32_t dst = raw0 + st * raw_bytes;
                        tc::mbar_arrive_expect_tx(&raw_full[st], kI8RawA + ((16 << bi) + (more ? 32 : 0)) * kI8StepK);
                        tc::tma_3d(dst, &g.tw, 4 * col, 4 * ks, e, &raw_full[st]);
                        tc::tma_3d(dst + kI8RawA / 2, &g.tw, 4 * (col + (kGated ? width : 64)), 4 * ks, e, &raw_full[st]);
                        tc::tma_2d(dst + kI8RawA, &g.tx[bi], 4 * (n0 + before), 4 * ks, &raw_full[st]);
                        if (more) tc::tma_2d(dst + kI8RawA + 8192, &g.tx[1], 4 * (n0 + before + 64), 4 * ks, &raw_full[st]);
                    }
                    if (++st == raw_stages) st = 0, ++use;
                }
            }
            if (leader) {
                issued = use * raw_stages + st;
                if (!ok) i8_fail(g, &waits, rank);
            }
        } else if (warp == 1 && rank == 0) {
            // -------------------------------------------------------------------- MMA issuer
            const bool leader = tc::elect_one();
            const uint64_t db0 = tc::sdesc_k128(tc::s_addr(convb));
            uint32_t st = 0, use = 0, n_acc = 0;
            bool ok = true;
            bool seen = false;   // (the leader's) the step's stage was already ready when the step before was issued
            for (; walk.more() && ok; walk.next()) {
                item();
                const uint32_t idesc = tc::pair_idesc(mma_n(), 0, false, false);
                for (int ks = 0; ks < ksteps; ++ks) {
                    const int in_seg = ks % kI8SegSteps;
                    const uint32_t buf = n_acc & 1, ub = n_acc >> 1;
                    if (in_seg == 0 && ub > 0 && !tc::mbar_wait_warp(&acc_empty[buf], ub - 1, &waits)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st1 = st + 1 == kI8ConvStages ? 0 : st + 1, use1 = use + (st1 == 0);
                    const bool last = in_seg + 1 == kI8SegSteps || ks + 1 == ksteps;
                    const bool two = g.K - ks * kI8StepK > kI8StepK / 2;
#pragma unroll
                    for (int part = 0; part < kParts; ++part) {
                        if (!__any_sync(0xffffffffu, seen) && !tc::mbar_wait_warp(&ready[st * kParts + part], use, &waits)) {
                            ok = false;
                            break;
                        }
                        seen = false;
                        tc::fence_after();
                        if (leader) {
                            const bool end = part + 1 == kParts;
                            const uint64_t db = db0 + st * (convb_bytes >> 4);
                            const uint32_t ta = tmem + kI8ACol + 64 * st;
#pragma unroll
                            for (int kk = part * 8 / kParts; kk < (part + 1) * 8 / kParts; ++kk)   // (64 columns of B's rows, then the next 64)
                                if (kk < 4 || two)
                                    i8_mma(tmem + buf * NT, ta + 8 * kk, db + (kk >> 2) * (convb_bytes >> 5) + 2 * (kk & 3), idesc, in_seg > 0 || kk > 0);
                            seen = tc::mbar_test_wait(&ready[end ? st1 * kParts : st * kParts + part + 1], (end ? use1 : use) & 1u);   // beside the MMAs
                            tc::pair_commit(&empty[st * kParts + part]);
                            if (end && last) tc::pair_commit(&acc_full[buf]);
                        }
                    }
                    if (!ok) break;
                    if (last) ++n_acc;
                    st = st1;
                    use = use1;
                }
            }
            if (leader && !ok) i8_fail(g, &waits, rank);
        } else if (warp >= kI8ConvA0 && warp < kI8Epi0) {
            // -------------------------------------------------------------------- codes to f16
            const bool is_a = warp < kI8ConvB0;
            const int q = warp & 3, t128 = tid & 127;
            const uint32_t by = 2, first = ((warp - kI8ConvA0) >> 2) & 1;   // two groups of four warps each
            const uint32_t raw0 = tc::s_addr(raw), conv0 = tc::s_addr(convb), ready0 = tc::peer_addr(tc::s_addr(&ready[0]), 0);
            // A lane of A takes the codes 8 t .. 8 t + 7 (t = lane % 4) of the rows lane / 4, + 8, + 16, + 24 in a panel's 32, so
            // that a warp's loads are runs of 256 bytes.  As fragments a panel's columns then come in the order of its 4-code
            // words 0 2 4 6 1 3 5 7; the rows of B are stored in the same order.
            // (the raw tile of A is two boxes of 64 rows; SwiGLU: gate rows, then up rows)
            const uint32_t alo = (kGated ? 16 * q * 32 : (q >> 1) * (kI8RawA / 2) + (q & 1) * 1024) + lane * 8;
            const uint32_t ahi = alo + (kGated ? kI8RawA / 2 : 512);
            // B: this lane's row and half of the step's columns; lanes 4-7 of 8 begin with the second 16 bytes of a panel, so
            // that 8 lanes meet all banks, here and in the swizzled stores.
            const int brow = t128 & 63, bset = t128 >> 6, bhalf = (brow >> 2) & 1;
            // (a piece's place in its row of 128 bytes is xored with the row; the rest of the address leaves those bits alone)
            const uint32_t bto = brow * 128 + ((bhalf ^ (brow & 7)) << 4);
            const uint32_t bfrom = kI8RawA + brow * 32 + bhalf * 16;
            auto store = [&](uint32_t to, int j, uint4 v) {   // half j of a panel: words 0 2 of 16 bytes to their piece, 1 3 to the piece two on
                uint32_t h[8];
                i8_f16(v.x, h), i8_f16(v.z, h + 2), i8_f16(v.y, h + 4), i8_f16(v.w, h + 6);
                sts128(to ^ (j << 4), h);
                sts128(to ^ ((j + 2) << 4), h + 4);
            };
            uint32_t rs = first, cs = first, ruse = 0, cuse = 0;
            int ks = static_cast<int>(first);   // of the step in its item
            bool ok = true;
            for (; walk.more() && ok; walk.next()) {
                item();
                const int half = mma_n() >> 1;
                int bi = 0;
                while (bi < 2 && (16 << bi) < half) ++bi;
                const uint32_t pstride = 32u * (16 << bi);   // of the panels of the rows' (first) box
                for (; ks < ksteps; ks += by) {
                    if (!tc::mbar_wait_warp(&raw_full[rs], ruse, &waits)) {
                        ok = false;
                        break;
                    }
                    const uint32_t src = raw0 + rs * raw_bytes;
                    const bool two = g.K - ks * kI8StepK > kI8StepK / 2;   // the step's second 64 columns are not all past K
                    if (is_a) {
                        // (the first panel is read before the wait for the MMAs that use the stage, the others ahead of their use)
                        uint2 r[2][4];
                        auto read = [&](int p, uint2* v) {
                            v[0] = lds64(src + p * 2048 + alo), v[1] = lds64(src + p * 2048 + alo + 256);
                            v[2] = lds64(src + p * 2048 + ahi), v[3] = lds64(src + p * 2048 + ahi + 256);
                        };
                        read(0, r[0]);
                        const uint32_t t = tmem + (static_cast<uint32_t>(q * 32) << 16) + kI8ACol + 64 * cs;
#pragma unroll
                        for (int part = 0; part < kParts; ++part) {
                            if (cuse > 0 && !tc::mbar_wait_warp(&empty[cs * kParts + part], cuse - 1, &waits)) {
                                ok = false;
                                break;
                            }
                            tc::fence_after();
#pragma unroll
                            for (int p = part * 4 / kParts; p < (part + 1) * 4 / kParts; ++p) {
                                if (p == 2 && !two) break;
                                if (p < 3) read(p + 1, r[(p + 1) & 1]);
                                const uint2* v = r[p & 1];
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    uint32_t h[8];
                                    i8_f16(v[2 * u].x, h), i8_f16(v[2 * u + 1].x, h + 2), i8_f16(v[2 * u].y, h + 4), i8_f16(v[2 * u + 1].y, h + 6);
                                    tmem_st_frag16(t + (static_cast<uint32_t>(16 * u) << 16) + 16 * p, h);
                                }
                            }
                            __syncwarp();
                            if (part + 1 == kParts && lane == 0) tc::mbar_arrive(&raw_empty[rs]);
                            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                            tc::fence_before();
                            if (part + 1 < kParts) {
                                __syncwarp();
                                if (lane == 0) tc::mbar_arrive_cluster(ready0 + (cs * kParts + part) * 8);
                            }
                        }
                    } else {
#pragma unroll
                        for (int part = 0; part < kParts; ++part) {
                            if (cuse > 0 && !tc::mbar_wait_warp(&empty[cs * kParts + part], cuse - 1, &waits)) {
                                ok = false;
                                break;
                            }
                            if (kParts == 1 && brow < half && (two || bset == 0)) {   // two panels a lane
                                const uint32_t to = conv0 + cs * convb_bytes + bset * (convb_bytes >> 1) + bto, from = src + bfrom + bset * 2 * pstride;
                                uint4 v[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) v[j] = lds128((from + (j >> 1) * pstride) ^ ((j & 1) * 16));
#pragma unroll
                                for (int j = 0; j < 4; ++j) store(to ^ ((j >> 1) << 6), j & 1, v[j]);
                            }
                            if (kParts == 2 && (part == 0 || two)) {
                                const uint32_t ph = conv0 + cs * convb_bytes + part * (convb_bytes >> 1);
                                if (brow < half) {   // a panel a lane
                                    const uint32_t from = src + bfrom + (2 * part + bset) * pstride, to = (ph + bto) ^ (bset << 6);
                                    const uint4 v0 = lds128(from), v1 = lds128(from ^ 16);
                                    store(to, 0, v0), store(to, 1, v1);
                                }
                                // rows 64 .. 95: two of the warps, the other two the next half of the columns
                                const int r = 64 + (t128 & 31), hf = (r >> 2) & 1;
                                if (part == bset && r < half) {
                                    const uint32_t from = src + kI8RawA + 8192 + (t128 >> 5) * 1024 + (r - 64) * 32 + hf * 16;
                                    const uint32_t to = (ph + r * 128 + ((hf ^ (r & 7)) << 4)) ^ (((t128 >> 5) & 1) << 6);
                                    const uint4 v0 = lds128(from), v1 = lds128(from ^ 16);
                                    store(to, 0, v0), store(to, 1, v1);
                                }
                            }
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            if (part + 1 < kParts) {
                                __syncwarp();
                                if (lane == 0) tc::mbar_arrive_cluster(ready0 + (cs * kParts + part) * 8);
                            }
                        }
                    }
                    if (!ok) break;
                    __syncwarp();
                    if (lane == 0) {
                        if (!is_a) tc::mbar_arrive(&raw_empty[rs]);
                        tc::mbar_arrive_cluster(ready0 + (cs * kParts + kParts - 1) * 8);
                    }
                    rs += by, cs += by;
                    if (rs >= raw_stages) rs -= raw_stages, ++ruse;
                    if (cs >= kI8ConvStages) cs -= kI8ConvStages, ++cuse;
                }
                ks -= ksteps;
            }
            // the MMAs' last arrivals on this CTA's barriers, which have to land before it ends (the warps for B: each group its stages)
            for (int i = 0; i < kI8ConvStages / 2 && ok && !is_a; ++i) {
                for (int part = 0; part < kParts && ok && cuse > 0; ++part) ok = tc::mbar_wait_warp(&empty[cs * kParts + part], cuse - 1, &waits);
                cs += by;
                if (cs >= kI8ConvStages) cs -= kI8ConvStages, ++cuse;
            }
            if (!ok && lane == 0) i8_fail(g, &waits, rank);
        }
    }

    // Every copy and MMA of the pair has landed before its memories are given back: the converters waited for every copy
    // and, at the end, for the MMAs, the epilogues for every accumulator.  Where a wait ran out (both CTAs know it then)
    // the copies that were issued are waited for, and one more commit tracks all MMAs; the first of these waits that runs
    // out ends them.
    __syncwarp();   // (roles end with one lane at work)
    tc::fence_before();
    tc::cluster_sync();
    if (waits.fail) {
        if (warp == 1 && rank == 0 && tc::elect_one()) tc::pair_commit(&drained);   // (the lane that issued them)
        __syncthreads();
        if (tid == 0) {
            bool ok = tc::mbar_wait(&drained, 0);
            for (uint32_t i = issued > raw_stages ? issued - raw_stages : 0; i < issued && ok; ++i)
                ok = tc::mbar_wait(&raw_full[i % raw_stages], i / raw_stages);
        }
        __syncwarp();
        tc::cluster_sync();
    }
    tc::fence_after();
    if (warp == 3) tc::pair_dealloc(tmem, kI8TmemCols);
}

// ------------------------------------------------------------------------------- host side
namespace {

using I8Kernel = void (*)(I8Args);

template <bool MULTI, int NT>
I8Kernel i8_kernel(int act, bool f32) {
    if (act == MOE_ACT_SWIGLU) return f32 ? int8_gemm_kernel<MOE_ACT_SWIGLU, true, MULTI, NT> : int8_gemm_kernel<MOE_ACT_SWIGLU, false, MULTI, NT>;
    if (act == MOE_ACT_RELU2) return f32 ? int8_gemm_kernel<MOE_ACT_RELU2, true, MULTI, NT> : int8_gemm_kernel<MOE_ACT_RELU2, false, MULTI, NT>;
    return f32 ? int8_gemm_kernel<MOE_ACT_NONE, true, MULTI, NT> : int8_gemm_kernel<MOE_ACT_NONE, false, MULTI, NT>;
}
I8Kernel i8_kernel(bool multi, int nt, int act, bool f32) {
    if (multi) return i8_kernel<true, 128>(act, f32);
    return nt > 128 ? i8_kernel<false, 192>(act, f32) : i8_kernel<false, 128>(act, f32);
}

// Which kernels for sums of more than 1024 columns, by activation and type, were compiled to fewer registers than they redistribute:
// the epilogue's warps would wait for theirs for ever, so these are not launched.
std::atomic<bool> i8_short[3][2];

}  // namespace

cudaError_t configure_int8_codec();

cudaError_t configure_int8_kernels() {
    cudaError_t e = configure_int8_codec();
    for (int act : {MOE_ACT_SWIGLU, MOE_ACT_RELU2, MOE_ACT_NONE})
        for (bool f32 : {false, true})
            for (int kind = 0; kind < 3; ++kind) {
                const bool multi = kind == 2;
                const void* fn = reinterpret_cast<const void*>(i8_kernel(multi, kind == 1 ? 192 : 128, act, f32));
                if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kI8Smem));
                if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
                cudaFuncAttributes attr{};
                if (e == cudaSuccess && multi) e = cudaFuncGetAttributes(&attr, fn);
                if (e == cudaSuccess && multi) i8_short[act][f32] = attr.numRegs < kI8RegsLaunch;
            }
    return e;
}

cudaError_t launch_stream_int8(const void*, int64_t, const void*, int64_t, int64_t, int64_t, const int32_t*, int, void*, int, int, cudaStream_t);

cudaError_t launch_int8_matmul(const void* xq, int64_t P, const void* wq, int64_t E, int64_t N, int64_t K, const int32_t* offsets,
                               int act, void* out, int ot, int32_t* err, int num_sms, cudaStream_t s) {
    if (stream_rows(P)) return launch_stream_int8(xq, P, wq, E, N, K, offsets, act, out, ot, num_sms, s);
    const bool multi = K > kI8SegSteps * kI8StepK;
    if (multi && i8_short[act][ot == MOE_F32]) return cudaErrorInvalidConfiguration;
    I8Args g;
    std::memset(&g, 0, sizeof(g));
    g.xq = static_cast<const uint8_t*>(xq);
    g.wq = static_cast<const uint8_t*>(wq);
    g.w_mat = i8_bytes(N, K);
    g.offsets = offsets;
    g.E = static_cast<int>(E), g.P = static_cast<int>(P), g.N = static_cast<int>(N), g.K = static_cast<int>(K);
    g.out = out;
    g.err = err;
    g.block = tile_block(static_cast<int>((N + 255) / 256));
    // codes as 8-byte elements, four a row and panel: a box takes 64 rows of a panel as one run
    cudaError_t e = tensor_map(&g.tw, CU_TENSOR_MAP_DATA_TYPE_INT64, CU_TENSOR_MAP_SWIZZLE_NONE, 3, g.wq + i8_scale_bytes(N), {4 * N, K / 32, E},
                               {32 * N, g.w_mat}, {256, 4, 1});
    for (int i = 0; i < 3 && e == cudaSuccess; ++i)
        e = tensor_map(&g.tx[i], CU_TENSOR_MAP_DATA_TYPE_INT64, CU_TENSOR_MAP_SWIZZLE_NONE, 2, g.xq + i8_scale_bytes(P), {4 * P, K / 32}, {32 * P},
                       {64 << i, 4});
    if (e != cudaSuccess) return e;
    // Tiles of up to 64 rows where experts have few: smaller stages leave room for more of them, and what is on its way from
    // memory bounds the kernel then.
    // Sums of up to 1024 columns in tiles of 192 rows where experts have many: weights are converted once for each row tile.
    // In between as many rounds of the pairs as it takes, each about 128 (the weights) and the height long, so that calls whose tiles
    // would leave most pairs idle take lower ones (one matrix: 674 rows, 672 -> 640, 16.1 -> 10.5 us; 114 rows, 1728 -> 1472, 14.0
    // -> 12.1; 4728 rows, 384 -> 896, 13.2 -> 11.5).
    const int64_t groups = std::min(E, P), avg = P / groups, mtiles = (N + 255) / 256;
    g.nt = 64;
    if (avg > 48) {
        int64_t least = INT64_MAX;
        for (int nt = multi || avg < 160 ? 128 : 192; nt >= 32; nt = nt > 64 ? nt - 64 : nt / 2) {
            const int64_t n = (avg + nt - 1) / nt, high = ((avg + n - 1) / n + 31) / 32 * 32;
            const int64_t tiles = mtiles * (groups * n + (groups > 1 ? groups / 2 : 0));   // (experts are not alike)
            const int64_t cost = (tiles + num_sms / 2 - 1) / (num_sms / 2) * (128 + high);
            if (cost < least) least = cost, g.nt = nt;
        }
    }
    const int64_t bound = (N + 255) / 256 * (std::min(E, P) + P / g.nt);
    const int pairs = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(num_sms / 2, bound)));
    return launch_pairs(i8_kernel(multi, g.nt, act, ot == MOE_F32), pairs, kI8Threads, i8_smem(g.nt), s, g);
}

}  // namespace moe
