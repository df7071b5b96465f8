// ffn.cu -- the gated feed-forward block over bf16 weights, rows sorted by expert, forward and backward, on the
// 5th-generation tensor cores: bf16 MMAs by CTA pairs (tcgen05 cta_group::2), accumulators in tensor memory.
//
// All six products are out[n][m] = sum_k A(m, k) B(n, k), m the contiguous column of the result:
//                                     A (M = 256 a pair)   B (N <= 256)           k
//   z = x Wgu^T, h = act(z)           Wgu[e]   K-major     x        K-major       columns of x
//   y = h Wd^T                        Wd[e]    K-major     h        K-major       neurons
//   dh = dy Wd, dz = dh * dh/dz       Wd[e]    M-major     dy       K-major       columns of y
//   dx = dz Wgu                       Wgu[e]   M-major     dz       K-major       columns of z
//   dWgu[e] = dz^T x                  x        M-major     dz       N-major       the expert's rows
//   dWd[e] = dy^T h                   h        M-major     dy       N-major       the expert's rows
// TMA lays every tile down as the tensor core reads it in either order, so nothing is transposed in memory.  Tokens are
// the MMA's N, which goes down to 32, so an expert with few rows does not pay for 256, and an expert's row tiles are
// equally high.
//
// A persistent grid, a CTA pair per two SMs; warps have fixed roles, linked by mbarriers:
//   warp 0      TMA: per K step of 64, the CTA's 128 rows of A and half of the tile's rows of B;
//   warp 1      of CTA 0: one thread issues the step's four MMAs for both CTAs;
//   warp 2      tells CTA 0 that the CTA's tiles have landed; for the weights' gradients it first clears the rows of
//               the last step that belong to the next expert (in both operands: 0 times infinity is no 0);
//   warps 4-11  epilogue, two groups of four warps (a warp reaches 32 lanes of tensor memory) that take 32 columns (rows
//               of the result) in turn.  Fragments of the accumulators go through stmatrix, transposed, into rows of the
//               result in shared memory, and from there to memory in 16-byte pieces of whole rows.
// Two accumulators alternate, so that the epilogue runs beside the next tile's MMAs.
//
// z is kept in fp32: from a bf16 z the gradients had three roundings to bf16 on their way (rms error 0.0030 of the result,
// now 0.0024; one rounding is 0.0017), for 8191 rows of 2816 x 5632 it costs 30 us of 430 in the forward pass.  h and dz are
// bf16 because the next product's MMA takes them so.
//
// Many rows an expert are bound by the MMAs: 8191 rows of 2816 x 5632 forward 403 us, 1,930 TFLOP/s (a library product of
// 8192^3 does 1,932), with z saved 435, backward 890, 1,750 TFLOP/s.  Few rows are bound by the weights' bytes: 4096 rows of 128
// experts, 2816 and 704, forward 251 us, 6.2 TB/s; their gradients by writing as many bytes: 1.0 GB of dWgu in 198 us, 5.1 TB/s
// (a library's fill of a gigabyte writes 4.1).  32768 rows: forward 334 us, z saved 372, backward 780.
// What it took, forward us of the dense block: barriers with release and acquire over the cluster 1288, without 406 (see
// pair.cuh), blocks of weight tiles 398 (z saved 466 -> 431).  Backward: 2926, 932; z read a step ahead 890 (dz 223 -> 174);
// two launches in place of four 967 -> 889 (fp32 z between).  A sixth stage of operands: 32768 rows 350 -> 334 forward.  Addresses
// of the result's rows by steps: backward of 4096 rows 593 -> 567, 8192 601 -> 577, 16384 638 -> 628, but 32768 769 -> 777.
// Tried and dropped: streaming stores for z and the weights' gradients (no change); fences over the cluster behind the
// cleared rows (dWgu of 32768 rows of 128 experts 259 -> 370 us).
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "pair.cuh"

namespace moe {

constexpr int kFfThreads = 384;
constexpr int kFfEpi0 = 4;              // first epilogue warp
constexpr int kFfNT = 256;              // rows of B of a tile at most
constexpr int kFfStepK = 64;            // 128 bytes of bf16
constexpr int kFfABytes = 128 * 128, kFfStage = 2 * kFfABytes;
constexpr uint32_t kFfTmemCols = 512;
constexpr int kFfLimitWord = 8;         // the waits' limit in ns (int64) in the workspace: 0 means a second
static_assert((kFfThreads - 1) * 3 >= kMaxE, "the last thread has no offsets");

// What is done with a tile's sums (kEpiSwiglu: h alone, kEpiSwigluZ: z too).
enum FfEpi { kEpiNone, kEpiBf16, kEpiF32, kEpiSwiglu, kEpiSwigluZ, kEpiRelu2, kEpiSwigluGrad, kEpiRelu2Grad };

// Staging of an epilogue group, and as many stages of operands as fit beside it.
constexpr int ff_staging(int epi) {
    return epi == kEpiNone ? 0 : epi == kEpiSwiglu ? 4096 : epi == kEpiBf16 ? 8192 : epi == kEpiF32 ? 16384 : epi == kEpiSwigluZ || epi == kEpiRelu2Grad ? 20480 : 24576;
}
template <int EPI, int GEPI>
struct FfCfg {
    static constexpr int kEpiBytes = ff_staging(EPI) > ff_staging(GEPI) ? ff_staging(EPI) : ff_staging(GEPI);
    static constexpr int kRoom = 227 * 1024 - static_cast<int>(sizeof(RowTiles)) - 512 - 1024 - 2 * kEpiBytes;
    static constexpr int kStages = kRoom / kFfStage < 6 ? kRoom / kFfStage : 6;
    static constexpr size_t kSmem = 1024 + kStages * kFfStage + 2 * kEpiBytes;
    static_assert(kStages >= 5, "ring");
};

// One product.  Rows of the experts by weights, or (grad) the gradient of weights: K is the expert's rows then, N columns.
struct FfArgs {
    CUtensorMap ta;       // {k, m, expert}, SwiGLU {k, 16, half, block, expert}; M-major {m, k, expert}; grad {m, row}
    CUtensorMap tb[4];    // {k, row}, boxes of 16 << i rows; grad tb[0] {n, row}
    const int32_t* offsets;
    int E, P, M, N, K;
    int block;            // tiles of M of a block (rows)
    int log_nt;           // rows of B of a tile at most, a power of two (ff_launch; a shift, as more code before the first tile costs
                          // a small launch half a microsecond)
    int f;                // neurons
    void* out;            // y, dx or the weights' gradient: rows of M values
    const float* z_in;
    float* z_out;         // may be null
    uint16_t *h_out, *dz_out;
    int32_t* err;
};

// A launch has a product over rows, a gradient of weights, or both: the two need nothing of one another, and together they
// fill the SMs where each alone would leave some idle at its end.
struct FfWork {
    FfArgs rows, grad;
    int has_rows, has_grad;
};

__device__ __forceinline__ void ff_fail(const FfArgs& g, volatile tc::Waits* waits, uint32_t rank) {
    waits->fail = 1;
    tc::st_cluster(tc::peer_addr(tc::s_addr(const_cast<const int*>(&waits->fail)), rank ^ 1u), 1u);
    set_error(g.err, tc::kErrTimeout);
}

__device__ __forceinline__ uint32_t ff_pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
// The sigmoid s and 1 - s.  exp(-|g|) is at most 1, so that the fast division's divisor lies in [1, 2], and neither s nor
// 1 - s comes of a difference.  The hardware's 2^x is off by a few 2^-23 per unit of |g|, far below a bf16's step.
__device__ __forceinline__ float2 ff_sigmoid(float g) {
    const float e = __expf(-fabsf(g)), r = __fdividef(1.0f, 1.0f + e), t = e * r;
    return g < 0.0f ? make_float2(t, r) : make_float2(r, t);
}

// The items of one role: (row tile, tile of M) of the product over rows, then (expert, tile of N, tile of M) of the gradient;
// M tiles fastest.
template <bool GRAD>
struct FfWalk {
    TileWalk w;
    const FfWork& g;
    bool grad = false;
    int e, n0, n, steps;   // of the item: expert, first row (column) of B's tile and how many, K steps
    int k0 = 0, rows = 0;  // grad: the expert's rows
    int mtiles, ntiles, tile, mtile, stride_t, stride_m;
    __device__ FfWalk(const RowTiles& t, const FfWork& g_, int first, int stride)
        : w(t, max(1, (g_.rows.M + 255) / 256), max(1, g_.rows.block), first, stride), g(g_) {
        if constexpr (GRAD) {
            mtiles = max(1, (g.grad.M + 255) / 256);
            ntiles = (g.grad.N + (1 << g.grad.log_nt) - 1) >> g.grad.log_nt;
            // this walk's first item past the product over rows
            const int64_t before = g.has_rows ? static_cast<int64_t>(t.n_tiles) * w.mtiles : 0;
            const int64_t skip = first < before ? (before - first + stride - 1) / stride * stride : 0;
            const int at = static_cast<int>(first + skip - before);
            tile = at / mtiles;
            mtile = at - tile * mtiles;
            stride_t = stride / mtiles;
            stride_m = stride - stride_t * mtiles;
        }
    }
    __device__ bool more() {
        if (!grad) {
            if (g.has_rows && w.more()) return true;
            if (!GRAD || !g.has_grad) return false;
            grad = true;
        }
        return tile < g.grad.E * ntiles;
    }
    __device__ void next() {
        if (!GRAD || !grad) {
            w.next();
            return;
        }
        tile += stride_t;
        mtile += stride_m;
        if (mtile >= mtiles) mtile -= mtiles, ++tile;
    }
    __device__ int m0() const { return (GRAD && grad ? mtile : w.mtile()) * 256; }
    __device__ void at() {
        if (GRAD && grad) {
            e = tile / ntiles;
            n0 = (tile - e * ntiles) << g.grad.log_nt;
            n = min(1 << g.grad.log_nt, g.grad.N - n0);
            int last;
            expert_rows(g.grad.offsets, e, g.grad.P, &k0, &last);
            k0 = __shfl_sync(0xffffffffu, k0, 0);
            rows = __shfl_sync(0xffffffffu, last - k0, 0);
            steps = (rows + kFfStepK - 1) / kFfStepK;
        } else {
            w.at(&e, &n0, &n);
            e = __shfl_sync(0xffffffffu, e, 0);
            n0 = __shfl_sync(0xffffffffu, n0, 0);
            n = __shfl_sync(0xffffffffu, n, 0);
            steps = (g.rows.K + kFfStepK - 1) / kFfStepK;
        }
    }
    __device__ int mma_n() const { return (n + 31) & ~31; }
};

// EPI: of the product over rows.  A_MN: its weights are M-major.  GEPI: of the gradient, or kEpiNone.
template <int EPI, bool A_MN, int GEPI>
__global__ void __launch_bounds__(kFfThreads, 1) ffn_kernel(const __grid_constant__ FfWork g) {
    constexpr bool kGrad = GEPI != kEpiNone;
    constexpr int kFfStages = FfCfg<EPI, GEPI>::kStages, kFfEpiBytes = FfCfg<EPI, GEPI>::kEpiBytes;
    constexpr bool kGated = EPI == kEpiSwiglu || EPI == kEpiSwigluZ;   // gate and up rows interleaved in A
    constexpr bool kActGrad = EPI == kEpiSwigluGrad || EPI == kEpiRelu2Grad;
    constexpr int kHalves = kGated || EPI == kEpiSwigluGrad ? 2 : 1;   // z has gate and up columns
    static_assert(!kGrad || A_MN, "both have one order of A");
    extern __shared__ __align__(16) unsigned char dsm_raw[];
    unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char* staging = ring + kFfStages * kFfStage;
    __shared__ uint64_t full[kFfStages], ready[kFfStages], empty[kFfStages];
    __shared__ uint64_t acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t issued, tmem_base;
    __shared__ volatile tc::Waits waits;
    __shared__ RowTiles tiles;
    // (through shuffles, so that the compiler takes the roles' branches as uniform and keeps descriptors and coordinates
    // in uniform registers, where the tensor core and the copy engine take them from)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = __shfl_sync(0xffffffffu, tc::cluster_rank(), 0);

    if (warp == 0 && lane == 0) {
        if (g.has_rows) tc::prefetch_map(&g.rows.ta);
        if (kGrad && g.has_grad) tc::prefetch_map(&g.grad.ta), tc::prefetch_map(&g.grad.tb[0]);
    }
    if (warp == 3) tc::pair_alloc(&tmem_base, kFfTmemCols);
    if (tid == 0) {
        for (int s = 0; s < kFfStages; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&ready[s], 2);
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
    pdl_wait();
    pdl_trigger();   // the next product's pairs come as this one's go (32 to 128 rows dense 20.9 -> 19.3 us, a step of four launches 27.8 -> 25.4)
    if (tid == kFfThreads - 1) {
        const long long limit = *reinterpret_cast<const volatile long long*>(g.rows.err + kFfLimitWord);
        waits.limit_ns = limit != 0 ? limit : tc::kWaitLimitNs;
    }
    if (g.has_rows) build_row_tiles<kFfThreads>(tiles, g.rows.offsets, g.rows.E, g.rows.P, [&](int n) { return (n + (1 << g.rows.log_nt) - 1) >> g.rows.log_nt; });
    tc::fence_before();
    tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = tmem_base;
    FfWalk<kGrad> walk(tiles, g, blockIdx.x >> 1, gridDim.x >> 1);

    if (warp == 0) {
        // -------------------------------------------------------------------- TMA producer
        const bool leader = tc::elect_one();
        const uint32_t ring0 = tc::s_addr(ring);
        uint32_t st = 0, use = 0;
        bool ok = true;
        for (; walk.more() && ok; walk.next()) {
            walk.at();
            const int half = walk.mma_n() >> 1, b0 = walk.n0 + static_cast<int>(rank) * half;
            const int am = walk.m0() + static_cast<int>(rank) * 128;
            int bi = 0;
            while ((16 << bi) < half) ++bi;   // the smallest box of rows of B
            const bool grad = kGrad && walk.grad;
            const uint32_t bytes = kFfABytes + (grad ? (half > 64 ? 2 : 1) * 8192 : (16 << bi) * 128);
            for (int ks = 0; ks < walk.steps; ++ks) {
                if (use > 0 && !tc::mbar_wait_warp(&empty[st], use - 1, &waits)) {
                    ok = false;
                    break;
                }
                if (leader) {
                    const uint32_t a = ring0 + st * kFfStage, b = a + kFfABytes;
                    tc::mbar_arrive_expect_tx(&full[st], bytes);
                    if (grad) {
                        const int k = walk.k0 + ks * kFfStepK;
                        tc::tma_2d(a, &g.grad.ta, am, k, &full[st]);
                        tc::tma_2d(a + 8192, &g.grad.ta, am + 64, k, &full[st]);
                        tc::tma_2d(b, &g.grad.tb[0], b0, k, &full[st]);
                        if (half > 64) tc::tma_2d(b + 8192, &g.grad.tb[0], b0 + 64, k, &full[st]);
                    } else {
                        const int k = ks * kFfStepK;
                        if constexpr (kGated) {
                            tc::tma_5d(a, &g.rows.ta, k, 0, 0, am >> 5, walk.e, &full[st]);
                        } else if constexpr (!A_MN) {
                            tc::tma_3d(a, &g.rows.ta, k, am, walk.e, &full[st]);
                        } else {
                            tc::tma_3d(a, &g.rows.ta, am, k, walk.e, &full[st]);
                            tc::tma_3d(a + 8192, &g.rows.ta, am + 64, k, walk.e, &full[st]);
                        }
                        tc::tma_2d(b, &g.rows.tb[bi], k, b0, &full[st]);
                    }
                }
                if (++st == kFfStages) st = 0, ++use;
            }
        }
        const uint32_t n_issued = use * kFfStages + st;
        // the MMAs' last arrivals on this CTA's barriers, which have to land before it ends
        for (uint32_t i = 0; i < kFfStages && ok; ++i) {
            if (use > 0) ok = tc::mbar_wait_warp(&empty[st], use - 1, &waits);
            if (++st == kFfStages) st = 0, ++use;
        }
        if (leader) {
            issued = n_issued;
            if (!ok) ff_fail(g.rows, &waits, rank);
        }
    } else if (warp == 1 && rank == 0) {
        // -------------------------------------------------------------------- MMA issuer
        const bool leader = tc::elect_one();
        const uint32_t ring0 = tc::s_addr(ring);
        constexpr uint32_t kStepK = 2, kStepMn = 128, kAstep = A_MN ? kStepMn : kStepK;   // 16 values of K, in 16 bytes
        const uint64_t da0 = A_MN ? tc::sdesc_mn128(ring0, 8192) : tc::sdesc_k128(ring0);
        const uint64_t db_k = tc::sdesc_k128(ring0 + kFfABytes), db_mn = tc::sdesc_mn128(ring0 + kFfABytes, 8192);
        uint32_t st = 0, use = 0, n_acc = 0;
        bool ok = true;
        for (; walk.more() && ok; walk.next()) {
            walk.at();
            if (walk.steps == 0) continue;
            const uint32_t buf = n_acc & 1, ub = n_acc >> 1;
            ++n_acc;
            if (ub > 0 && !tc::mbar_wait_warp(&acc_empty[buf], ub - 1, &waits)) {
                ok = false;
                break;
            }
            const uint32_t dt = tmem + buf * kFfNT, idesc = tc::pair_idesc(walk.mma_n(), 1, A_MN, kGrad && walk.grad);
            const uint64_t db0 = kGrad && walk.grad ? db_mn : db_k;
            const uint32_t bstep = kGrad && walk.grad ? kStepMn : kStepK;
            for (int ks = 0; ks < walk.steps; ++ks) {
                if (!tc::mbar_wait_warp(&ready[st], use, &waits)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                if (leader) {
                    const uint64_t da = da0 + st * (kFfStage >> 4), db = db0 + st * (kFfStage >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc::pair_mma(dt, da + kk * kAstep, db + kk * bstep, idesc, ks > 0 || kk > 0);
                    tc::pair_commit(&empty[st]);
                    if (ks + 1 == walk.steps) tc::pair_commit(&acc_full[buf]);
                }
                if (++st == kFfStages) st = 0, ++use;
            }
        }
        if (leader && !ok) ff_fail(g.rows, &waits, rank);
    } else if (warp == 2) {
        // -------------------------------------------------------------------- landed tiles
        uint32_t st = 0, use = 0;
        bool ok = true;
        const uint32_t ready0 = tc::peer_addr(tc::s_addr(&ready[0]), 0);
        for (; walk.more() && ok; walk.next()) {
            walk.at();
            for (int ks = 0; ks < walk.steps; ++ks) {
                if (!tc::mbar_wait_warp(&full[st], use, &waits)) {
                    ok = false;
                    break;
                }
                if (kGrad && walk.grad) {
                    const int valid = walk.rows - ks * kFfStepK;
                    if (valid < kFfStepK) {   // rows valid .. 63 of every box
                        unsigned char* p = ring + st * kFfStage;
                        const int boxes = 2 + (walk.mma_n() > 128 ? 2 : 1);
                        for (int b = 0; b < boxes; ++b)
                            for (int i = valid * 8 + lane; i < kFfStepK * 8; i += 32)
                                *reinterpret_cast<uint4*>(p + b * 8192 + i * 16) = make_uint4(0, 0, 0, 0);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                }
                if (lane == 0) tc::mbar_arrive_cluster(ready0 + st * 8);
                if (++st == kFfStages) st = 0, ++use;
            }
        }
        if (!ok && lane == 0) ff_fail(g.rows, &waits, rank);
    } else if (warp >= kFfEpi0) {
        // -------------------------------------------------------------------- epilogue
        const int q = warp & 3, grp = (warp - kFfEpi0) >> 2, t128 = tid & 127;
        const uint32_t sb = tc::s_addr(staging + grp * kFfEpiBytes);
        const uint32_t acc0 = tc::peer_addr(tc::s_addr(&acc_empty[0]), 0);
        const int mrow = lane >> 2, ncol = 2 * (lane & 3);        // this lane's place in a fragment
        // stmatrix / ldmatrix: this lane's row (of 8 tokens) and 16-byte piece, rows of 256 bytes (32 neurons of the warp)
        // and of 128 bytes (16).  A piece's place is xored with its row, so that 8 rows of a piece meet all banks.
        const int r8 = lane & 7, p4 = q * 4 + (lane >> 3);
        const uint32_t at256 = sb + r8 * 256 + ((p4 ^ r8) << 4);
        const uint32_t at128 = sb + r8 * 128 + (((q * 2 + ((lane >> 3) & 1)) ^ r8) << 4);
        uint32_t n_acc = 0;
        bool ok = true;
        for (; walk.more(); walk.next()) {
            walk.at();
            // (an expert without rows: zeros; after a wait that ran out too, as the group's warps meet at barriers and
            // all have to come there)
            const bool grad = kGrad && walk.grad;
            bool none = !ok || walk.steps == 0;
            [[maybe_unused]] uint4 zr[4 * kHalves];
            [[maybe_unused]] auto read_z = [&](int c) {   // z of rows c .. c + 15 of the tile, 16 bytes of a row a lane
#pragma unroll
                for (int j = 0; j < 4 * kHalves; ++j) {
                    const int i = j * 128 + t128, half = i >> 9, r = c + ((i >> 5) & 15);
                    const int m = walk.m0() + static_cast<int>(rank) * 128 + 4 * (i & 31);
                    zr[j] = make_uint4(0, 0, 0, 0);
                    if (r < walk.n && m < g.rows.M)
                        zr[j] = __ldg(reinterpret_cast<const uint4*>(g.rows.z_in + static_cast<int64_t>(walk.n0 + r) * (kHalves * g.rows.f) + half * g.rows.f + m));
                }
            };
            if (kActGrad && !grad) read_z(16 * grp);
            const uint32_t buf = n_acc & 1;
            if (!none) {
                ok = tc::mbar_wait_warp(&acc_full[buf], n_acc >> 1, &waits);
                none = !ok;
                ++n_acc;
                tc::fence_after();
            }
            const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * kFfNT;
            const int am = walk.m0() + static_cast<int>(rank) * 128;
            // whole rows from shared memory to memory, 16 bytes a lane
            auto copy = [&](uint32_t from, int n_rows, void* to, int64_t first, int left, int64_t ld, int col, int cols, int row_bytes, int elem) {
                const int per = row_bytes / 16, each = 16 / elem, step = 128 / per, r = t128 / per, p = t128 % per;
                const uint32_t place = elem == 4 ? p ^ (2 * ((r >> 1) & 3)) : p ^ (r & 7), at = from + r * row_bytes + (place << 4);
                char* d = static_cast<char*>(to) + ((first + r) * ld + col + p * each) * elem;
                const int rows = p * each < cols ? left - r : 0;
#pragma unroll
                for (int j = 0; j < n_rows / step; ++j, d += step * ld * elem) {
                    if (j * step >= rows) continue;
                    uint4 v;   // (fp32 rows of 512 bytes: every other of a lane's has bit 2 of its place turned)
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"((at ^ (elem == 4 && step == 4 && (j & 1) ? 64u : 0u)) + j * step * row_bytes));
                    *reinterpret_cast<uint4*>(d) = v;
                }
            };
            auto tile = [&](auto tag, auto of_grad) {   // the item's epilogue
                constexpr int kE = decltype(tag)::value;
                constexpr bool kG = decltype(of_grad)::value;
                const FfArgs& a = kG ? g.grad : g.rows;
                if constexpr (kE == kEpiSwigluGrad || kE == kEpiRelu2Grad) {
#pragma unroll 1
                    for (int c0 = 16 * grp; c0 < walk.n; c0 += 32) {   // 16 rows of dh
                        float v[16];   // 16 lanes' neurons, the other 16's
                        const int left = walk.n - c0;
                        if (none) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = 0.0f;
                        } else {
                            tc::tmem_ld_frag16(tb + c0, v);
                            tc::tmem_ld_frag16(tb + (16u << 16) + c0, v + 8);
                        }
                        // z of these rows and neurons into shared memory, the next rows' on their way to registers
#pragma unroll
                        for (int j = 0; j < 4 * kHalves; ++j) {
                            const int i = j * 128 + t128, half = i >> 9, r = (i >> 5) & 15, p = i & 31;
                            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(sb + half * 8192 + r * 512 + ((p ^ (2 * ((r >> 1) & 3))) << 4)),
                                         "r"(zr[j].x), "r"(zr[j].y), "r"(zr[j].z), "r"(zr[j].w)
                                         : "memory");
                        }
                        if (left > 32) read_z(c0 + 32);
                        tc::named_sync(1 + grp, 128);
                        if (!none) tc::tmem_ld_wait(v);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t wa[4], wb[4];   // rows lane / 4, + 8, + 16, + 24 of the warp's neurons, a pair of rows of dz each
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const float* d = v + 8 * (m >> 1) + 4 * i + 2 * (m & 1);   // dh of the pair
                                float ga[2], gb[2];
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const int r = 8 * i + ncol + u, c = q * 32 + 8 * m + mrow;
                                    const uint32_t at = sb + r * 512 + ((c ^ (8 * (lane & 3))) << 2);
                                    const float z = lds_f32(at);
                                    if constexpr (kE == kEpiSwigluGrad) {
                                        const float2 s = ff_sigmoid(z);
                                        const float silu = z * s.x;
                                        ga[u] = d[u] * lds_f32(at + 8192) * (s.x + silu * s.y);
                                        gb[u] = d[u] * silu;
                                    } else {
                                        ga[u] = d[u] * (2.0f * relu_nan(z));
                                    }
                                }
                                wa[m] = ff_pack(ga[0], ga[1]);
                                if constexpr (kE == kEpiSwigluGrad) wb[m] = ff_pack(gb[0], gb[1]);
                            }
                            tc::stsm4_t(at256 + 16384 + i * 2048, wa[0], wa[1], wa[2], wa[3]);
                            if constexpr (kE == kEpiSwigluGrad) tc::stsm4_t(at256 + 20480 + i * 2048, wb[0], wb[1], wb[2], wb[3]);
                        }
                        tc::named_sync(1 + grp, 128);   // (the next rows' z goes where z has been read, their dz behind a barrier)
                        const int64_t row0 = walk.n0 + c0;
                        copy(sb + 16384, 16, a.dz_out, row0, left, kHalves * a.f, am, a.f - am, 256, 2);
                        if (kHalves == 2) copy(sb + 20480, 16, a.dz_out, row0, left, 2 * a.f, a.f + am, a.f - am, 256, 2);
                    }
                } else {
#pragma unroll 1
                    for (int c0 = 32 * grp; c0 < walk.n; c0 += 64) {
                        float lo[16], hi[16];
                        const int left = walk.n - c0;   // rows of the result from c0 on
                        const int64_t row0 = (kG ? static_cast<int64_t>(walk.e) * a.N : 0) + walk.n0 + c0;
                        if (none) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) lo[i] = hi[i] = 0.0f;
                        } else {
                            tc::tmem_ld_frag(tb + c0, lo);
                            tc::tmem_ld_frag(tb + (16u << 16) + c0, hi);
                        }
                        if (!none) tc::tmem_wait32(lo, hi);
                        if constexpr (kE == kEpiBf16) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                tc::stsm4_t(at256 + i * 2048, ff_pack(lo[4 * i], lo[4 * i + 1]), ff_pack(lo[4 * i + 2], lo[4 * i + 3]),
                                            ff_pack(hi[4 * i], hi[4 * i + 1]), ff_pack(hi[4 * i + 2], hi[4 * i + 3]));
                        } else if constexpr (kE == kEpiF32) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {   // (column ^ 8 * row / 2: the lanes of a store meet all banks)
                                const float v = j < 16 ? lo[j] : hi[j - 16];
                                const int i = (j & 15) >> 2, r = 8 * i + ncol + (j & 1), c = q * 32 + (j >> 4) * 16 + ((j >> 1) & 1) * 8 + mrow;
                                asm volatile("st.shared.f32 [%0], %1;" ::"r"(sb + r * 512 + ((c ^ (8 * (lane & 3))) << 2)), "f"(v) : "memory");
                            }
                        } else if constexpr (kE == kEpiSwiglu || kE == kEpiSwigluZ) {
                            if constexpr (kE == kEpiSwigluZ) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) {   // gate, up
                                    const float v = j < 16 ? lo[j] : hi[j - 16];
                                    const int r = 8 * ((j & 15) >> 2) + ncol + (j & 1), c = q * 16 + ((j >> 1) & 1) * 8 + mrow;
                                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(sb + 4096 + (j >> 4) * 8192 + r * 256 + ((c ^ (8 * (lane & 3))) << 2)), "f"(v)
                                                 : "memory");
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) lo[j] = lo[j] * ff_sigmoid(lo[j]).x * hi[j];
#pragma unroll
                            for (int i = 0; i < 4; i += 2)
                                tc::stsm4_t(at128 + (i + (lane >> 4)) * 1024, ff_pack(lo[4 * i], lo[4 * i + 1]), ff_pack(lo[4 * i + 2], lo[4 * i + 3]),
                                            ff_pack(lo[4 * i + 4], lo[4 * i + 5]), ff_pack(lo[4 * i + 6], lo[4 * i + 7]));
                        } else if constexpr (kE == kEpiRelu2) {
                            if (a.z_out) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) {
                                    const float v = j < 16 ? lo[j] : hi[j - 16];
                                    const int r = 8 * ((j & 15) >> 2) + ncol + (j & 1), c = q * 32 + (j >> 4) * 16 + ((j >> 1) & 1) * 8 + mrow;
                                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(sb + 8192 + r * 512 + ((c ^ (8 * (lane & 3))) << 2)), "f"(v) : "memory");
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                lo[j] = relu_nan(lo[j]) * relu_nan(lo[j]);
                                hi[j] = relu_nan(hi[j]) * relu_nan(hi[j]);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                tc::stsm4_t(at256 + i * 2048, ff_pack(lo[4 * i], lo[4 * i + 1]), ff_pack(lo[4 * i + 2], lo[4 * i + 3]),
                                            ff_pack(hi[4 * i], hi[4 * i + 1]), ff_pack(hi[4 * i + 2], hi[4 * i + 3]));
                        }
                        tc::named_sync(1 + grp, 128);
                        if constexpr (kE == kEpiBf16) {
                            copy(sb, 32, a.out, row0, left, a.M, am, a.M - am, 256, 2);
                        } else if constexpr (kE == kEpiF32) {
                            copy(sb, 32, a.out, row0, left, a.M, am, a.M - am, 512, 4);
                        } else if constexpr (kE == kEpiSwiglu || kE == kEpiSwigluZ) {
                            const int j0 = am >> 1;   // the CTA's first neuron
                            copy(sb, 32, a.h_out, row0, left, a.f, j0, a.f - j0, 128, 2);
                            if constexpr (kE == kEpiSwigluZ) {
                                copy(sb + 4096, 32, a.z_out, row0, left, 2 * a.f, j0, a.f - j0, 256, 4);
                                copy(sb + 12288, 32, a.z_out, row0, left, 2 * a.f, a.f + j0, a.f - j0, 256, 4);
                            }
                        } else {
                            copy(sb, 32, a.h_out, row0, left, a.f, am, a.f - am, 256, 2);
                            if (a.z_out) copy(sb + 8192, 32, a.z_out, row0, left, a.f, am, a.f - am, 512, 4);
                        }
                        tc::named_sync(1 + grp, 128);   // the staging is free again
                    }
                }
            };
            if constexpr (kGrad) {
                if (grad) tile(std::integral_constant<int, GEPI>{}, std::true_type{});
                else tile(std::integral_constant<int, EPI>{}, std::false_type{});
            } else {
                tile(std::integral_constant<int, EPI>{}, std::false_type{});
            }
            if (!none) {
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(acc0 + buf * 8);
            }
        }
        if (!ok && lane == 0) ff_fail(g.rows, &waits, rank);
    }

    // Every copy and MMA of the pair has landed before its memories are given back: the producers waited for the MMAs, the
    // epilogues for every accumulator.  Where a wait ran out (both CTAs know it then) the copies that were issued are
    // waited for, and one more commit tracks all MMAs; the first of these waits that runs out ends them.
    __syncwarp();   // (roles end with one lane at work)
    tc::fence_before();
    tc::cluster_sync();
    if (waits.fail) {
        if (warp == 1 && rank == 0 && tc::elect_one()) tc::pair_commit(&drained);   // (the lane that issued them)
        __syncthreads();
        if (tid == 0) {
            bool ok = tc::mbar_wait(&drained, 0);
            for (uint32_t n = issued > kFfStages ? issued - kFfStages : 0; n < issued && ok; ++n)
                ok = tc::mbar_wait(&full[n % kFfStages], n / kFfStages);
        }
        __syncwarp();
        tc::cluster_sync();
    }
    tc::fence_after();
    if (warp == 3) tc::pair_dealloc(tmem, kFfTmemCols);
}

// ------------------------------------------------------------------------------- host side
namespace {

// bf16 values in 128-byte-swizzled boxes; strides in values.
cudaError_t ff_map(CUtensorMap* m, int rank, const void* base, std::initializer_list<int64_t> dims, std::initializer_list<int64_t> strides,
                   std::initializer_list<int64_t> box) {
    int64_t st[4];
    std::transform(strides.begin(), strides.end(), st, [](int64_t v) { return 2 * v; });
    return tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, rank, base, dims.begin(), st, box.begin());
}

// Rows of B, K-major: boxes of 16, 32, 64, 128 rows.
cudaError_t ff_map_rows(FfArgs& g, const uint16_t* rows, int64_t P, int64_t cols) {
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 4 && e == cudaSuccess; ++i) e = ff_map(&g.tb[i], 2, rows, {cols, P}, {cols}, {kFfStepK, 16 << i});
    return e;
}

// The tiles' height (its logarithm, `least` to 8) for `rows` in `groups`: as many rounds of the pairs as it takes, each about 128 (the
// weights' side of a step) and the height long.  So calls whose tiles would leave most pairs idle take lower ones: dense blocks,
// forward and backward, with tiles of 256 / these: 245 rows of 2272 x 2208 88 / 65 us, 194 of 1600 x 432 47 / 35, 2078 of 800 x 256
// 51 / 41, 10056 of 880 x 272 143 / 123; where tiles fill the pairs anyway nothing changes.
int ff_tile_log(int64_t mtiles, int64_t groups, int64_t rows, int least, int64_t pairs) {
    int best = 8;
    int64_t best_cost = INT64_MAX;
    for (int log = 8; log >= least; --log) {
        const int64_t each = (rows + groups - 1) / groups, n = (each + (1 << log) - 1) >> log, high = ((each + n - 1) / n + 31) / 32 * 32;
        const int64_t tiles = mtiles * (groups * n + (groups > 1 ? groups / 2 : 0));   // (groups are not alike)
        const int64_t cost = (tiles + pairs - 1) / pairs * (128 + high);
        if (cost < best_cost) best_cost = cost, best = log;
    }
    return best;
}

template <int EPI, bool A_MN, int GEPI>
cudaError_t ff_launch(FfWork& g, int num_sms, cudaStream_t s) {
    int64_t items = 0;
    if (g.has_rows) {
        const int64_t mtiles = (g.rows.M + 255) / 256, groups = std::min(g.rows.E, g.rows.P);
        g.rows.block = tile_block(static_cast<int>(mtiles));
        g.rows.log_nt = ff_tile_log(mtiles, groups, g.rows.P, 5, num_sms / 2);
        items += mtiles * (groups + (g.rows.P >> g.rows.log_nt));
    }
    if (g.has_grad) {   // (its B comes in boxes of 64 for each CTA)
        const int64_t mtiles = (g.grad.M + 255) / 256 * static_cast<int64_t>(g.grad.E);
        g.grad.log_nt = ff_tile_log(mtiles, 1, g.grad.N, 7, num_sms / 2);
        items += mtiles * ((g.grad.N + (1 << g.grad.log_nt) - 1) >> g.grad.log_nt);
    }
    const int pairs = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(num_sms / 2, items)));
    return launch_pairs(ffn_kernel<EPI, A_MN, GEPI>, pairs, kFfThreads, FfCfg<EPI, GEPI>::kSmem, s, g);
}

template <int EPI, bool A_MN, int GEPI>
cudaError_t ff_configure() {
    const void* fn = reinterpret_cast<const void*>(&ffn_kernel<EPI, A_MN, GEPI>);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(FfCfg<EPI, GEPI>::kSmem));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    return e;
}

FfWork ff_work(int64_t P, int64_t E, int64_t f, const int32_t* offsets, int32_t* err) {
    FfWork g;
    std::memset(&g, 0, sizeof(g));
    for (FfArgs* a : {&g.rows, &g.grad})
        a->offsets = offsets, a->E = static_cast<int>(E), a->P = static_cast<int>(P), a->f = static_cast<int>(f), a->err = err;
    return g;
}

// The gradient [E][n][m] of weights from rows a [P][m] and b [P][n].
cudaError_t ff_set_grad(FfWork& g, const uint16_t* a, int64_t m, const uint16_t* b, int64_t n, int64_t P, void* out) {
    g.has_grad = 1;
    g.grad.M = static_cast<int>(m), g.grad.N = static_cast<int>(n), g.grad.out = out;
    const cudaError_t e = ff_map(&g.grad.ta, 2, a, {m, P}, {m}, {64, kFfStepK});
    return e != cudaSuccess ? e : ff_map(&g.grad.tb[0], 2, b, {n, P}, {n}, {64, kFfStepK});
}

}  // namespace

cudaError_t configure_ffn_kernels() {
    cudaError_t e = ff_configure<kEpiSwiglu, false, kEpiNone>();
    if (e == cudaSuccess) e = ff_configure<kEpiSwigluZ, false, kEpiNone>();
    if (e == cudaSuccess) e = ff_configure<kEpiRelu2, false, kEpiNone>();
    if (e == cudaSuccess) e = ff_configure<kEpiBf16, false, kEpiNone>();
    if (e == cudaSuccess) e = ff_configure<kEpiSwigluGrad, true, kEpiBf16>();
    if (e == cudaSuccess) e = ff_configure<kEpiSwigluGrad, true, kEpiF32>();
    if (e == cudaSuccess) e = ff_configure<kEpiRelu2Grad, true, kEpiBf16>();
    if (e == cudaSuccess) e = ff_configure<kEpiRelu2Grad, true, kEpiF32>();
    if (e == cudaSuccess) e = ff_configure<kEpiBf16, true, kEpiBf16>();
    if (e == cudaSuccess) e = ff_configure<kEpiBf16, true, kEpiF32>();
    return e;
}

cudaError_t launch_stream_bf16(const uint16_t*, int64_t, const uint16_t*, int64_t, int64_t, int64_t, const int32_t*, int, uint16_t*, float*, int,
                               cudaStream_t);

cudaError_t launch_ffn_forward(const uint16_t* x, int64_t P, const uint16_t* wgu, const uint16_t* wd, int64_t E, int64_t d, int64_t f,
                               const int32_t* offsets, int act, uint16_t* y, float* z, uint16_t* h, int32_t* err, int num_sms,
                               cudaStream_t s) {
    if (stream_rows(P)) {
        const cudaError_t r = launch_stream_bf16(x, P, wgu, E, act == MOE_ACT_SWIGLU ? 2 * f : f, d, offsets, act, h, z, num_sms, s);
        return r == cudaSuccess ? launch_stream_bf16(h, P, wd, E, d, f, offsets, MOE_ACT_NONE, y, nullptr, num_sms, s) : r;
    }
    FfWork g = ff_work(P, E, f, offsets, err);
    g.has_rows = 1;
    g.rows.z_out = z, g.rows.h_out = h;
    g.rows.K = static_cast<int>(d);
    cudaError_t e = ff_map_rows(g.rows, x, P, d);
    if (e == cudaSuccess) {
        if (act == MOE_ACT_SWIGLU) {   // 16 gate rows, the same neurons' 16 up rows, four times
            g.rows.M = static_cast<int>(2 * f);
            e = ff_map(&g.rows.ta, 5, wgu, {d, 16, 2, f / 16, E}, {d, f * d, 16 * d, 2 * f * d}, {kFfStepK, 16, 2, 4, 1});
            if (e == cudaSuccess) e = z ? ff_launch<kEpiSwigluZ, false, kEpiNone>(g, num_sms, s) : ff_launch<kEpiSwiglu, false, kEpiNone>(g, num_sms, s);
        } else {
            g.rows.M = static_cast<int>(f);
            e = ff_map(&g.rows.ta, 3, wgu, {d, f, E}, {d, f * d}, {kFfStepK, 128, 1});
            if (e == cudaSuccess) e = ff_launch<kEpiRelu2, false, kEpiNone>(g, num_sms, s);
        }
    }
    if (e == cudaSuccess) e = ff_map_rows(g.rows, h, P, f);
    if (e == cudaSuccess) e = ff_map(&g.rows.ta, 3, wd, {f, d, E}, {f, d * f}, {kFfStepK, 128, 1});
    g.rows.M = static_cast<int>(d), g.rows.K = static_cast<int>(f), g.rows.out = y;
    if (e == cudaSuccess) e = ff_launch<kEpiBf16, false, kEpiNone>(g, num_sms, s);
    return e;
}

// Two launches: dz beside the gradient of w_down, then dx beside that of w_gate_up.
cudaError_t launch_ffn_backward(const uint16_t* dy, const uint16_t* x, int64_t P, const uint16_t* wgu, const uint16_t* wd, int64_t E,
                                int64_t d, int64_t f, const int32_t* offsets, int act, const float* z, const uint16_t* h,
                                uint16_t* dz, uint16_t* dx, void* dwgu, void* dwd, int gt, int32_t* err, int num_sms, cudaStream_t s) {
    const int64_t nz = act == MOE_ACT_SWIGLU ? 2 * f : f;
    cudaError_t e = cudaSuccess;
    FfWork g = ff_work(P, E, f, offsets, err);
    if (dx || dwgu) {
        g.has_rows = 1;
        g.rows.M = static_cast<int>(f), g.rows.K = static_cast<int>(d), g.rows.z_in = z, g.rows.dz_out = dz;
        e = ff_map_rows(g.rows, dy, P, d);
        if (e == cudaSuccess) e = ff_map(&g.rows.ta, 3, wd, {f, d, E}, {f, d * f}, {64, kFfStepK, 1});
    }
    if (dwd && e == cudaSuccess) e = ff_set_grad(g, h, f, dy, d, P, dwd);
    if ((g.has_rows || g.has_grad) && e == cudaSuccess) {
        if (act == MOE_ACT_SWIGLU)
            e = gt == MOE_F32 ? ff_launch<kEpiSwigluGrad, true, kEpiF32>(g, num_sms, s) : ff_launch<kEpiSwigluGrad, true, kEpiBf16>(g, num_sms, s);
        else
            e = gt == MOE_F32 ? ff_launch<kEpiRelu2Grad, true, kEpiF32>(g, num_sms, s) : ff_launch<kEpiRelu2Grad, true, kEpiBf16>(g, num_sms, s);
    }
    g = ff_work(P, E, f, offsets, err);
    if (dx && e == cudaSuccess) {
        g.has_rows = 1;
        g.rows.M = static_cast<int>(d), g.rows.K = static_cast<int>(nz), g.rows.out = dx;
        e = ff_map_rows(g.rows, dz, P, nz);
        if (e == cudaSuccess) e = ff_map(&g.rows.ta, 3, wgu, {d, nz, E}, {d, nz * d}, {64, kFfStepK, 1});
    }
    if (dwgu && e == cudaSuccess) e = ff_set_grad(g, x, d, dz, nz, P, dwgu);
    if ((g.has_rows || g.has_grad) && e == cudaSuccess)
        e = gt == MOE_F32 ? ff_launch<kEpiBf16, true, kEpiF32>(g, num_sms, s) : ff_launch<kEpiBf16, true, kEpiBf16>(g, num_sms, s);
    return e;
}

}  // namespace moe
