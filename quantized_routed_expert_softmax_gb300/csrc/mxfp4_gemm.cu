// mxfp4_gemm.cu -- the expert-indexed product of MXFP4 rows with MXFP4 weights on the 5th-generation
// tensor cores: block-scaled 4-bit MMAs (tcgen05 kind::mxf4), accumulators in tensor memory.
//
//   z[r][n] = sum over blocks b of 32:  2^(sx[r][b] + sw[n][b]) * sum_{i in b} x[r][i] w[n][i]
//
// The MMA takes the codes as they lie in memory and both scales per block, so nothing is dequantised:
// the kernel moves bytes and issues instructions.  Weight rows fill the MMA's M = 128 and an expert's
// rows its N = 16 .. 192, so a decode batch pads its few rows to 16 and not to 128.
//
// A persistent grid (one CTA per SM) walks the (expert, row tile of x, tile of weight rows) items that
// every CTA derives from the offsets.  Warps have fixed roles, linked by mbarriers:
//   warp 0      TMA: per K step of 256, 128 weight rows and up to NT rows of x, 128 bytes each, into
//               128-byte-swizzled tiles;
//   warp 1      one thread issues the step's four K = 64 MMAs, operands in shared memory, scales in
//               tensor memory;
//   warps 4-11  epilogue: accumulators to registers, activation, stores; each quadrant of 32 lanes has two
//               warps that take 16 rows of x in turn.  Two accumulators alternate;
//   warps 12-19 the scales, every other step by each group of four: a panel's 4-byte words (128 columns) of
//               the weight rows and of the rows of x, read some steps ahead into registers and written
//               straight into the form that the MMA takes them from tensor memory in: row r's word in lane
//               r % 32 of every quadrant, column r / 32 (a warp writes the quadrant warp % 4).  Rows of x
//               start anywhere and SwiGLU interleaves gate and up rows, so no bulk copy makes that form.
// SwiGLU tiles hold 16 gate rows and the same neurons' 16 up rows in every 32 lanes, so one shuffle
// pairs them.
//
// Codes past a matrix or past K arrive as zero; rows of the tile that are no rows of the item are computed
// and not stored, and the last panel's blocks past K hold 2^0.
//
// Decode and short prefills are bound by the weights' bytes: up of 512 latent experts (1024 -> 2688, ReLU^2)
// for 32 tokens 77.2 us, 6.5 TB/s (499 MB of the experts that have rows, every byte read once); gate.up (2816 -> 2 x
// 704) of 128 experts for 512 tokens 48.0 us, 5.9 TB/s.  Long prefills are bound by storing the output while tiles come
// from L2: down (704 -> 2816) for 8191 tokens 114 us, 4.6 TB/s (into fp32 157); 83 us without its stores and 71 us
// without its epilogue.  One token (16.9 MB from L2 or HBM over 88 CTAs) takes 6.1 us, most of it the chain offsets -> items -> first
// tiles -> 11 steps -> epilogue.
// What it took to get there, 512-expert up for 32 tokens / down for 8191 tokens, us: scales by asynchronous copies
// and tcgen05.cp 176 / 240; scales through registers 157 / 260; role branches on a uniform warp number, which
// keeps the operands of MMAs and TMA in uniform registers, 109 / 208; one barrier a step, slots found 32 at a
// time 78 / 148; epilogue compiled per activation 78 / 127; 192-row tiles 78 / 115; eight epilogue warps 78 / 114
// (and gate.up of 256 rows an expert 134 -> 108).
#include <cuda.h>   // CUtensorMap and its enums; the encoder is looked up in the driver at run time
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "mxfp4.cuh"
#include "tc.cuh"

namespace moe {

constexpr int kMxThreads = 640, kMxWarps = kMxThreads / 32;
constexpr int kMxEpi0 = 4, kMxSf0 = 12;   // first epilogue and first scale warp (a warp's quadrant is its number mod 4; 2 and 3 idle)
constexpr int kMxTileM = 128;            // weight rows of an item (SwiGLU: 64 gate and 64 up rows)
constexpr int kMxStepK = 256;            // one 128-byte swizzle row of 4-bit codes
constexpr int kMxABytes = kMxTileM * 128;
constexpr int kMxAhead = 2;              // own K steps that a group of scale warps reads ahead
constexpr uint32_t kMxTmemCols = 512;
constexpr int kMxTransChunks = 3 * 31 + 2 * 3 + 2;   // 16-byte chunks of an epilogue warp's transposition
constexpr int kMxMaxBoxes = 5;
constexpr long long kMxMaxItems = 1ll << 30;
// The waits' limit in ns (int64) sits at this 32-bit word of the workspace, as in a layer's: 0 means a second; tests set
// another (-1: a wait gives up at its first look past the hardware's own suspension).
constexpr int kMxLimitWord = 8;
static_assert((kMxThreads - 1) * 2 >= kMaxE, "the last thread has no offsets");

__device__ const uint32_t kMxOne = 0x7f7f7f7fu;   // scales of 2^0

// Shared memory and tensor memory by the width of the row tile.  Tensor memory: two accumulators of
// NT columns, then per stage 8 columns of the weights' scale words (panel 0, panel 1) and two times
// kXCols of those of x.
template <int NT>
struct MxCfg {
    static constexpr int kStage = kMxABytes + NT * 128;
    static constexpr int kStages = NT > 128 ? 4 : (NT > 32 ? 6 : 9);
    static constexpr int kPair = NT > 128 ? 1 : (NT > 32 ? 2 : 3);   // stages that one commit gives back (a commit takes 190 cycles to issue)
    static constexpr int kXWords = (NT + 31) / 32;   // columns of a panel's scales of x
    static constexpr int kXCols = NT > 128 ? 8 : 4;
    static constexpr uint32_t kSfCol = 2 * NT, kSfStage = 8 + 2 * kXCols;
    static constexpr int kBoxes = NT > 128 ? 5 : (NT > 32 ? 4 : 2);
    static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStage;
    static_assert(kSmem + 30 * 1024 <= 227 * 1024, "ring fits beside the item table");
    static_assert(kStages % kPair == 0, "whole pairs");
    static_assert(kSfCol + kSfStage * kStages <= kMxTmemCols, "scale columns of every stage");
};
// Rows of box i of x: 16, 32, 64, 128, 192.
__host__ __device__ constexpr int mx_box(int i) { return i == 4 ? 192 : 16 << i; }

struct MxArgs {
    CUtensorMap tw;                  // weights: {bytes, rows, matrix}, SwiGLU {bytes, 16, half, block, matrix}
    CUtensorMap tx[kMxMaxBoxes];     // rows of x: {bytes, rows}, boxes of mx_box(i) rows
    const uint8_t* xs;               // scale panels of x
    const uint8_t* ws;               // scale panels of the first weight matrix
    int64_t w_mat;                   // bytes between weight matrices
    const int32_t* offsets;
    int E, P, N, K;
    void* out;
    int32_t* err;
};

__device__ __forceinline__ void mx_fail(const MxArgs& g, volatile tc::Waits* waits) {
    waits->fail = 1;
    set_error(g.err, tc::kErrTimeout);
}

struct MxItem {
    int e, r_first, nt, mtile;
};

// The items in order: experts with rows (slots), then row tiles, then weight tiles.  Every role walks
// them in increasing order: the row tile and the weight tile advance by the quotient and the rest of the
// stride (a division an item would be on the MMA warp's path), and a warp looks for the row tile's slot
// from the last one on, 32 slots at a time.
template <int NT>
struct MxWalk {
    const int* prefix;    // [slots] first row tile of a slot
    const int2* rows;     // first row, last row + 1
    const uint16_t* height;   // rows of a row tile, at most NT
    const uint16_t* expert;
    int n_slots, mtiles, lane;
    int stride_t, stride_m;   // stride / mtiles, stride % mtiles
    int tile, mtile;          // of the item that `at` describes
    int slot;
    __device__ MxWalk(const int* prefix_, const int2* rows_, const uint16_t* height_, const uint16_t* expert_, int mtiles_,
                      int lane_, int item, int stride)
        : prefix(prefix_), rows(rows_), height(height_), expert(expert_), n_slots(0), mtiles(mtiles_), lane(lane_),
          stride_t(stride / mtiles_), stride_m(stride % mtiles_), tile(item / mtiles_), mtile(item % mtiles_), slot(0) {}
    __device__ void next() {
        tile += stride_t;
        mtile += stride_m;
        if (mtile >= mtiles) mtile -= mtiles, ++tile;
    }
    __device__ MxItem at() {   // the whole warp
        for (;;) {
            const int i = slot + 1 + lane;
            const int n = __popc(__ballot_sync(0xffffffffu, i < n_slots && prefix[i] <= tile));
            slot += n;
            if (n < 32) break;
        }
        const int2 r = rows[slot];
        MxItem it;
        it.e = expert[slot];
        it.mtile = mtile;
        const int h = height[slot];
        it.r_first = r.x + (tile - prefix[slot]) * h;
        it.nt = min(h, r.y - it.r_first);
        return it;
    }
};

// Output forms: fp32; bf16 where 16 bytes of a row are aligned; other bf16.
enum { kOutF32 = 0, kOutWide = 1, kOutBf16 = 2 };

// SiLU to a few units in the last place at any gate: exp(-|g|) is at most 1, so that the divisor of the fast division
// lies in [1, 2], where it is good to 2 units (past 2^126 it would give 0, and a fast exponential is off by |g| units).
// Below -87 silu is still a normal fp32, down to -3e-37, and then a subnormal one.  With a correctly
// rounded division the SwiGLU epilogue of 128 x 128 results took 10,000 cycles; with the fast exponential
// 4096 tokens' gate.up (256 rows an expert) takes 78.1 us in place of 81.2, 512 tokens' 47.8 in place of 48.0.
__device__ __forceinline__ float mx_silu(float g) {
    const float e = expf(-fabsf(g));
    return __fdividef(g < 0.0f ? g * e : g, 1.0f + e);
}

// The epilogue's transposition: column f's 16 values (32 bytes) start at this 16-byte chunk.  Both the
// writes and the gathered reads of 8 lanes then meet 8 different chunks mod 8.
__device__ __forceinline__ int mx_chunk(int f) { return 3 * f + 2 * (f >> 3); }
__device__ __forceinline__ void mx_store8(uint32_t addr, const float* y) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
__device__ __forceinline__ void mx_ldsm4_t(uint32_t* w, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
}

template <int NT, int ACT, int OUT>
__global__ void __launch_bounds__(kMxThreads, 1) mxfp4_gemm_kernel(const __grid_constant__ MxArgs g) {
    using Cfg = MxCfg<NT>;
    constexpr bool kSwiglu = ACT == MOE_ACT_SWIGLU;
    extern __shared__ __align__(16) unsigned char dsm_raw[];
    unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) &
                                                           ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[Cfg::kStages], empty[Cfg::kStages / Cfg::kPair];
    __shared__ uint64_t acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t issued;   // steps whose loads this CTA has issued
    __shared__ uint32_t tmem_base;
    __shared__ int stage_nt[Cfg::kStages];   // rows of x of the stage's item, written before the TMA's arrival
    __shared__ int prefix[kMaxE];
    __shared__ int2 rows[kMaxE];
    __shared__ uint16_t height[kMaxE], expert[kMaxE];
    __shared__ int2 warp_sums[kMxWarps];
    __shared__ int n_slots, n_items;
    __shared__ uint4 trans[8][kMxTransChunks];
    __shared__ volatile tc::Waits waits;
    // the warp number through a shuffle, so that the compiler takes the roles' branches as uniform and
    // keeps descriptors and coordinates in uniform registers, where the tensor core and the copy engine
    // take them from (read out of divergent code, a step's four MMAs took 800 cycles to issue)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (warp == 1) {
        tc::prefetch_map(&g.tw);
        tc::prefetch_map(&g.tx[0]);
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::s_addr(&tmem_base)),
                     "r"(kMxTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int s = 0; s < Cfg::kStages; ++s) {
            tc::mbar_init(&full[s], 5);   // the TMA's arrival and bytes, four scale warps
            if (s % Cfg::kPair == 0) tc::mbar_init(&empty[s / Cfg::kPair], 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&acc_full[s], 1);
            tc::mbar_init(&acc_empty[s], 8);
        }
        tc::mbar_init(&drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        waits.fail = 0;
        issued = 0;
    }
    const int mtiles = (g.N + kMxTileM - 1) / kMxTileM;
    MxWalk<NT> walk(prefix, rows, height, expert, mtiles, lane, blockIdx.x, gridDim.x);
    pdl_wait();
    if (tid == kMxThreads - 1) {   // (a thread without offsets to read)
        const long long limit = *reinterpret_cast<const volatile long long*>(g.err + kMxLimitWord);
        waits.limit_ns = limit != 0 ? limit : tc::kWaitLimitNs;
    }
    {   // the slots and an exclusive prefix over them of the row tiles (2^18 and a few an expert at most, so
        // 32 bits hold their sum even where a caller's offsets overlap)
        constexpr int kPer = (kMaxE + kMxThreads - 1) / kMxThreads;
        int first[kPer], last[kPer], tiles = 0, live = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            first[i] = last[i] = 0;
            if (tid * kPer + i < g.E) mx_expert_rows(g.offsets, tid * kPer + i, g.P, &first[i], &last[i]);
            tiles += (last[i] - first[i] + NT - 1) / NT;
            live += last[i] > first[i];
        }
        int t_incl = tiles, l_incl = live;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, t_incl, o), l = __shfl_up_sync(0xffffffffu, l_incl, o);
            if (lane >= o) t_incl += t, l_incl += l;
        }
        if (lane == 31) warp_sums[warp] = make_int2(t_incl, l_incl);
        __syncthreads();
        const int2 before = lane < warp ? warp_sums[lane] : make_int2(0, 0);
        int run = __reduce_add_sync(0xffffffffu, before.x) + t_incl - tiles;
        int slot = __reduce_add_sync(0xffffffffu, before.y) + l_incl - live;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (last[i] > first[i]) {
                // an expert's row tiles are equally high, up to the 16 that the MMA's N is a multiple of
                const int n = last[i] - first[i], n_tiles = (n + NT - 1) / NT;
                prefix[slot] = run;
                height[slot] = static_cast<uint16_t>(n_tiles == 1 ? (n + 15) & ~15 : ((n + n_tiles - 1) / n_tiles + 15) & ~15);
                rows[slot] = make_int2(first[i], last[i]);
                expert[slot] = static_cast<uint16_t>(tid * kPer + i);
                ++slot;
                run += n_tiles;
            }
        }
        if (tid == kMxThreads - 1) {
            n_slots = slot;
            // (increasing offsets stay far below the cut)
            n_items = static_cast<int>(min(static_cast<long long>(run) * mtiles, kMxMaxItems));
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tmem_base;
    const int total = n_items;
    const int ksteps = (g.K + kMxStepK - 1) / kMxStepK;
    constexpr uint32_t stages = Cfg::kStages;
    walk.n_slots = n_slots;
    uint32_t sf_steps = 0;   // own K steps that a scale warp has arrived for

    if (warp == 0) {
        // -------------------------------------------------------------------- TMA producer
        const bool leader = tc::elect_one();
        const uint32_t ring0 = tc::s_addr(ring);
        uint32_t st = 0, use = 0;
        bool ok = true;
        for (int item = blockIdx.x; item < total && ok; item += gridDim.x, walk.next()) {
            const MxItem it = walk.at();
            int bi = 0;
            while (bi + 1 < Cfg::kBoxes && mx_box(bi) < it.nt) ++bi;   // smallest box covering the rows
            const uint32_t bytes = static_cast<uint32_t>(kMxABytes + mx_box(bi) * 128);
            for (int ks = 0; ks < ksteps; ++ks) {
                if (use > 0 && !tc::mbar_wait_warp(&empty[st / Cfg::kPair], use - 1, &waits)) {
                    ok = false;
                    break;
                }
                if (leader) {
                    stage_nt[st] = it.nt;
                    tc::mbar_arrive_expect_tx(&full[st], bytes);
                    const uint32_t dst = ring0 + st * Cfg::kStage;
                    if (kSwiglu) tc::tma_5d(dst, &g.tw, ks * 128, 0, 0, it.mtile * 4, it.e, &full[st]);
                    else tc::tma_3d(dst, &g.tw, ks * 128, it.mtile * kMxTileM, it.e, &full[st]);
                    tc::tma_2d(dst + kMxABytes, &g.tx[bi], ks * 128, it.r_first, &full[st]);
                }
                if (++st == stages) st = 0, ++use;
            }
        }
        if (leader) {
            issued = use * stages + st;
            if (!ok) mx_fail(g, &waits);
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------------- MMA issuer
        const bool leader = tc::elect_one();
        const uint64_t da0 = tc::sdesc_k128(tc::s_addr(ring));
        const uint64_t db0 = tc::sdesc_k128(tc::s_addr(ring + kMxABytes));
        const int items = total > static_cast<int>(blockIdx.x) ? (total - 1 - blockIdx.x) / gridDim.x + 1 : 0;
        uint32_t st = 0, use = 0;
        bool ok = true;
        bool ready = false;   // (the leader's) the step's stage was already full when the step before was issued
        for (int n_item = 0; n_item < items && ok; ++n_item) {
            const uint32_t buf = n_item & 1, ub = n_item >> 1;
            if (ub > 0 && !tc::mbar_wait_warp(&acc_empty[buf], ub - 1, &waits)) {
                ok = false;
                break;
            }
            const uint32_t dt = tmem + buf * NT;
            uint32_t idesc = 0;
            for (int ks = 0; ks < ksteps; ++ks) {
                if (!__any_sync(0xffffffffu, ready) && !tc::mbar_wait_warp(&full[st], use, &waits)) {
                    ok = false;
                    break;
                }
                if (ks == 0) {
                    __syncwarp();   // (the leader alone may have seen the stage full)
                    idesc = tc::idesc_mxf4((stage_nt[st] + 15) & ~15);
                }
                const uint32_t st1 = st + 1 == stages ? 0 : st + 1, use1 = use + (st1 == 0);
                ready = false;
                tc::fence_after();
                if (leader) {
                    // (the descriptors' start address, bytes / 16, is linear in the address)
                    const uint64_t da = da0 + st * (Cfg::kStage >> 4);
                    const uint64_t db = db0 + st * (Cfg::kStage >> 4);
                    const uint32_t ta = tmem + Cfg::kSfCol + st * Cfg::kSfStage, tb = ta + 8;
                    // (slices past K multiply zero codes by scales of 2^0)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)   // 32 bytes of codes; blocks 2 (kk % 2), + 1 of panel kk / 2
                        tc::umma_mxf4(dt, da + 2 * kk, db + 2 * kk, idesc | tc::idesc_sf((kk & 1) * 2),
                                      ta + 4 * (kk >> 1), tb + Cfg::kXCols * (kk >> 1), ks > 0 || kk > 0);
                    ready = tc::mbar_test_wait(&full[st1], use1 & 1u);   // beside the MMAs
                    if (st % Cfg::kPair == Cfg::kPair - 1) tc::commit(&empty[st / Cfg::kPair]);
                    if (ks + 1 == ksteps) tc::commit(&acc_full[buf]);
                }
                st = st1;
                use = use1;
            }
        }
        if (leader && !ok) mx_fail(g, &waits);
    } else if (warp >= kMxSf0) {
        // -------------------------------------------------------------------- scales
        // Group grp takes the steps whose number has parity grp, so that one group's waits overlap the
        // other's.  Words are read kMxAhead own steps before they are written.
        constexpr int kXW = Cfg::kXWords;
        struct Words {
            uint32_t w[2][4], x[2][kXW];
        } buf[kMxAhead];
        const int grp = (warp - kMxSf0) >> 2;
        const int f = g.N / 2, npan = static_cast<int>(mx_panels(g.K));
        const int64_t w_pitch = 4ll * g.N, x_pitch = 4ll * g.P;
        // This lane's words in the step's first panel.  Rows past the end read another row's word, and a
        // panel past the end reads kMxOne: a read that always happens is not waited for until its word is
        // used.
        const uint8_t *wp[4], *xp[kXW];
        int ld_item = blockIdx.x, ld_ks = 0;
        auto point = [&](int ks) {   // the pointers at step ks of ld_item
            const MxItem it = walk.at();
            const uint8_t* base = g.ws + it.e * g.w_mat + 2 * ks * w_pitch;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                int n = min(it.mtile * kMxTileM + 32 * j + lane, g.N - 1);
                if (kSwiglu) n = (lane >> 4) * f + min(it.mtile * 64 + 16 * j + (lane & 15), f - 1);
                wp[j] = base + 4ll * n;
            }
#pragma unroll
            for (int j = 0; j < kXW; ++j)
                xp[j] = g.xs + 4ll * (it.r_first + min(32 * j + lane, it.nt - 1)) + 2 * ks * x_pitch;
        };
        auto advance = [&](int by) {   // on to the group's next step
            ld_ks += by;
            if (ld_ks < ksteps) {
#pragma unroll
                for (int j = 0; j < 4; ++j) wp[j] += 2 * by * w_pitch;
#pragma unroll
                for (int j = 0; j < kXW; ++j) xp[j] += 2 * by * x_pitch;
                return;
            }
            while (ld_ks >= ksteps && ld_item < total) {
                ld_ks -= ksteps;
                ld_item += gridDim.x;
                walk.next();
            }
            if (ld_item < total) point(ld_ks);
        };
        auto read = [&](Words& b) {
            if (ld_item >= total) return;
            const bool two = 2 * ld_ks + 1 < npan;
            auto word = [](const void* p) { return __ldg(static_cast<const uint32_t*>(p)); };
            const void* one = &kMxOne;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                b.w[0][j] = word(wp[j]);
                b.w[1][j] = word(two ? wp[j] + w_pitch : one);
            }
#pragma unroll
            for (int j = 0; j < kXW; ++j) {
                b.x[0][j] = word(xp[j]);
                b.x[1][j] = word(two ? xp[j] + x_pitch : one);
            }
            advance(2);
        };
        const uint32_t t0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + Cfg::kSfCol;
        const int items = total > static_cast<int>(blockIdx.x) ? (total - 1 - blockIdx.x) / gridDim.x + 1 : 0;
        const int64_t steps = (static_cast<int64_t>(items) * ksteps - grp + 1) / 2;   // of this group
        uint32_t st = grp, use = 0;
        bool ok = true;
        if (ld_item < total) {
            point(0);
            if (grp) advance(1);
        }
#pragma unroll
        for (int i = 0; i < kMxAhead; ++i) read(buf[i]);
        for (int64_t g0 = 0; g0 < steps && ok; g0 += kMxAhead) {
#pragma unroll
            for (int i = 0; i < kMxAhead; ++i) {
                if (g0 + i >= steps || !ok) break;
                if (use > 0 && !tc::mbar_wait_warp(&empty[st / Cfg::kPair], use - 1, &waits)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint32_t t = t0 + st * Cfg::kSfStage;
                tc::tmem_st4(t, buf[i].w[0]);
                tc::tmem_st4(t + 4, buf[i].w[1]);
                tc::tmem_st<kXW>(t + 8, buf[i].x[0]);
                tc::tmem_st<kXW>(t + 8 + Cfg::kXCols, buf[i].x[1]);
                read(buf[i]);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&full[st]);
                ++sf_steps;
                st += 2;
                if (st >= stages) st -= stages, ++use;
            }
        }
        if (!ok && lane == 0) mx_fail(g, &waits);
    } else if (warp >= kMxEpi0) {
        // -------------------------------------------------------------------- epilogue
        // (activation and output form are template parameters: the loop over 16 rows of x has to stay
        // short, as a warp that runs alone on its scheduler pays for every instruction it fetches)
        const int q = warp & 3, half = (warp - kMxEpi0) >> 2;   // lane quadrant of tensor memory; which 16 rows of 32
        const int nout = kSwiglu ? g.N / 2 : g.N;
        const bool up = kSwiglu && lane >= 16;
        const int wcol = kSwiglu ? 16 * q : 32 * q;   // the warp's first column in the tile
        // kOutWide: where this lane writes, and reads back, the transposition, and the column it stores
        const uint32_t tr = tc::s_addr(&trans[warp - kMxEpi0][0]);
        const uint32_t tr_st = tr + 16 * (kSwiglu ? mx_chunk(lane & 15) + (up ? 1 : 0) : mx_chunk(lane));
        const int c8 = lane & 7, m4 = lane >> 3;
        const uint32_t tr_ld = tr + 16 * (kSwiglu ? mx_chunk(4 * (c8 >> 1) + 2 * (m4 & 1) + (c8 & 1)) + (m4 >> 1)
                                                  : mx_chunk(8 * (c8 >> 1) + 2 * m4 + (c8 & 1)));
        const int lcol = wcol + (OUT == kOutWide ? (kSwiglu ? 4 : 8) * (lane & 3) : (kSwiglu ? lane & 15 : lane));
        const int lrow = 16 * half + (OUT == kOutWide ? lane >> 2 : (up ? 8 : 0));   // this lane's first row of the tile
        uint32_t n_item = 0;
        bool ok = true;
        for (int item = blockIdx.x; item < total; item += gridDim.x, ++n_item, walk.next()) {
            const MxItem it = walk.at();
            const uint32_t buf = n_item & 1;
            if (!tc::mbar_wait_warp(&acc_full[buf], n_item >> 1, &waits)) {
                ok = false;
                break;
            }
            tc::fence_after();
            const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * NT;
            const int col = it.mtile * (kSwiglu ? 64 : kMxTileM) + lcol;
            const bool in = col < nout;
            int left = it.nt - lrow;   // rows of the item from this lane's first on
            char* o = static_cast<char*>(g.out) +
                      (static_cast<int64_t>(it.r_first + lrow) * nout + col) * (OUT == kOutF32 ? 4 : 2);
            const int64_t pitch = static_cast<int64_t>(nout) * (OUT == kOutF32 ? 4 : 2);
            float v[16];
            if (16 * half < it.nt) tc::tmem_ld16(tb + 16 * half, v);
#pragma unroll 1
            for (int c0 = 16 * half; c0 < it.nt; c0 += 32) {   // 16 rows of x
                float y[16];
                tc::tmem_ld_wait(v);
#pragma unroll
                for (int j = 0; j < 16; ++j) y[j] = v[j];
                if (c0 + 32 < it.nt) tc::tmem_ld16(tb + c0 + 32, v);
                if (kSwiglu) {
                    // lanes 0-15 hold gate rows, 16-31 the same neurons' up rows: the low half takes
                    // the first 8 rows of x and the high half the others
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float other = __shfl_xor_sync(0xffffffffu, up ? y[j] : y[j + 8], 16);
                        const float gate = up ? other : y[j], value = up ? y[j + 8] : other;   // (no branch)
                        y[j] = mx_silu(gate) * value;
                    }
                } else if (ACT == MOE_ACT_RELU2) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = y[j] > 0.0f ? y[j] * y[j] : (y[j] <= 0.0f ? 0.0f : y[j]);
                }
                if (OUT == kOutWide) {
                    // A lane has one column of the output and 16 rows of x, so that a store of a warp would
                    // be 64 bytes of one row (32 for SwiGLU).  The 16 rows go through shared memory, packed
                    // by rows, and come back transposed: lane 4 n + u has columns 8 u .. 8 u + 7 (4 u ..) of
                    // rows n and n + 8.
                    __syncwarp();
                    mx_store8(tr_st, y);
                    if (!kSwiglu) mx_store8(tr_st + 16, y + 8);
                    __syncwarp();
                    uint32_t w[8];
                    mx_ldsm4_t(w, tr_ld);
                    if (!kSwiglu) mx_ldsm4_t(w + 4, tr_ld + 16);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!in || 8 * t >= left) continue;
                        if (kSwiglu) *reinterpret_cast<uint2*>(o + 8 * t * pitch) = make_uint2(w[2 * t], w[2 * t + 1]);
                        else *reinterpret_cast<uint4*>(o + 8 * t * pitch) = make_uint4(w[4 * t], w[4 * t + 1], w[4 * t + 2], w[4 * t + 3]);
                    }
                } else {
                    char* p = o;
#pragma unroll
                    for (int j = 0; j < (kSwiglu ? 8 : 16); ++j, p += pitch) {
                        if (!in || j >= left) continue;
                        if (OUT == kOutF32) *reinterpret_cast<float*>(p) = y[j];
                        else *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(y[j]);
                    }
                }
                o += 32 * pitch;
                left -= 32;
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&acc_empty[buf]);
        }
        if (!ok && lane == 0) mx_fail(g, &waits);
    }

    // Every copy and MMA this CTA issued has landed before its memories are given back: the MMAs waited
    // for every copy and the epilogue for every MMA.  Where a wait ran out that has to be made up for.  A stage
    // is full with its copies' bytes and four scale warps: those that gave up arrive for what else was issued (at
    // most one use of each stage, as the copies wait for the MMAs), so that only the bytes are waited for, and
    // one more commit tracks all MMAs.  The first of these waits that runs out ends them: then copies or MMAs
    // have not moved for a second, and no wait would bring them to an end.
    tc::fence_before();
    __syncthreads();
    if (waits.fail) {
        if (warp >= kMxSf0 && lane == 0)
            for (uint32_t n = 2 * sf_steps + ((warp - kMxSf0) >> 2); n < issued; n += 2) tc::mbar_arrive(&full[n % stages]);
        if (warp == 1 && tc::elect_one()) tc::commit(&drained);   // (the lane that issued them)
        __syncthreads();
        if (tid == 0) {
            bool ok = tc::mbar_wait(&drained, 0);
            for (uint32_t n = issued > stages ? issued - stages : 0; n < issued && ok; ++n) ok = tc::mbar_wait(&full[n % stages], n / stages);
        }
        __syncthreads();
    }
    tc::fence_after();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kMxTmemCols));
}

// ------------------------------------------------------------------------------- host side
namespace {

PFN_cuTensorMapEncodeTiled_v12000 g_mx_encode = nullptr;

cudaError_t mx_encoder() {
    static std::once_flag once;
    static cudaError_t status = cudaSuccess;
    std::call_once(once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q{};
        status = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (status == cudaSuccess && (q != cudaDriverEntryPointSuccess || fn == nullptr)) status = cudaErrorNotSupported;
        if (status == cudaSuccess) g_mx_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return status;
}

// Bytes in 128-byte-swizzled boxes; what lies outside the tensor reads as zero.
cudaError_t mx_map(CUtensorMap* m, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    const CUresult r = g_mx_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(rank),
                                   const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

using MxKernel = void (*)(MxArgs);

template <int NT, int ACT>
MxKernel mx_kernel(int out) {
    if (out == kOutF32) return mxfp4_gemm_kernel<NT, ACT, kOutF32>;
    if (out == kOutWide || ACT == MOE_ACT_SWIGLU) return mxfp4_gemm_kernel<NT, ACT, kOutWide>;   // (N / 2 is a multiple of 32)
    return mxfp4_gemm_kernel<NT, ACT, ACT == MOE_ACT_SWIGLU ? kOutWide : kOutBf16>;
}
template <int NT>
MxKernel mx_kernel(int act, int out, size_t* smem) {
    *smem = MxCfg<NT>::kSmem;
    if (act == MOE_ACT_SWIGLU) return mx_kernel<NT, MOE_ACT_SWIGLU>(out);
    if (act == MOE_ACT_RELU2) return mx_kernel<NT, MOE_ACT_RELU2>(out);
    return mx_kernel<NT, MOE_ACT_NONE>(out);
}
MxKernel mx_kernel(int nt, int act, int out, size_t* smem) {
    if (nt == 32) return mx_kernel<32>(act, out, smem);
    return nt == 128 ? mx_kernel<128>(act, out, smem) : mx_kernel<192>(act, out, smem);
}

}  // namespace

cudaError_t configure_mxfp4_kernels() {
    cudaError_t e = mx_encoder();
    for (int nt : {32, 128, 192})
        for (int act : {MOE_ACT_SWIGLU, MOE_ACT_RELU2, MOE_ACT_NONE})
            for (int out : {kOutF32, kOutWide, kOutBf16}) {
                size_t smem = 0;
                const void* fn = reinterpret_cast<const void*>(mx_kernel(nt, act, out, &smem));
                if (e == cudaSuccess)
                    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
                if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
            }
    return e;
}

cudaError_t launch_mxfp4_matmul(const void* xq, int64_t P, const void* wq, int64_t E, int64_t N, int64_t K,
                                const int32_t* offsets, int act, void* out, int ot, int32_t* err, int num_sms,
                                cudaStream_t s) {
    MxArgs g;
    std::memset(&g, 0, sizeof(g));
    g.xs = static_cast<const uint8_t*>(xq) + mx_code_bytes(P, K);
    g.ws = static_cast<const uint8_t*>(wq) + mx_code_bytes(N, K);
    g.w_mat = mx_bytes(N, K);
    g.offsets = offsets;
    g.E = static_cast<int>(E);
    g.P = static_cast<int>(P);
    g.N = static_cast<int>(N);
    g.K = static_cast<int>(K);
    g.out = out;
    g.err = err;
    const cuuint64_t kb = static_cast<cuuint64_t>(K / 2), mat = static_cast<cuuint64_t>(g.w_mat);
    cudaError_t e;
    if (act == MOE_ACT_SWIGLU) {   // 16 gate rows, the same neurons' 16 up rows, four times
        const cuuint64_t f = static_cast<cuuint64_t>(N / 2);
        const cuuint64_t d[5] = {kb, 16, 2, f / 16, static_cast<cuuint64_t>(E)};
        const cuuint64_t st[4] = {kb, f * kb, 16 * kb, mat};
        const cuuint32_t box[5] = {128, 16, 2, 4, 1};
        e = mx_map(&g.tw, 5, wq, d, st, box);
    } else {
        const cuuint64_t d[3] = {kb, static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(E)};
        const cuuint64_t st[2] = {kb, mat};
        const cuuint32_t box[3] = {128, kMxTileM, 1};
        e = mx_map(&g.tw, 3, wq, d, st, box);
    }
    if (e != cudaSuccess) return e;
    const int64_t avg = P / std::min(E, P);
    // Row tiles of 128; of 192 from 160 rows an expert on, where the loads of weights and x from L2 bound the
    // kernel; of 32 for calls of few rows, whose deeper ring has a whole item's loads on their way at once.  us:
    //   down (704 -> 2816) of 128 experts, 64 rows an expert: 33.5 (192: 35.2); 128: 44.1 (43.6); 256: 72.0 (66.7)
    //   gate.up (2816 -> 2 x 704), 8 rows in all: 7.2 (32: 6.6); 64: 21.1 (20.6); 512: 42.0 (41.5)
    //   up of 512 experts (1024 -> 2688), 176 rows in all: 35.2 (35.5); 1408: 98.2 (99.1)
    const int nt = P <= 512 && avg <= 16 ? 32 : (avg <= 160 ? 128 : 192);
    // boxes of x: the powers of two from 16 up to the tile, so that a short group does not load a tile
    const cuuint64_t xd[2] = {kb, static_cast<cuuint64_t>(P)}, xst[1] = {kb};
    for (int i = 0; i < kMxMaxBoxes && mx_box(i) <= nt; ++i) {
        const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(mx_box(i))};
        if ((e = mx_map(&g.tx[i], 2, xq, xd, xst, box)) != cudaSuccess) return e;
    }
    const int64_t nout = act == MOE_ACT_SWIGLU ? N / 2 : N, mtiles = (N + kMxTileM - 1) / kMxTileM;
    const int64_t bound = mtiles * (std::min(E, P) + P / nt);
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(num_sms, bound)));
    size_t smem = 0;
    const MxKernel kernel = mx_kernel(nt, act, ot == MOE_F32 ? kOutF32 : (nout % 8 == 0 ? kOutWide : kOutBf16), &smem);
    return launch_pdl(kernel, dim3(grid), dim3(kMxThreads), smem, s, g);
}

}  // namespace moe
