// pair.cuh -- two CTAs on one tile (tcgen05 cta_group::2): cluster barriers, tensor-memory and MMA instructions, and the
// table of row tiles that the persistent expert products walk (sm_103a).
//
// A pair's MMA has M = 256: each CTA holds 128 rows of A, half of B's rows, and in its own tensor memory the
// accumulators of its 128 rows for all of B's.  CTA 0 issues the MMAs for both.
#pragma once

#include <initializer_list>

#include "int8.cuh"
#include "tc.cuh"

namespace moe {
namespace tc {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of both CTAs.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of CTA `rank`'s copy of a shared variable.
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
// Arrivals and waits between the pair's CTAs hand over tiles that the async proxy wrote (or that a fence.proxy.async in the
// writer's CTA has made visible to it) and tensor memory, to MMAs that read each CTA's memories from that CTA's own side.
// They go without release and acquire over the cluster, which costs some 900 cycles each: with them a K step took 1950
// cycles, without them 500.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t cluster_addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
__device__ __forceinline__ void pair_alloc(uint32_t* base, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s_addr(base)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void pair_dealloc(uint32_t base, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}
// Arrives on the barrier at this address in both CTAs once every MMA that this thread has issued is complete.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(s_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
// Instruction descriptor of a 16-bit MMA with fp32 accumulators; `format` 0 f16, 1 bf16 (both operands); M = 256.
__device__ __forceinline__ uint32_t pair_idesc(int n, uint32_t format, bool a_mn, bool b_mn) {
    return (1u << 4) | (format << 7) | (format << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | ((256u >> 4) << 24);
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
// Shared-memory descriptor of an M/N-major tile in 128-byte swizzle: per K row 64 values of M (N) in 128 bytes, 8 K rows
// 1024 bytes apart (stride byte offset), the next 64 values of M (N) `group` bytes on (leading byte offset).
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr, uint32_t group) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(group >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// 16 lanes by 32 columns of tensor memory as MMA fragments: v[4 i + 0, 1] row lane / 4, columns 8 i + 2 (lane % 4) and
// the next, v[4 i + 2, 3] the same of row lane / 4 + 8.  Valid after tmem_wait32.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_frag16(uint32_t taddr, float* v) {   // of 16 columns
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait32(float* a, float* b) {   // (the registers pass through: no use moves in front)
    tmem_ld_wait(a);
    tmem_ld_wait(b);
}

// Four 8 x 8 matrices of 16-bit values from registers (fragments as above, column pairs packed) to shared memory, transposed:
// lane l has the address of row l % 8 of matrix l / 8 as it lies in shared memory.
__device__ __forceinline__ void stsm4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace tc

// The row tiles of the experts that have rows, in shared memory.  An expert's tiles are equally high, a multiple of 32
// (a pair's MMA takes N in steps of 32).
struct RowTiles {
    int prefix[kMaxE];   // first tile of a slot
    int2 rows[kMaxE];    // first row, last row + 1
    uint16_t height[kMaxE], expert[kMaxE];
    int2 warp_sums[32];
    int n_slots, n_tiles;
};

// By all THREADS threads of the CTA; ends with a __syncthreads().  tiles_of(n): how many tiles n rows take.
template <int THREADS, typename TilesOf>
__device__ __forceinline__ void build_row_tiles(RowTiles& t, const int32_t* offsets, int E, int P, TilesOf tiles_of) {
    constexpr int kPer = (kMaxE + THREADS - 1) / THREADS;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int first[kPer], last[kPer], tiles = 0, live = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        first[i] = last[i] = 0;
        if (tid * kPer + i < E) expert_rows(offsets, tid * kPer + i, P, &first[i], &last[i]);
        tiles += tiles_of(last[i] - first[i]);
        live += last[i] > first[i];
    }
    int t_incl = tiles, l_incl = live;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, t_incl, o), b = __shfl_up_sync(0xffffffffu, l_incl, o);
        if (lane >= o) t_incl += a, l_incl += b;
    }
    if (lane == 31) t.warp_sums[warp] = make_int2(t_incl, l_incl);
    __syncthreads();
    const int2 before = lane < warp ? t.warp_sums[lane] : make_int2(0, 0);
    int run = __reduce_add_sync(0xffffffffu, before.x) + t_incl - tiles;
    int slot = __reduce_add_sync(0xffffffffu, before.y) + l_incl - live;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (last[i] > first[i]) {
            const int n = last[i] - first[i], n_tiles = tiles_of(n);
            t.prefix[slot] = run;
            t.height[slot] = static_cast<uint16_t>(((n + n_tiles - 1) / n_tiles + 31) & ~31);
            t.rows[slot] = make_int2(first[i], last[i]);
            t.expert[slot] = static_cast<uint16_t>(tid * kPer + i);
            ++slot;
            run += n_tiles;
        }
    }
    if (tid == THREADS - 1) {
        t.n_slots = slot;
        t.n_tiles = run;   // (2^25 rows in tiles of 32 at least: 2^20 an expert, 2^30 were the ranges of 1024 experts to overlap)
    }
    __syncthreads();
}

// One role's walk over the items (weight tiles in blocks of `block`, row tile, weight tile of the block), weight tiles fastest,
// from item `first` in steps of `stride`.  Blocks make the tiles that are at work at a time share weights and rows alike
// (tile_block).
struct TileWalk {
    const RowTiles& t;
    int mtiles, block, stride, lane;
    int b = 0, width, tile, m, stride_t, stride_m, slot = 0;   // block, its weight tiles; row tile and weight tile in it
    __device__ TileWalk(const RowTiles& table, int mtiles_, int block_, int first, int stride_)
        : t(table), mtiles(mtiles_), block(block_), stride(stride_), lane(threadIdx.x & 31) {
        enter(first);
        leave();
    }
    __device__ void enter(int item) {   // item of block b
        width = min(block, mtiles - b * block);
        tile = item / width;
        m = item - tile * width;
        stride_t = stride / width;
        stride_m = stride - stride_t * width;
        slot = 0;
    }
    __device__ void leave() {           // on to the block that the item is in
        while (tile >= t.n_tiles && (b + 1) * block < mtiles) {
            const int item = (tile - t.n_tiles) * width + m;
            ++b;
            enter(item);
        }
    }
    __device__ bool more() const { return tile < t.n_tiles; }
    __device__ void next() {
        tile += stride_t;
        m += stride_m;
        if (m >= width) m -= width, ++tile;
        leave();
    }
    __device__ int mtile() const { return b * block + m; }
    // The item's expert, first row and rows (the whole warp; a block's tiles are asked for in increasing order).
    __device__ void at(int* e, int* r_first, int* n) {
        for (;;) {
            const int i = slot + 1 + lane;
            const int k = __popc(__ballot_sync(0xffffffffu, i < t.n_slots && t.prefix[i] <= tile));
            slot += k;
            if (k < 32) break;
        }
        const int2 r = t.rows[slot];
        const int h = t.height[slot];
        *e = t.expert[slot];
        *r_first = r.x + (tile - t.prefix[slot]) * h;
        *n = min(h, r.y - *r_first);
    }
};

// Weight tiles of a block: about ten, as 76 pairs at work on 10 by 8 tiles read least (weight tiles and row tiles 18 in all,
// 44 by 2 take 46).  Gate and up of 8191 rows, 2816 -> 2 x 5632, z saved, read 815 MB from memory in one block of 44, as the
// results drive the weights out of L2.
inline int tile_block(int mtiles) {
    const int blocks = mtiles <= 12 ? 1 : (mtiles + 9) / 10;
    return (mtiles + blocks - 1) / blocks;
}

// A tiled tensor map (strides in bytes, one fewer than dimensions); what lies outside the tensor reads as zero.  The driver's
// encoder is looked up at run time (pair.cu).
cudaError_t tensor_map(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, int rank, const void* base, const int64_t* dims,
                       const int64_t* strides, const int64_t* box);
inline cudaError_t tensor_map(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, int rank, const void* base,
                              std::initializer_list<int64_t> dims, std::initializer_list<int64_t> strides,
                              std::initializer_list<int64_t> box) {
    return tensor_map(m, type, swizzle, rank, base, dims.begin(), strides.begin(), box.begin());
}

// Launch of CTA pairs, with the overlap that launch_pdl allows.
template <typename... Exp, typename... Act>
inline cudaError_t launch_pairs(void (*kernel)(Exp...), int pairs, int threads, size_t smem, cudaStream_t s, Act&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Act>(args)...);
}

}  // namespace moe
