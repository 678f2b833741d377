// Products on pairs of SMs (tcgen05, cta_group::2) with a fused epilogue, shared by the passes of
// cross_entropy.cu:  D[m,n] = sum_k A[m,k] B[n,k], fp16 or bf16 operands, fp32 sums.
//
// A cluster of two blocks owns tiles of 256 x 256.  Each block holds 128 rows of A and 128 rows
// of B of a stage (64 terms: 32 KB, six stages) and accumulates its 128 rows of D in its own
// tensor memory, in two buffers, so that a tile's epilogue runs beside the next one's
// products.  One block alone would read 48 KB a stage for the same 128 x 256; the pair's
// products read the other half of B from its peer.  Operands may lie either way in memory:
// K-major (rows of terms) or MN-major (rows of m or n, one a term); both come by TMA with the
// 128-byte swizzle.
//
// Roles of a block's 12 warps: 0 loads, 1 issues the products (first block) or tells the
// first block that its own stage has landed (second block), 2 holds the tensor memory, 4 to 11
// run the epilogue (a thread: one row of D, half of the columns).  Every wait is bounded.
// A role that gives up stops; what it leaves undone makes the others give up; before the block
// leaves, its own copies have landed, its products are done and the pair has met.
#pragma once

#include "layer_common.cuh"
#include "tc_common.cuh"

namespace ssm {
namespace pair {

using namespace tc;

constexpr int kTileM = 256, kTileN = 256;     // of the pair
constexpr int kRowsB = 128;                   // of A and of B in one block
constexpr int kTerms = 64;                    // of a stage
constexpr int kStages = 6;
constexpr int kOperand = kRowsB * kTerms * 2; // bytes
constexpr int kThreads = 384, kFirstEpilogue = 4, kEpilogueWarps = 8;
constexpr int kHalf = kTileN / 2;             // columns of an epilogue thread

constexpr int kLimit = 1 << 22;               // polls before a wait gives up (seconds)

struct Smem {
    static constexpr int kBar = kStages * 2 * kOperand;
    static constexpr int kBars = 3 * kStages + 5;
    static constexpr int kBlock = kBar + (kBars * 8 + 16 + 15) / 16 * 16;   // 32 x 32 values of each epilogue warp, rows of 33
    static constexpr int kTotal = kBlock + kEpilogueWarps * 32 * 33 * 4;
};
static_assert(Smem::kTotal <= 227 * 1024, "one block an SM");

// Tiles of a launch: numbers that the device works out from how many rows there are.  With `splits` > 1 the
// terms of a tile are shared by that many pairs, each of which runs the epilogue on its own sum.
struct Shape {
    int m, n, k, splits;                      // rows of A, of B, terms
};

__device__ __forceinline__ uint64_t desc_mn(uint32_t addr)      // MN-major, 128-byte swizzle: 64 x 64 blocks of 8 KB
{
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(8192 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

template <bool BF16, bool A_MN, bool B_MN>
__device__ __forceinline__ constexpr uint32_t idesc()
{
    return idesc_f16(kTileM, kTileN) | (BF16 ? (1u << 7) | (1u << 10) : 0u) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
                 ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(acc) : "memory");
}

// Arrive on the mbarrier at this offset of both blocks once the products issued so far are done.
__device__ __forceinline__ void commit_both(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n"
                 ::"r"(bar), "h"((uint16_t)3) : "memory");
}

// ... of this block alone.
__device__ __forceinline__ void commit_own(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}

// Arrive on an mbarrier of the pair's first block.  What it tells of has been done by then (a copy whose
// mbarrier was waited for, loads of tensor memory that were waited for), so no wider
// release is asked for: at the cluster's scope it and the wait became memory barriers, 1900 cycles a
// stage where the products take 512.
__device__ __forceinline__ void arrive_first(uint32_t bar)
{
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
                 "mbarrier.arrive.shared::cluster.b64 _, [r];\n\t}\n" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;\n" ::: "memory");
}

// What a launch does: its tiles, and the epilogue of each.
template <class Epi>
struct Work {
    Shape shape;
    Epi epi;
};

// One launch: groups of `group_m` row tiles, in which the row tile runs fastest.  make() says what there is to do; it
// and everything else that reads memory comes after the kernel before has finished, barriers and tensor
// memory are set up while it still runs.
// epi.tile(row, first column, tensor memory address, whether the sums are there, whether there are any terms, split, the
// warp's block of shared memory) runs for each tile with a thread's half row of D.
template <bool BF16, bool A_MN, bool B_MN, class Make>
__device__ __forceinline__ void run(int group_m, const CUtensorMap &amap, const CUtensorMap &bmap, int fail_waits, Make make)
{
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t base = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int pairs = gridDim.x / 2, pair_id = blockIdx.x / 2;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Smem::kBar);
    uint32_t *slot = reinterpret_cast<uint32_t *>(bars + Smem::kBars);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, peer = empty + 8 * kStages;
    const uint32_t accfull = peer + 8 * kStages, accempty = accfull + 16, drain = accempty + 16;
    const int cap = fail_waits ? 0 : kLimit;

    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bars + i, 1);
            mbar_init(bars + kStages + i, 1);
            mbar_init(bars + 2 * kStages + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + 3 * kStages + i, 1);
            mbar_init(bars + 3 * kStages + 2 + i, 2 * kEpilogueWarps);
        }
        mbar_init(bars + 3 * kStages + 4, 1);
        mbar_init_fence();
    }
    fence_before();
    __syncthreads();
    fence_after();
    cluster_sync();                                         // both blocks' barriers are there
    const uint32_t tmem = *slot;
    griddep_entry();
    auto work = make();
    const Shape shape = work.shape;
    auto &epi = work.epi;
    const int tiles_m = (shape.m + kTileM - 1) / kTileM, tiles_n = (shape.n + kTileN - 1) / kTileN;
    const int stages = (shape.k + kTerms - 1) / kTerms, per_split = (stages + shape.splits - 1) / shape.splits;
    const int places = tiles_m * tiles_n, tiles = places * shape.splits;
    // a tile's rows, columns and range of stages
    auto place = [&](int tile, int &m, int &n, int &k0) {
        const int split = tile / places;
        tile -= split * places;
        k0 = split * per_split;
        const int per = group_m * tiles_n, g = tile / per, in = tile - g * per;
        const int gm = min(group_m, tiles_m - g * group_m);
        m = (g * group_m + in % gm) * kTileM;
        n = in / gm * kTileN;
        return max(0, min(per_split, stages - k0));
    };

    if (warp == 0) {
        Ring<kStages> r;
        int issued = 0;
        bool ok = true;
        for (int tile = pair_id; tile < tiles && ok; tile += pairs) {
            int m, n, k0;
            const int k1 = place(tile, m, n, k0) + k0;
            m += rank * kRowsB;
            n += rank * kRowsB;
            for (int k = k0; k < k1; ++k) {
                ok = __all_sync(kFullMask, mbar_poll(empty + 8 * r.s, r.phase ^ 1, cap));
                if (!ok)
                    break;
                if (elect_one()) {
                    const uint32_t a = base + r.s * 2 * kOperand, b = a + kOperand;
                    mbar_expect_tx(bars + r.s, 2 * kOperand);
                    if (A_MN) {
                        tma_2d(a, &amap, m, k * kTerms, bars + r.s);
                        tma_2d(a + kOperand / 2, &amap, m + 64, k * kTerms, bars + r.s);
                    } else {
                        tma_2d(a, &amap, k * kTerms, m, bars + r.s);
                    }
                    if (B_MN) {
                        tma_2d(b, &bmap, n, k * kTerms, bars + r.s);
                        tma_2d(b + kOperand / 2, &bmap, n + 64, k * kTerms, bars + r.s);
                    } else {
                        tma_2d(b, &bmap, k * kTerms, n, bars + r.s);
                    }
                }
                __syncwarp();
                ++issued;
                r.next();
            }
        }
        // every copy has landed, and every stage been given back (the products' last arrivals on this block)
        for (int j = max(0, issued - kStages); j < issued; ++j) {
            mbar_poll(full + 8 * (j % kStages), (j / kStages) & 1, kLimit);
            if (ok)
                mbar_poll(empty + 8 * (j % kStages), (j / kStages) & 1, kLimit);
        }
    } else if (warp == 1 && rank == 1) {
        Ring<kStages> r;
        bool ok = true;
        for (int tile = pair_id; tile < tiles && ok; tile += pairs) {
            int m, n, k0;
            for (int k = place(tile, m, n, k0); k > 0; --k) {
                ok = __all_sync(kFullMask, mbar_poll(full + 8 * r.s, r.phase, cap));
                if (!ok)
                    break;
                if (lane == 0)
                    arrive_first(peer + 8 * r.s);
                __syncwarp();
                r.next();
            }
        }
    } else if (warp == 1) {
        constexpr uint32_t id = idesc<BF16, A_MN, B_MN>();
        Ring<kStages> r;
        Ring<2> acc;
        bool ok = true;
        for (int tile = pair_id; tile < tiles && ok; tile += pairs) {
            int m, n, k0;
            const int n_k = place(tile, m, n, k0);
            if (n_k == 0)
                continue;
            ok = __all_sync(kFullMask, mbar_poll(accempty + 8 * acc.s, acc.phase ^ 1, cap));
            if (!ok)
                break;
            const uint32_t d = tmem + kTileN * acc.s;
            for (int k = 0; k < n_k; ++k) {
                ok = mbar_poll(full + 8 * r.s, r.phase, cap) && mbar_poll(peer + 8 * r.s, r.phase, cap);
                ok = __all_sync(kFullMask, ok);
                if (!ok)
                    break;
                fence_after();
                if (elect_one()) {
                    const uint32_t a = base + r.s * 2 * kOperand, b = a + kOperand;
                    const uint64_t ad = A_MN ? desc_mn(a) : desc_sw128(a), bd = B_MN ? desc_mn(b) : desc_sw128(b);
#pragma unroll
                    for (int kk = 0; kk < kTerms / 16; ++kk)    // 16 terms: 32 bytes of a row, or 16 rows
                        mma_pair(d, ad + kk * (A_MN ? 128 : 2), bd + kk * (B_MN ? 128 : 2), id, k > 0 || kk > 0);
                    commit_both(empty + 8 * r.s);
                    if (k == n_k - 1)
                        commit_both(accfull + 8 * acc.s);
                }
                __syncwarp();
                r.next();
            }
            acc.next();
        }
        if (elect_one())
            commit_own(drain);                              // products that were issued are done before the pair leaves
        __syncwarp();
        mbar_poll(drain, 0, kLimit);
    } else if (warp >= kFirstEpilogue) {
        const int e = warp - kFirstEpilogue, quarter = e & 3, half = e >> 2;
        Ring<2> acc;
        bool ok = true;
        for (int tile = pair_id; tile < tiles; tile += pairs) {
            int m, n, k0;
            const int n_k = place(tile, m, n, k0);
            if (n_k > 0) {
                ok = ok && mbar_poll(accfull + 8 * acc.s, acc.phase, cap);
                ok = __all_sync(kFullMask, ok);
                fence_after();
            }
            const uint32_t at = tmem + kTileN * acc.s + half * kHalf + ((uint32_t)(32 * quarter) << 16);
            epi.tile(m + (int)rank * kRowsB + 32 * quarter + lane, n + half * kHalf, at, ok, n_k > 0, tile / places,
                     reinterpret_cast<float *>(sm + Smem::kBlock) + e * 32 * 33);
            if (n_k > 0) {
                fence_before();
                __syncwarp();
                if (lane == 0)
                    arrive_first(accempty + 8 * acc.s);
                acc.next();
            }
        }
    }
    __syncthreads();
    __syncwarp();
    cluster_sync();
    if (warp == 2) {
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
    }
}

// 32 columns of a thread's half row, or NaN where a wait gave up, or zeros where there are no terms.  For a whole
// warp: its lanes meet first, whatever branches an epilogue took for single rows (the load needs them together).
__device__ __forceinline__ void columns(float (&v)[32], uint32_t at, int j, bool ok, bool any)
{
    __syncwarp();
    if (any) {
        uint32_t r[32];
        tmem_ld32u(r, at + j);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] = ok ? __uint_as_float(r[i]) : __int_as_float(0x7fc00000);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] = 0.f;
    }
}

}  // namespace pair
}  // namespace ssm
