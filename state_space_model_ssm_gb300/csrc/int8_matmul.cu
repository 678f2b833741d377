// 8-bit integer matrix product with a scale for each token and each output
// channel (sm_103a):
//
//   out[t][n] = (sum_k x[t][k] w[n][k]) xs[t] ws[n] + bias[n]
//
// On sm_103a the tensor cores have no fast path for 8-bit integers, but fp16 holds
// every 8-bit integer exactly and a product of two is an integer of at most 2^14,
// so the fp16 tensor cores with their fp32 accumulator give the exact integer as
// long as the partial sums stay within 2^24: for 1024 terms.  Every kFold stages
// (1024 terms) the accumulator is moved to 32-bit integers in registers and
// starts again from zero, so the sum is the exact integer for every input.
//
// Many tokens (int8_tile_kernel).  A block owns 128 output channels and NT
// tokens, M = 128 channels x N = NT tokens x K: the weights are the A operand, which
// the tensor core reads from tensor memory.  They cross HBM, L2 and shared memory as
// bytes and become fp16 on their way from shared to tensor memory: 8 warps turn each
// byte b into the fp16 number 1024 + (b ^ 0x80) by placing it under the constant's
// exponent, and subtract 1152 (5 instructions for 4 values).  So a weight costs one
// byte of bandwidth in every place that is short of it.  The tokens are the B operand,
// K-major in shared memory with the 128-byte swizzle; a kernel in front has written
// them as fp16 once, since every block of a column of tiles reads them.  Weights that
// TMA cannot describe (an address or a stride that is no multiple of 16) are repacked
// by that kernel.
//
// Roles: one warp loads weights by TMA, one fp16 tokens, one issues the MMAs, 8
// convert and afterwards write the result (thread: one output channel, NT / 2
// tokens).  They hand stages of 128 terms to each other through mbarriers.  Every wait
// is bounded; a block that gave up drains its copies and products, frees its tensor
// memory and writes NaN.
//
// With few tokens (int8_few_kernel) the weights are read once and their bytes are the
// bound, so the work is spread over warps and not over tiles; see there.
#include "layer_common.cuh"
#include "tc_common.cuh"

namespace ssm {

namespace {

using namespace tc;

constexpr int kRows = 128;                    // output channels of a block
constexpr int kTerms = 128;                   // terms of a stage (with 64, issuing a stage took longer than its products)
constexpr int kFold = 8;                      // stages whose sum is exact in fp32: 8 x 128 x 2^14 = 2^24
constexpr int kConvWarps = 8;                 // two groups of four: a group converts every other stage
constexpr int kGroupWarps = 4;
constexpr int kWarpW = 8, kWarpMma = 9, kWarpX = 10;
constexpr int kThreads = 352;

struct I8Args {
    const float *xs, *ws, *bias;
    void *out;
    int M, N, K;
    long long so;
    int tiles_m, tiles_n;                     // token tiles, channel tiles
    int fail_waits;
};

// Shared memory (bytes; tiles 1024-aligned) and tensor memory of a block, one an SM.
template <int NT>
struct I8Layout {
    // Weight stages, 16 KB each.  An even number, so that a group meets every use of its
    // stages: with three it met every other one, and its parity wait could pass on the use before.
    static constexpr int kWStages = NT == 256 ? 2 : 4;
    static_assert(kWStages % 2 == 0, "two converting groups");
    static constexpr int kABufs = 4;                        // converted weight stages in tensor memory
    static constexpr int kACols = kTerms / 2;               // columns of one
    static constexpr int kXStages = NT == 256 ? 3 : 4;
    static constexpr int kXTile = NT * 128;                 // 64 fp16 terms of NT tokens; two to a stage
    static constexpr int kW = 0;
    static constexpr int kX = kW + kWStages * kRows * kTerms;
    static constexpr int kBar = kX + kXStages * 2 * kXTile; // mbarriers, then the tokens' scales
    static constexpr int kBars = 2 * kWStages + 2 * kXStages + 2 * kABufs + 4;
    static constexpr int kTotal = kBar + kBars * 8 + 16 + NT * 4;
    static constexpr int kTmem = 512;                       // NT + 4 x 64 columns are in use
};

__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
                 ::"r"(d), "r"(a), "l"(b), "r"(id), "r"(acc) : "memory");
}

// Four signed bytes as fp16: lo = bytes 0, 2 and hi = bytes 1, 3 (the terms' order
// within a product is free as long as weights and tokens agree, and a mask is cheaper
// than putting neighbours side by side).
__device__ __forceinline__ void bytes_to_half(uint32_t b, uint32_t &lo, uint32_t &hi)
{
    const uint32_t l = (b & 0x00FF00FFu) ^ 0x64806480u, h = (b >> 8 & 0x00FF00FFu) ^ 0x64806480u;
    const uint32_t off = 0xE480E480u;                       // -1152 twice
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(l), "r"(off));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(h), "r"(off));
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                   "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

template <class T, int NT>
__global__ void __launch_bounds__(kThreads, 1)
int8_tile_kernel(const I8Args a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap)
{
    using L = I8Layout<NT>;
    constexpr int kWStages = L::kWStages, kABufs = L::kABufs, kXRing = L::kXStages;
    griddep_entry();
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t base = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tile = blockIdx.x;
    // Tiles in groups of 8 token tiles: the blocks that run together share weights and tokens in L2.
    const int group = tile / (8 * a.tiles_n), in_group = tile - group * 8 * a.tiles_n;
    const int gm = min(8, a.tiles_m - 8 * group);
    const int m0 = (8 * group + in_group % gm) * NT, n0 = in_group / gm * kRows;
    const int n = (a.K + kTerms - 1) / kTerms;              // stages
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kBar);
    uint64_t *wfull = bars, *wempty = wfull + kWStages, *xfull = wempty + kWStages, *xempty = xfull + kXRing;
    uint64_t *afull = xempty + kXRing, *aempty = afull + kABufs, *accfull = aempty + kABufs, *accempty = accfull + 1;
    uint64_t *drain = accempty + 1;
    uint32_t *slot = reinterpret_cast<uint32_t *>(bars + L::kBars);
    float *xsc = reinterpret_cast<float *>(slot + 4);       // the tokens' scales
    const int cap = a.fail_waits ? 0 : (int)kSpinLimit;
    const uint32_t b_wfull = smem_u32(wfull), b_wempty = smem_u32(wempty), b_xfull = smem_u32(xfull);
    const uint32_t b_xempty = smem_u32(xempty), b_afull = smem_u32(afull), b_aempty = smem_u32(aempty);
    const uint32_t b_accfull = smem_u32(accfull), b_accempty = smem_u32(accempty);

    if (warp == kWarpMma)
        tmem_alloc(slot, L::kTmem);
    if (tid == 0) {
        for (int i = 0; i < kWStages; ++i) {
            mbar_init(wfull + i, 1);
            mbar_init(wempty + i, kGroupWarps);
        }
        for (int i = 0; i < kXRing; ++i) {
            mbar_init(xfull + i, 1);
            mbar_init(xempty + i, 1);
        }
        for (int i = 0; i < kABufs; ++i) {
            mbar_init(afull + i, kGroupWarps);
            mbar_init(aempty + i, 1);
        }
        mbar_init(accfull, 1);
        mbar_init(accempty, kConvWarps);
        mbar_init(drain, 1);
        mbar_init_fence();
    }
    for (int i = tid; i < NT; i += kThreads)
        xsc[i] = m0 + i < a.M ? __ldg(a.xs + m0 + i) : 0.f;
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *slot, tmem_a = tmem + NT;

    if (warp == kWarpW) {
        Ring<kWStages> w;
        int i = 0;
        for (; i < n; ++i) {
            if (!__all_sync(kFullMask, mbar_poll(b_wempty + 8 * w.s, w.phase ^ 1, cap))) {
                break;
            }
            if (elect_one()) {
                mbar_expect_tx(wfull + w.s, kRows * kTerms);
                tma_2d(base + L::kW + w.s * kRows * kTerms, &wmap, i * kTerms, n0, wfull + w.s);
            }
            w.next();
        }
        for (int j = max(0, i - kWStages); j < i; ++j)      // no copy lands after the block has gone
            mbar_poll(b_wfull + 8 * (j % kWStages), (j / kWStages) & 1, (int)kSpinLimit);
    } else if (warp == kWarpX) {
        Ring<L::kXStages> x;
        int i = 0;
        for (; i < n; ++i) {
            if (!__all_sync(kFullMask, mbar_poll(b_xempty + 8 * x.s, x.phase ^ 1, cap)))
                break;
            if (elect_one()) {
                mbar_expect_tx(xfull + x.s, 2 * L::kXTile);
                for (int b = 0; b < 2; ++b)
                    tma_2d(base + L::kX + (2 * x.s + b) * L::kXTile, &xmap, i * kTerms + 64 * b, m0, xfull + x.s);
            }
            x.next();
        }
        for (int j = max(0, i - L::kXStages); j < i; ++j)
            mbar_poll(b_xfull + 8 * (j % L::kXStages), (j / L::kXStages) & 1, (int)kSpinLimit);
    } else if (warp == kWarpMma) {
        constexpr uint32_t id = idesc_f16(kRows, NT);
        Ring<kABufs> ab;
        Ring<L::kXStages> x;                
        const uint64_t bd0 = desc_sw128(base + L::kX);
        uint32_t chunk = 0;
        int left = kFold;                                   // stages until the accumulator is moved
        int issued = 0;
        for (int i = 0; i < n; ++i) {
            bool ok = mbar_poll(b_afull + 8 * ab.s, ab.phase, cap) && mbar_poll(b_xfull + 8 * x.s, x.phase, cap);
            if (left == kFold)
                ok = ok && mbar_poll(b_accempty, (chunk & 1) ^ 1, cap);
            if (!__all_sync(kFullMask, ok)) {
                break;
            }
            fence_after();
            if (elect_one()) {
                const uint64_t bd = bd0 + x.s * (2 * L::kXTile >> 4);
                const uint32_t at = tmem_a + L::kACols * ab.s;
#pragma unroll
                for (int kk = 0; kk < kTerms / 16; ++kk)
                    mma_f16_ts(tmem, at + 8 * kk, bd + (kk / 4) * (L::kXTile >> 4) + 2 * (kk % 4), id,
                               left != kFold || kk > 0);
                commit_bar(b_aempty + 8 * ab.s);
                commit_bar(b_xempty + 8 * x.s);
                if (left == 1 || i == n - 1)
                    commit_bar(b_accfull);
            }
            __syncwarp();
            ++issued;
            if (--left == 0) {
                left = kFold;
                ++chunk;
            }
            ab.next();
            x.next();
        }
        if (elect_one())
            commit_bar(smem_u32(drain));                    // every product issued is done before TMEM is freed
        __syncwarp();
        mbar_poll(smem_u32(drain), 0, (int)kSpinLimit);
        // ... and every arrival a commit makes has come before the block goes
        for (int j = max(0, issued - kABufs); j < issued; ++j)
            mbar_poll(b_aempty + 8 * (j % kABufs), (j / kABufs) & 1, (int)kSpinLimit);
        for (int j = max(0, issued - L::kXStages); j < issued; ++j)
            mbar_poll(b_xempty + 8 * (j % L::kXStages), (j / L::kXStages) & 1, (int)kSpinLimit);
    } else {
        const int q = warp & 3, half = warp >> 2;           // TMEM lanes 32 q ..; group, and half of the tokens
        const int row = 32 * q + lane;
        const uint32_t lanes = (uint32_t)(32 * q) << 16;
        constexpr int HT = NT / 2;                          // tokens of this thread
        int acc[HT];
        const int chunks = (n + kFold - 1) / kFold;
        const bool ints = chunks > 1;
        if (ints)
#pragma unroll
            for (int j = 0; j < HT; ++j)
                acc[j] = 0;
        int folded = 0;
        bool ok = true;
        // the accumulator into the integers
        constexpr int LC = 32;                              // columns of a TMEM load
        auto fold = [&]() {
            ok = ok && mbar_poll(b_accfull, folded & 1, cap);
            if (__all_sync(kFullMask, ok)) {
                fence_after();
#pragma unroll
                for (int j = 0; j < HT; j += LC) {
                    uint32_t v[LC];
                    tmem_ld32u(v, tmem + lanes + half * HT + j);
#pragma unroll
                    for (int e = 0; e < LC; ++e)
                        acc[j + e] += __float2int_rn(__uint_as_float(v[e]));
                }
                fence_before();
            }
            __syncwarp();
            if (lane == 0)
                arrive_bar(b_accempty);
            ++folded;
        };
        int fold_at = kFold + 2 + half;                     // a stage of each group of the next sum is ready then
        Ring<kWStages> w;
        Ring<kABufs> ab;
        if (half) {
            w.next();
            ab.next();
        }
        for (int i = half; i < n; i += 2) {
            if (i == fold_at) {
                fold();
                fold_at += kFold;
            }
            const uint32_t s = w.s, b = ab.s;
            ok = ok && mbar_poll(b_wfull + 8 * s, w.phase, cap);
            if (!__all_sync(kFullMask, ok)) {
                ok = false;
                break;
            }
            // this thread's weight row, 16-byte chunks of the 128-byte swizzle
            const unsigned char *wr = sm + L::kW + s * kRows * kTerms + row * kTerms;
            uint4 c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                c[j] = *reinterpret_cast<const uint4 *>(wr + ((j ^ (row & 7)) << 4));
            ok = mbar_poll(b_aempty + 8 * b, ab.phase ^ 1, cap);
            if (!__all_sync(kFullMask, ok)) {
                ok = false;
                break;
            }
            fence_after();
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                uint32_t h[16];
                bytes_to_half(c[j].x, h[0], h[1]);
                bytes_to_half(c[j].y, h[2], h[3]);
                bytes_to_half(c[j].z, h[4], h[5]);
                bytes_to_half(c[j].w, h[6], h[7]);
                bytes_to_half(c[j + 1].x, h[8], h[9]);
                bytes_to_half(c[j + 1].y, h[10], h[11]);
                bytes_to_half(c[j + 1].z, h[12], h[13]);
                bytes_to_half(c[j + 1].w, h[14], h[15]);
                tmem_st16u(tmem_a + lanes + L::kACols * b + 8 * j, h);
            }
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) {
                // the bytes are in tensor memory now: only here is their stage given back (given
                // back before the wait above, single rows came out as the next stage's)
                arrive_bar(b_wempty + 8 * s);
                arrive_bar(b_afull + 8 * b);
            }
            w.next();
            w.next();
            ab.next();
            ab.next();
        }
        if (ok)
            while (folded < chunks - 1)
                fold();
        ok = ok && mbar_poll(b_accfull, (chunks - 1) & 1, cap);
        ok = __all_sync(kFullMask, ok);
        fence_after();
        const int c = n0 + row;
        const bool in = c < a.N;
        const float ws = in ? __ldg(a.ws + c) : 0.f, bias = in && a.bias ? __ldg(a.bias + c) : 0.f;
        T *out = static_cast<T *>(a.out) + (long long)(m0 + half * HT) * a.so + c;
        const int left = in ? a.M - m0 - half * HT : 0;     // tokens of this thread that exist
#pragma unroll
        for (int j = 0; j < HT; j += LC) {
            uint32_t v[LC];
            tmem_ld32u(v, tmem + lanes + half * HT + j);
#pragma unroll
            for (int e = 0; e < LC; ++e) {
                float sum = __uint_as_float(v[e]);
                if (ints)
                    sum = __int2float_rn(acc[j + e] + __float2int_rn(sum));
                const float o = ok ? fmaf(sum * xsc[half * HT + j + e], ws, bias) : __int_as_float(0x7fc00000);
                if (j + e < left)
                    *out = from_float<T>(o);
                out += a.so;
            }
        }
        fence_before();
    }
    __syncthreads();
    __syncwarp();
    if (warp == kWarpMma) {
        fence_after();
        tmem_dealloc(tmem, L::kTmem);
    }
}

// Few tokens.  Each weight byte is read once, from HBM into the registers of the lane
// that multiplies it, with no shared memory, barrier or tensor memory between (so
// nothing waits): a warp owns 16 MT channels and every `warps`-th run of kAhead chunks
// of 64 terms, and each lane loads 16 consecutive bytes of 2 MT of its rows, kAhead
// chunks ahead.  In a 16 x 8 x 16 product a lane holds four terms of its rows; which terms
// those are is free as long as both operands agree, so lane t of a quarter takes the
// 16 bytes at 16 t of the chunk, four to a product, and no lane ever needs another's
// bytes.  The tokens are loaded alike; their few rows stay in L1.  Sums leave fp32
// every 1024 terms and are added as integers (in any order: exact) in shared memory,
// where the warps of a block meet.
//
// Measured with weights of 12288 x 4096 from HBM (7.6 us at the copy rate): 13.2 us for
// 1 and 8 tokens, 15.7 for 16, 22.5 for 32.  From 16 tokens on the conversion of the tokens,
// which every warp repeats, is what it waits for (without the products: 15.8 of
// 18.2 us at the time), with 16 warps an SM.
// Runs of four chunks instead of single ones: 16.4 -> 15.7 at 16 tokens; two chunks
// ahead 16.3, eight 16.8; fewer registers (80 a thread) for more warps 18.0.
constexpr int kFewTokens = 64, kChunk = 64, kFewWarps = 16;
constexpr int kFewFold = 1024 / kChunk;
// 33 to 64 tokens: a block of the tile kernel takes 24 us for 4096 terms however few
// channels there are, this kernel 13.5 us for 4096 channels and 37.7 for 12288.  Up to
// 32 tokens it is the faster one at 12288 channels too (23 us against 24).
constexpr int kFewWide = 8192;
constexpr int kFewFill = kSms * 16;             // warps below which a block's share of the terms is split further

struct FewArgs {
    const int8_t *x, *w;                      // rows 16-byte aligned, K a multiple of 16
    const float *xs, *ws, *bias;
    void *out;
    int M, N, K;
    long long sx, sw, so;
};

// 16 weights, each read once: past L1.  Volatile, or the compiler could take it for a function of
// the address alone and move it above the wait for the kernel that packs the weights.
__device__ __forceinline__ uint4 load_once(const int8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <class T, int MT, int NG>                          // 16 MT channels, 8 NG tokens
__global__ void __launch_bounds__(32 * kFewWarps / MT, 1)
int8_few_kernel(const FewArgs a)
{
    griddep_entry();
    constexpr int kAhead = 4 / MT;
    constexpr int C = 16 * MT, CS = C + 4;                  // CS: the sums of a quarter's tokens fall in different banks
    __shared__ int sums[8 * NG * CS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int g = lane >> 2, t = lane & 3, n0 = blockIdx.x * C;
    for (int i = tid; i < 8 * NG * CS; i += blockDim.x)
        sums[i] = 0;
    __syncthreads();

    const int chunks = (a.K + kChunk - 1) / kChunk;
    // A row that is not there stands for row 0 (its sums are not written), and so do
    // tokens past the last term (their weights are zeros).
    const int8_t *wp[2 * MT], *xp[NG];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
        wp[i] = a.w + (n0 + 8 * i + g < a.N ? n0 + 8 * i + g : 0) * a.sw;
#pragma unroll
    for (int j = 0; j < NG; ++j)
        xp[j] = a.x + (8 * j + g < a.M ? 8 * j + g : 0) * a.sx;
    uint4 wv[kAhead][2 * MT], xv[NG];
    auto fetch = [&](uint4 (&v)[2 * MT], int c) {
        const int k = c * kChunk + 16 * t;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
            v[i] = k < a.K ? load_once(wp[i] + k) : make_uint4(0, 0, 0, 0);
    };
    auto token = [&](int j, int c) {
        return __ldg(reinterpret_cast<const uint4 *>(xp[j] + min(c * kChunk + 16 * t, a.K - 16)));
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        fetch(wv[u], warp * kAhead + u);
#pragma unroll
    for (int j = 0; j < NG; ++j)
        xv[j] = token(j, warp * kAhead);

    float acc[MT][NG][4] = {};
    auto fold = [&]() {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NG; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    atomicAdd(sums + (8 * j + 2 * t + (e & 1)) * CS + 16 * i + g + 8 * (e >> 1), __float2int_rn(acc[i][j][e]));
                    acc[i][j][e] = 0.f;
                }
    };
    int left = kFewFold;
    for (int c0 = warp * kAhead; c0 < chunks; c0 += kAhead * warps) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int c = c0 + u;                           // past the end: zeros
            uint32_t h[2 * MT][8];                          // this lane's weights as fp16
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                bytes_to_half(wv[u][i].x, h[i][0], h[i][1]);
                bytes_to_half(wv[u][i].y, h[i][2], h[i][3]);
                bytes_to_half(wv[u][i].z, h[i][4], h[i][5]);
                bytes_to_half(wv[u][i].w, h[i][6], h[i][7]);
            }
            fetch(wv[u], c + kAhead * warps);
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                uint32_t b[8];
                bytes_to_half(xv[j].x, b[0], b[1]);
                bytes_to_half(xv[j].y, b[2], b[3]);
                bytes_to_half(xv[j].z, b[4], b[5]);
                bytes_to_half(xv[j].w, b[6], b[7]);
                xv[j] = token(j, u + 1 < kAhead ? c + 1 : c0 + kAhead * warps);
#pragma unroll
                for (int s = 0; s < 8; s += 2)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        mma_16816(acc[i][j], h[2 * i][s], h[2 * i + 1][s], h[2 * i][s + 1], h[2 * i + 1][s + 1], b[s], b[s + 1]);
            }
        }
        left -= kAhead;
        if (left == 0) {
            fold();
            left = kFewFold;
        }
    }
    if (left != kFewFold)
        fold();
    __syncthreads();
    T *out = static_cast<T *>(a.out);
    for (int i = tid; i < 8 * NG * C; i += blockDim.x) {
        const int m = i / C, c = n0 + i % C;
        if (m < a.M && c < a.N)
            out[m * a.so + c] = from_float<T>(fmaf(__int2float_rn(sums[m * CS + i % C]) * __ldg(a.xs + m), __ldg(a.ws + c),
                                                   a.bias ? __ldg(a.bias + c) : 0.f));
    }
}

// Tokens as rows of `kp` fp16 values, or bytes where `x16` is NULL (blocks below
// `xblocks`), weights as rows of `kp` bytes (the others); 16 values a thread.
struct PackArgs {
    const int8_t *x, *w;
    __half *x16;
    int8_t *xp, *wp;
    int M, N, K, kp;
    long long sx, sw;
    unsigned xblocks;
};

__global__ void __launch_bounds__(256)
int8_pack_kernel(const PackArgs a)
{
    griddep_entry();
    const bool tokens = blockIdx.x < a.xblocks;
    const long long i = (long long)(blockIdx.x - (tokens ? 0 : a.xblocks)) * 256 + threadIdx.x;
    const int per_row = a.kp / 16, rows = tokens ? a.M : a.N;
    const long long r = i / per_row;
    const int k = (int)(i - r * per_row) * 16;
    if (r >= rows)
        return;
    const int8_t *src = (tokens ? a.x + r * a.sx : a.w + r * a.sw) + k;
    uint32_t v[4] = {0, 0, 0, 0};
    if (k + 16 <= a.K && (reinterpret_cast<uintptr_t>(src) & 15) == 0) {
        const uint4 q = *reinterpret_cast<const uint4 *>(src);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (k + e < a.K)
                v[e >> 2] |= (uint32_t)(uint8_t)src[e] << (8 * (e & 3));
    }
    if (tokens && a.x16) {
        uint4 o[2];
        bytes_to_half(v[0], o[0].x, o[0].y);
        bytes_to_half(v[1], o[0].z, o[0].w);
        bytes_to_half(v[2], o[1].x, o[1].y);
        bytes_to_half(v[3], o[1].z, o[1].w);
        uint4 *dst = reinterpret_cast<uint4 *>(a.x16 + r * a.kp + k);
        dst[0] = o[0];
        dst[1] = o[1];
    } else {
        *reinterpret_cast<uint4 *>((tokens ? a.xp : a.wp) + r * a.kp + k) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// [rows][width] of bytes or fp16 in boxes of `terms` x box_rows; zeros outside.
bool encode_rows(CUtensorMap *map, const void *p, bool half, int terms, int width, int rows, long long stride_bytes,
                 int box_rows)
{
    const auto fn = tensor_map_encoder();
    if (!fn)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)terms, (cuuint32_t)box_rows}, step[2] = {1, 1};
    return fn(map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p),
              dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tma_rows(const void *p, long long stride) { return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride) & 15) == 0; }

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Which kernel runs, and what has to be packed for it.
struct Plan {
    bool few, pack_x, pack_w;
    size_t x_bytes, w_bytes;                  // workspace of either
};

Plan plan(const void *x, const void *w, int M, int N, int K, long long sx, long long sw)
{
    Plan p;
    p.few = M <= kFewTokens && (M <= 32 || N < kFewWide);
    // int8_few_kernel loads whole 16-byte words; TMA fills what is past a row's end
    const bool whole = !p.few || K % 16 == 0;
    const size_t kp = ((size_t)K + 15) / 16 * 16;
    p.pack_x = !p.few || !whole || !tma_rows(x, sx);
    p.pack_w = !whole || !tma_rows(w, sw);
    p.x_bytes = p.pack_x ? up256((size_t)M * kp * (p.few ? 1 : 2)) : 0;
    p.w_bytes = p.pack_w ? up256((size_t)N * kp) : 0;
    return p;
}

template <class T, int NT>
cudaError_t launch_tile(const I8Args &a, const CUtensorMap &wmap, const CUtensorMap &xmap, cudaStream_t st)
{
    const auto kernel = int8_tile_kernel<T, NT>;
    const cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kernel), I8Layout<NT>::kTotal);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kernel, dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(kThreads), I8Layout<NT>::kTotal, st, a, wmap, xmap);
}

template <class T, int MT, int NG>
cudaError_t launch_few_shape(const FewArgs &a, cudaStream_t st)
{
    const int blocks = (a.N + 16 * MT - 1) / (16 * MT), chunks = (a.K + kChunk - 1) / kChunk;
    int warps = 4;
    while (warps < kFewWarps / MT && blocks * warps < kFewFill && chunks >= 4 * warps)
        warps *= 2;
    return launch_pdl(int8_few_kernel<T, MT, NG>, dim3((unsigned)blocks), dim3(32 * warps), 0, st, a);
}

template <class T>
cudaError_t launch_few(const FewArgs &a, cudaStream_t st)
{
    if (a.M <= 8)
        return launch_few_shape<T, 1, 1>(a, st);
    if (a.M <= 16)
        return launch_few_shape<T, 1, 2>(a, st);
    if (a.M <= 32)
        return launch_few_shape<T, 1, 4>(a, st);
    return launch_few_shape<T, 2, 8>(a, st);
}

}  // namespace

size_t int8_matmul_workspace_bytes(const void *x, const void *w, int M, int N, int K, long long sx, long long sw)
{
    const Plan p = plan(x, w, M, N, K, sx, sw);
    return p.x_bytes + p.w_bytes;
}

cudaError_t launch_int8_matmul(const int8_t *x, const float *xs, const int8_t *w, const float *ws, const float *bias,
                               void *out, int M, int N, int K, int dtype, long long sx, long long sw, long long so,
                               void *workspace, cudaStream_t st)
{
    const Plan pl = plan(x, w, M, N, K, sx, sw);
    const int kp = (K + 15) / 16 * 16;
    int8_t *xp = static_cast<int8_t *>(workspace), *wp = xp + pl.x_bytes;
    if (pl.pack_x || pl.pack_w) {
        const long long xb = pl.pack_x ? ((long long)M * (kp / 16) + 255) / 256 : 0;
        const long long wb = pl.pack_w ? ((long long)N * (kp / 16) + 255) / 256 : 0;
        const PackArgs p{x, w, pl.few ? nullptr : reinterpret_cast<__half *>(xp), xp, wp, M, N, K, kp, sx, sw, (unsigned)xb};
        const cudaError_t e = launch_pdl(int8_pack_kernel, dim3((unsigned)(xb + wb)), dim3(256), 0, st, p);
        if (e != cudaSuccess)
            return e;
    }
    if (pl.few) {
        const FewArgs a{pl.pack_x ? xp : x, pl.pack_w ? wp : w, xs, ws, bias, out, M, N, kp,
                        pl.pack_x ? kp : sx, pl.pack_w ? kp : sw, so};
        switch (dtype) {
        case kF32: return launch_few<float>(a, st);
        case kBF16: return launch_few<__nv_bfloat16>(a, st);
        case kF16: return launch_few<__half>(a, st);
        default: return cudaErrorInvalidValue;
        }
    }
    // 256 tokens a block, or 128 where that leaves SMs without a block
    const int tiles_n = (N + kRows - 1) / kRows;
    const int nt = (long long)tiles_n * ((M + 255) / 256) < kSms ? 128 : 256;
    // The packed tokens are kp values wide, zeros past the last term: bytes_to_half puts a word's
    // terms in the order 0, 2, 1, 3, so term K - 1 may stand at place K (K = 4 m + 2).  The weights'
    // bytes lie in natural order until the kernel converts them.
    CUtensorMap wmap, xmap;
    if (!encode_rows(&wmap, pl.pack_w ? wp : w, false, kTerms, K, N, pl.pack_w ? kp : sw, kRows) ||
        !encode_rows(&xmap, xp, true, 64, kp, M, (long long)kp * 2, nt))
        return cudaErrorInvalidValue;
    const I8Args a{xs, ws, bias, out, M, N, K, so, (M + nt - 1) / nt, tiles_n, debug_fail_waits() ? 1 : 0};
    switch (dtype) {
    case kF32: return nt == 128 ? launch_tile<float, 128>(a, wmap, xmap, st) : launch_tile<float, 256>(a, wmap, xmap, st);
    case kBF16:
        return nt == 128 ? launch_tile<__nv_bfloat16, 128>(a, wmap, xmap, st)
                         : launch_tile<__nv_bfloat16, 256>(a, wmap, xmap, st);
    case kF16: return nt == 128 ? launch_tile<__half, 128>(a, wmap, xmap, st) : launch_tile<__half, 256>(a, wmap, xmap, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssm
