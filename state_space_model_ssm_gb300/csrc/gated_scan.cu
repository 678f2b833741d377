// Forward kernels of the gated linear recurrence (sm_103a); the mathematics and
// the walk over time are in gated_common.cuh.
#include <climits>

#include "gated_common.cuh"

namespace ssm {

namespace {

// ---- short sequences (decode: one token each; any lengths up to step_most are right) ----
// A thread owns two channels of one sequence and steps through its tokens, four
// tokens' loads at a time: one launch, a handful of loads in flight at once.
template <class T>
__global__ void __launch_bounds__(128)
gated_step_kernel(const GatedArgs a, int pairs)
{
    griddep_entry();
    constexpr int B = 4;
    const int c0 = (blockIdx.x * blockDim.x + threadIdx.x) * 2;
    if (c0 >= a.C)
        return;
    const bool two = c0 + 1 < a.C;
    const float2 lam = make_float2(__ldg(a.lam + c0), two ? __ldg(a.lam + c0 + 1) : 0.f);
    for (int seq = blockIdx.y; seq < a.n_seqs; seq += gridDim.y) {
        long long t0;
        const int len = gated_seq_len(a, seq, t0);
        float *slot = a.state + (long long)seq * a.C + c0;
        float2 h = both(0.f);
        if (a.resume[seq] != 0)
            h = make_float2(slot[0], two ? slot[1] : 0.f);
        if (len > a.step_most)                              // the walk has done it
            continue;
        float2 rate;
        for (int t = 0; t < len; t += B) {
            float2 x[B], ga[B], gx[B];
#pragma unroll
            for (int k = 0; k < B; ++k)
                if (t + k < len) {
                    x[k] = global_pair<T>(a.x, (t0 + t + k) * a.sx + c0, pairs, two);
                    ga[k] = global_pair<T>(a.gate_a, (t0 + t + k) * a.sga + c0, pairs, two);
                    gx[k] = global_pair<T>(a.gate_x, (t0 + t + k) * a.sgx + c0, pairs, two);
                }
            if (t == 0)
                rate = make_float2(a.decay_scale * softplus_f(lam.x), a.decay_scale * softplus_f(lam.y));
            if (a.chunk_states && t % kGatedChunk == 0) {
                float *cs = a.chunk_states + gated_chunk_row(a.n_seqs, seq, t0, t / kGatedChunk) * a.C + c0;
                cs[0] = h.x;
                if (two)
                    cs[1] = h.y;
            }
#pragma unroll
            for (int k = 0; k < B; ++k)
                if (t + k < len) {
                    const Decay d = decay_of(mul2(rate, sigmoid2(ga[k])));
                    h = fma2(d.a, h, mul2(mul2(d.m, sigmoid2(gx[k])), x[k]));
                    store_pair(static_cast<T *>(a.y) + (t0 + t + k) * a.sy + c0, h, pairs, two);
                }
        }
        slot[0] = h.x;
        if (two)
            slot[1] = h.y;
    }
}

// ---- walk over time ----
// Block: 64 channels of one sequence (of one rank of the cluster), 8 warps; a lane
// owns two channels, a warp 8 tokens of the chunk.  Per round: decays and inputs of
// the next chunk from shared memory, the warp's run from zero in registers, the
// runs' maps to the other warps and the chunk's map to the other blocks; then the
// round before: every warp composes the maps before its own onto the carried state
// and stores y.  So the maps travel while the next chunk is worked on (waiting
// for them at once took 2000 of 5400 cycles a round), and TMA fills the stages of
// later chunks.  Two runs in registers: two blocks an SM.
// LONGS: the long sequences of a call of short ones, a block taking one after another.
template <class T, bool TMA>
struct GatedForward {
    static constexpr int kStages = sizeof(T) == 2 ? 3 : 2;  // 24 KB a stage (48 KB for fp32)
    static constexpr size_t kSmem = 128 + kStages * 3 * kGatedTile * sizeof(T);
};

template <class T, bool TMA, bool LONGS>
__device__ __forceinline__ void
gated_walk(const GatedArgs &a, const int seq, const int cb, const int rank, const int pairs, const int words,
           const GatedMap &mx, const GatedMap &mga, const GatedMap &mgx)
{
    constexpr int L = kForwardRun, W = kForwardWarps, S = GatedForward<T, TMA>::kStages;
    extern __shared__ __align__(128) unsigned char raw[];
    T *buf = reinterpret_cast<T *>(align128(raw));
    __shared__ float2 tot_p[3][W][32], tot_h[3][W][32];
    __shared__ uint64_t full[S], exbar[kGatedBufs];
    const GatedExchange ex{reinterpret_cast<GatedMsg *>(buf + S * 3 * kGatedTile), exbar, a.cluster};
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cap = a.fail_waits == 1 ? 0 : (int)tc::kSpinLimit;
    // the exchange's limit after the first round: with the hook at 2 one warp gives up, and the peers soon after
    const int late_cap = a.fail_waits != 2 ? cap : rank == 1 && warp == 3 ? 0 : 1 << 12;
    long long t0;
    const int len = gated_seq_len(a, seq, t0), R = gated_ranks(len, a.cluster);
    if (rank >= R)
        return;
    if (tid == 0) {
        exchange_init(ex);
        for (int i = 0; i < S; ++i)
            tc::mbar_init(&full[i], 1);
        tc::mbar_init_fence();
    }
    gated_cluster_start(R);
    const int rounds = (len + kGatedChunk * R - 1) / (kGatedChunk * R);
    uint32_t filled = 0, fill_parity = 0;                   // (thread 0) by stage: filled at all; an odd number of times
    auto fetch = [&](int k) {                               // round k's rows into its stage
        const int j = k * R + rank, t = (int)t0 + j * kGatedChunk, n = min(kGatedChunk, len - j * kGatedChunk);
        T *to = buf + k % S * 3 * kGatedTile;
        if (TMA) {
            if (tid == 0 && n > 0) {
                uint64_t *bar = &full[k % S];
                filled |= 1u << (k % S);
                fill_parity ^= 1u << (k % S);
                tc::mbar_expect_tx(bar, 3 * kGatedTile * sizeof(T));
                tma_rows(to, &mx, cb * kGatedCh, t, bar);
                tma_rows(to + kGatedTile, &mga, cb * kGatedCh, t, bar);
                tma_rows(to + 2 * kGatedTile, &mgx, cb * kGatedCh, t, bar);
            }
        } else if (n > 0) {
            gated_copy<T>(to, a.x, a.sx, t, n, cb * kGatedCh, a.C, words);
            gated_copy<T>(to + kGatedTile, a.gate_a, a.sga, t, n, cb * kGatedCh, a.C, words);
            gated_copy<T>(to + 2 * kGatedTile, a.gate_x, a.sgx, t, n, cb * kGatedCh, a.C, words);
        }
        if (!TMA)
            cp_async_commit();
    };
    for (int k = 0; k < S; ++k)
        if (k < rounds)
            fetch(k);
    const int c0 = cb * kGatedCh + 2 * lane;
    const bool inside = c0 < a.C, two = c0 + 1 < a.C;
    float2 rate = both(0.f), s = both(0.f);                 // s: the state entering the round
    if (inside) {
        rate = make_float2(a.decay_scale * softplus_f(__ldg(a.lam + c0)),
                           two ? a.decay_scale * softplus_f(__ldg(a.lam + c0 + 1)) : 0.f);
        if (a.resume[seq] != 0) {
            const float *slot = a.state + (long long)seq * a.C + c0;
            s = make_float2(slot[0], two ? slot[1] : 0.f);
        }
    }
    // ok: no wait of this thread gave up; live: none of the block's had at the last barrier, so
    // the whole block goes on or stops by it (one warp may give up in a round that others finish)
    bool ok = true, live = true;
    // round k's run from zero: h[i] and the product of decays p[i] up to token i; its maps sent
    auto begin = [&](int k, float2 (&h)[L], float2 (&p)[L]) {
        const int j = k * R + rank;                         // this block's chunk
        const int cnt = min(L, len - j * kGatedChunk - warp * L);
        const T *bx = buf + k % S * 3 * kGatedTile, *bga = bx + kGatedTile, *bgx = bga + kGatedTile;
        if (TMA) {
            if (len > j * kGatedChunk)
                ok = ok && gated_wait(&full[k % S], (k / S) & 1, cap);
        } else {
            if (k + S - 1 < rounds)
                cp_async_wait<S - 1>();
            else
                cp_async_wait<0>();
            __syncthreads();
        }
        const int at = warp * L * kGatedCh + 2 * lane;
        float2 hh = both(0.f), pp = both(1.f);
        auto run = [&](auto whole, auto low) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (whole.value || i < cnt) {
                    float2 r, g;
                    gates2<low.value>(load_pair(bga + at + i * kGatedCh), load_pair(bgx + at + i * kGatedCh), r, g);
                    const Decay d = decay_of(mul2(rate, r));
                    hh = fma2(d.a, hh, mul2(mul2(d.m, g), load_pair(bx + at + i * kGatedCh)));
                    pp = mul2(pp, d.a);
                }
                h[i] = hh;
                p[i] = pp;
            }
        };
        if (cnt >= L && gates_above<T, L>(bga + at, bgx + at))
            run(Flag<true>(), Flag<false>());
        else
            run(Flag<false>(), Flag<true>());
        tot_p[k % 3][warp][lane] = pp;
        tot_h[k % 3][warp][lane] = hh;
        ok = live = __syncthreads_and(ok);                  // the runs' maps are there, the stage is read
        if (live && k + S < rounds)
            fetch(k + S);
        if (live && R > 1 && warp == 0) {
            GatedMsg m{both(1.f), both(0.f)};
#pragma unroll
            for (int w = 0; w < W; ++w) {
                m.h = fma2(tot_p[k % 3][w][lane], m.h, tot_h[k % 3][w][lane]);
                m.p = mul2(m.p, tot_p[k % 3][w][lane]);
            }
            exchange_send(ex, k, rank, R, lane, m);
        }
    };
    // round k's states and its y
    auto finish = [&](int k, const float2 (&h)[L], const float2 (&p)[L]) {
        const int j = k * R + rank;
        const int cnt = min(L, len - j * kGatedChunk - warp * L);
        float2 mine = s, next = s;                          // the states entering this block's chunk and the next round
        if (R > 1) {
            ok = ok && exchange_wait(ex, k, k > 0 ? late_cap : cap);
            __syncwarp();
#pragma unroll
            for (int r = 0; r < kGatedMaxCluster; ++r)
                if (r < R) {
                    if (r == rank)
                        mine = next;
                    const GatedMsg &m = ex.at(k, r, lane);
                    next = fma2(m.p, next, m.h);
                }
        }
        if (!ok)
            mine = next = both(__int_as_float(0x7fc00000)); // a wait gave up: seen in y and in the slot
        if (a.chunk_states && warp == 0 && inside && len > j * kGatedChunk) {
            float *cs = a.chunk_states + gated_chunk_row(a.n_seqs, seq, t0, j) * a.C + c0;
            cs[0] = mine.x;
            if (two)
                cs[1] = mine.y;
        }
        float2 run_s = mine;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == warp)
                run_s = mine;
            mine = fma2(tot_p[k % 3][w][lane], mine, tot_h[k % 3][w][lane]);
        }
        s = R > 1 ? next : mine;
        if (inside) {
            T *y = static_cast<T *>(a.y) + (t0 + j * (long long)kGatedChunk + warp * L) * a.sy + c0;
            if (cnt >= L && pairs) {
#pragma unroll
                for (int i = 0; i < L; ++i)
                    store_pair(y + i * a.sy, fma2(p[i], run_s, h[i]), true, true);
            } else {
#pragma unroll
                for (int i = 0; i < L; ++i)
                    if (i < cnt)
                        store_pair(y + i * a.sy, fma2(p[i], run_s, h[i]), pairs, two);
            }
        }
    };
    float2 h0[L], p0[L], h1[L], p1[L];
    int done = 0;
    if (rounds > 0)
        begin(0, h0, p0);
    for (; done < rounds && live; done += 2) {
        if (done + 1 < rounds)
            begin(done + 1, h1, p1);
        if (!live)
            break;
        finish(done, h0, p0);
        if (done + 1 < rounds) {
            if (done + 2 < rounds)
                begin(done + 2, h0, p0);
            if (!live)
                break;
            finish(done + 1, h1, p1);
        }
    }
    ok = __syncthreads_and(ok);
    if (!ok) {                                              // a wait gave up: NaN, once the copies in flight have landed
        s = both(__int_as_float(0x7fc00000));
        gated_poison(static_cast<T *>(a.y), a.sy, t0, len, (done > 2 ? done - 2 : 0) * R + rank, R, cb * kGatedCh, a.C);
        if (TMA && tid == 0)
            for (int i = 0; i < S; ++i)
                if (filled >> i & 1)
                    gated_wait(&full[i], (fill_parity >> i & 1) ^ 1, (int)tc::kSpinLimit);
        if (!TMA)
            cp_async_wait<0>();
        __syncthreads();
    }
    if (rank == 0 && warp == 0 && inside) {                 // (an empty sequence: what it began with)
        float *slot = a.state + (long long)seq * a.C + c0;
        slot[0] = s.x;
        if (two)
            slot[1] = s.y;
    }
    gated_cluster_end(R, ok);
    if (LONGS) {                                            // the barriers' places for the next sequence
        __syncthreads();
        if (tid == 0) {
            for (int i = 0; i < S; ++i)
                mbar_inval(&full[i]);
            for (int i = 0; i < kGatedBufs; ++i)
                mbar_inval(&exbar[i]);
        }
    }
}

template <class T, bool TMA, bool LONGS>
__global__ void __launch_bounds__(32 * kForwardWarps, 2)
gated_scan_kernel(const GatedArgs a, int pairs, int words, const __grid_constant__ GatedMap mx,
                  const __grid_constant__ GatedMap mga, const __grid_constant__ GatedMap mgx)
{
    griddep_entry();
    if constexpr (LONGS) {
        __shared__ uint32_t masks[GatedLongs<kForwardWarps>::kEach][kForwardWarps];
        GatedLongs<kForwardWarps> longs{masks};
        for (long long u = blockIdx.x;; u += gridDim.x) {
            const int seq = longs.find(a, u / a.cblocks);
            if (seq < 0)
                return;
            gated_walk<T, TMA, true>(a, seq, (int)(u % a.cblocks), 0, pairs, words, mx, mga, mgx);
        }
    } else {
        const int rank = blockIdx.x % a.cluster, job = blockIdx.x / a.cluster;
        gated_walk<T, TMA, false>(a, gated_job_seq(a, job / a.cblocks, threadIdx.x & 31), job % a.cblocks, rank, pairs, words,
                                  mx, mga, mgx);
    }
}

// The walk over every sequence, or over the long ones of a call of short ones.
template <class T, bool LONGS>
cudaError_t launch_walk(const GatedArgs &a, bool pairs, int dtype, cudaStream_t stream)
{
    const unsigned blocks = LONGS ? gated_mixed_blocks(a) : gated_walk_blocks(a);
    GatedMap mx, mga, mgx;
    if (gated_map(&mx, a.x, dtype, a.n_tokens, a.C, a.sx) && gated_map(&mga, a.gate_a, dtype, a.n_tokens, a.C, a.sga) &&
        gated_map(&mgx, a.gate_x, dtype, a.n_tokens, a.C, a.sgx))
        return launch_clusters(gated_scan_kernel<T, true, LONGS>, a, blocks, kForwardWarps,
                               GatedForward<T, true>::kSmem + gated_exchange_bytes(a.cluster), stream, a, pairs ? 1 : 0, 0,
                               mx, mga, mgx);
    const bool words = gated_words(a.x, dtype, a.C, a.sx) && gated_words(a.gate_a, dtype, a.C, a.sga) &&
                       gated_words(a.gate_x, dtype, a.C, a.sgx);
    return launch_clusters(gated_scan_kernel<T, false, LONGS>, a, blocks, kForwardWarps,
                           GatedForward<T, false>::kSmem + gated_exchange_bytes(a.cluster), stream, a, pairs ? 1 : 0,
                           words ? 1 : 0, mx, mga, mgx);
}

// pairs: y's rows take pairs; all: those of every tensor (the stepping kernel loads them too).
template <class T>
cudaError_t launch_forward(GatedArgs a, bool pairs, bool all, int dtype, cudaStream_t stream)
{
    if (!gated_short(a))
        return launch_walk<T, false>(a, pairs, dtype, stream);
    if (gated_mixed(a)) {
        a.step_most = kGatedStep;
        const cudaError_t e = launch_walk<T, true>(a, pairs, dtype, stream);
        if (e != cudaSuccess)
            return e;
    }
    const dim3 grid((unsigned)((a.C + 255) / 256), (unsigned)(a.n_seqs < 65535 ? a.n_seqs : 65535));
    return launch_pdl(gated_step_kernel<T>, grid, dim3(128), 0, stream, a, all ? 1 : 0);
}

}  // namespace

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

long long gated_chunk_rows(long long n_seqs, long long n_tokens) { return n_seqs + n_tokens / kGatedChunk + 1; }

// As many blocks a sequence as fit the device at once (two an SM; one where fp32
// stages and the exchange of four or more blocks fill shared memory), and at
// most one for every two chunks it has on average.  The lengths are not known here: of
// more than four sequences a sixth are taken to be long.  Forward / backward in us
// with 1, 2, 4, 8 blocks (64 channel blocks unless stated):
//   1 x 4096 bf16                88 55 44 51     225 129 104 109
//   12 uneven, 7889 tokens bf16  131 81 93 120   255 184 192 236
//   4 x 16384 fp32, 32 blocks    346 312 407 499 1186 795 801 817
//   32 x 512 bf16, 32 blocks     69 89 113 180   158 185 217 292
//   1 x 16384 bf16, 1 block      338 203 104 56  876 490 255 138
int gated_cluster(int n_seqs, int n_tokens, int C, bool wide)
{
    const long long cb = (C + kGatedCh - 1) / kGatedCh, chunks = (long long)n_tokens / n_seqs / kGatedChunk;
    const long long uneven = n_seqs <= 4 ? n_seqs : n_seqs / 6 > 2 ? n_seqs / 6 : 2;
    int r = 1;
    while (r < kGatedMaxCluster && 4 * r <= chunks && uneven * cb * 2 * r <= (wide && r >= 2 ? kSms : 2 * kSms))
        r *= 2;
    return r;
}

bool gated_map(GatedMap *map, const void *p, int dtype, int n_tokens, int C, long long stride)
{
    const auto fn = tensor_map_encoder();
    const long long bytes = stride * dtype_size(dtype);
    static_assert(sizeof(CUtensorMap) == sizeof(map->image), "tensor map size");
    if (!fn || n_tokens <= 0 || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)bytes) & 15) != 0 || bytes >= 1LL << 40)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)C, (cuuint64_t)n_tokens};
    const cuuint64_t strides[1] = {(cuuint64_t)bytes};
    const cuuint32_t box[2] = {kGatedCh, kGatedChunk}, step[2] = {1, 1};
    const CUtensorMapDataType type = dtype == kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(reinterpret_cast<CUtensorMap *>(map->image), type, 2, const_cast<void *>(p), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool gated_words(const void *p, int dtype, int C, long long stride)
{
    return dtype == kF32 || (((C | stride) & 1) == 0 && (reinterpret_cast<uintptr_t>(p) & 3) == 0);
}

cudaError_t launch_gated_scan(GatedArgs a, int dtype, cudaStream_t stream)
{
    a.cblocks = (a.C + kGatedCh - 1) / kGatedCh;
    a.cluster = gated_cluster(a.n_seqs, a.n_tokens, a.C, dtype == kF32);
    a.fail_waits = debug_fail_waits();
    a.step_most = INT_MAX;
    const bool pairs = ((a.C | a.sy) & 1) == 0 && reinterpret_cast<uintptr_t>(a.y) % (2 * dtype_size(dtype)) == 0;
    const bool all = pairs && ((a.sx | a.sga | a.sgx) & 1) == 0 &&
                     ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.gate_a) |
                       reinterpret_cast<uintptr_t>(a.gate_x)) % (2 * dtype_size(dtype))) == 0;
    switch (dtype) {
    case kF32: return launch_forward<float>(a, pairs, all, dtype, stream);
    case kBF16: return launch_forward<__nv_bfloat16>(a, pairs, all, dtype, stream);
    case kF16: return launch_forward<__half>(a, pairs, all, dtype, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssm
