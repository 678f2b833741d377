// Backward kernel of the gated linear recurrence (sm_103a); the mathematics of
// the forward pass and the walk over time are in gated_common.cuh.
//
// With g_t the gradient of h_t through y_t and everything after it, and
// E_t = a_t g_t what token t passes to the token before:
//
//   g_t = dy_t + E_{t+1}          (the last token: dy_t + the slot's gradient)
//   d log a = g (a h_{t-1} - (a^2 / m) i x)           [dm / d log a = -a^2 / m]
//   dx = g m i,  dgate_x = g m x i (1 - i),  dgate_a = (d log a) log a (1 - r)
//   dlam = sum_t (d log a) r * (-decay_scale sigmoid(lam)),  d slot before = E_first
//
// E of a run of tokens is an affine map of the E arriving from after it, with the
// same product of decays P as the forward map: E_first = P E_in + sum_t p_t dy_t,
// p_t the product of the decays up to and including t.  So one pass over a
// thread's tokens gives P, H and E.  The state entering a chunk was saved by the
// forward pass (fp32: h is recomputed in registers instead of read back rounded);
// E is carried from the last chunk to the first as the forward kernel carries h.
#include <climits>

#include "gated_common.cuh"

namespace ssm {

namespace {

// The chunk's rows stay in shared memory for both passes over them (the gates are
// computed twice: their registers would cost half the resident blocks).  Two stages
// of 32 KB for 16-bit types; fp32 rows take 64 KB, there one stage.  Two blocks an SM
// in either case (512 threads of 64 registers), the other of which covers the wait.
template <class T>
struct GatedBackward {
    static constexpr int kStages = sizeof(T) == 2 ? 2 : 1;
    static constexpr size_t kSmem = 128 + kStages * 4 * kGatedTile * sizeof(T);
};

// LONGS: the long sequences of a call of short ones, a block taking one after another.
template <class T, bool TMA, bool LONGS>
__device__ __forceinline__ void
gated_walk_back(const GatedArgs &a, const int seq, const int cb, const int rank, const int pairs, const int words,
                const GatedMap &mx, const GatedMap &mga, const GatedMap &mgx, const GatedMap &mdy)
{
    constexpr int L = kBackwardRun, W = kBackwardWarps, S = GatedBackward<T>::kStages;
    extern __shared__ __align__(128) unsigned char raw[];
    T *buf = reinterpret_cast<T *>(align128(raw));
    __shared__ float2 tot_p[W][32], tot_h[W][32], tot_e[W][32], enter[W][32], arrive[W][32];
    __shared__ uint64_t full[S], exbar[kGatedBufs];
    const GatedExchange ex{reinterpret_cast<GatedMsg *>(buf + S * 4 * kGatedTile), exbar, a.cluster};
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cap = a.fail_waits == 1 ? 0 : (int)tc::kSpinLimit;
    // as in the forward kernel (one warp waits for the block here)
    const int late_cap = a.fail_waits != 2 ? cap : rank == 1 ? 0 : 1 << 12;
    long long t0;
    const int len = gated_seq_len(a, seq, t0), R = gated_ranks(len, a.cluster);
    if (rank >= R) {                                        // this rank's share of dlam
        if (warp == 0)
            for (int c = cb * kGatedCh + lane; c < min(a.C, (cb + 1) * kGatedCh); c += 32)
                a.lam_part[((long long)seq * a.cluster + rank) * a.C + c] = 0.f;
        return;
    }
    if (tid == 0) {
        exchange_init(ex);
        for (int i = 0; i < S; ++i)
            tc::mbar_init(&full[i], 1);
        tc::mbar_init_fence();
    }
    gated_cluster_start(R);
    const int rounds = (len + kGatedChunk * R - 1) / (kGatedChunk * R);
    // the chunk of this block's n-th round, the last tokens first (it may lie past the end: no tokens)
    auto chunk_of = [&](int n) { return (rounds - 1 - n) * R + rank; };
    uint32_t phases = 0;                                    // parity of each stage's next fill
    uint32_t filled = 0, fill_parity = 0;                   // (thread 0) by stage: filled at all; an odd number of times
    auto fetch = [&](int k) {
        const int j = chunk_of(k), t = (int)t0 + j * kGatedChunk, n = min(kGatedChunk, len - j * kGatedChunk);
        T *to = buf + k % S * 4 * kGatedTile;
        if (TMA) {
            if (tid == 0 && n > 0) {
                uint64_t *bar = &full[k % S];
                filled |= 1u << (k % S);
                fill_parity ^= 1u << (k % S);
                tc::mbar_expect_tx(bar, 4 * kGatedTile * sizeof(T));
                tma_rows(to, &mx, cb * kGatedCh, t, bar);
                tma_rows(to + kGatedTile, &mga, cb * kGatedCh, t, bar);
                tma_rows(to + 2 * kGatedTile, &mgx, cb * kGatedCh, t, bar);
                tma_rows(to + 3 * kGatedTile, &mdy, cb * kGatedCh, t, bar);
            }
        } else {
            if (n > 0) {
                gated_copy<T>(to, a.x, a.sx, t, n, cb * kGatedCh, a.C, words);
                gated_copy<T>(to + kGatedTile, a.gate_a, a.sga, t, n, cb * kGatedCh, a.C, words);
                gated_copy<T>(to + 2 * kGatedTile, a.gate_x, a.sgx, t, n, cb * kGatedCh, a.C, words);
                gated_copy<T>(to + 3 * kGatedTile, a.grad_y, a.sy, t, n, cb * kGatedCh, a.C, words);
            }
            cp_async_commit();
        }
    };
    if (rounds > 0)
        fetch(0);
    const int c0 = cb * kGatedCh + 2 * lane;
    const bool inside = c0 < a.C, two = c0 + 1 < a.C;
    float2 rate = both(0.f), s = both(0.f), part = both(0.f);   // s: the E arriving at the round; part: dlam's sum
    if (inside) {
        rate = make_float2(a.decay_scale * softplus_f(__ldg(a.lam + c0)),
                           two ? a.decay_scale * softplus_f(__ldg(a.lam + c0 + 1)) : 0.f);
        if (a.grad_state) {
            const float *g = a.grad_state + (long long)seq * a.C + c0;
            s = make_float2(g[0], two ? g[1] : 0.f);
        }
    }
    bool ok = true;
    int k = 0;
    for (; k < rounds; ++k) {
        const int j = chunk_of(k);
        const bool some = len > j * kGatedChunk;            // this block's chunk has tokens
        const int cnt = min(L, len - j * kGatedChunk - warp * L);
        const T *bx = buf + k % S * 4 * kGatedTile, *bga = bx + kGatedTile, *bgx = bga + kGatedTile,
                *bdy = bgx + kGatedTile;
        if (TMA) {
            if (some) {
                ok = ok && gated_wait(&full[k % S], (phases >> (k % S)) & 1, cap);
                phases ^= 1u << (k % S);
            }
        } else {
            cp_async_wait<0>();
            __syncthreads();
        }
        // decays dec[i] and inputs hb[i] of the run; its maps of h and of E
        float2 dec[L], hb[L], hh = both(0.f), pp = both(1.f), ee = both(0.f);
        auto run = [&](auto whole, auto low) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                dec[i] = both(1.f);
                hb[i] = both(0.f);
                if (whole.value || i < cnt) {
                    const int at = (warp * L + i) * kGatedCh + 2 * lane;
                    float2 r, g;
                    gates2<low.value>(load_pair(bga + at), load_pair(bgx + at), r, g);
                    const Decay d = decay_of(mul2(rate, r));
                    hb[i] = mul2(mul2(d.m, g), load_pair(bx + at));
                    dec[i] = d.a;
                    hh = fma2(d.a, hh, hb[i]);
                    pp = mul2(pp, d.a);
                    ee = fma2(pp, load_pair(bdy + at), ee);
                }
            }
        };
        const bool fast = cnt >= L && gates_above<T, L>(bga + warp * L * kGatedCh + 2 * lane, bgx + warp * L * kGatedCh + 2 * lane);
        if (fast)
            run(Flag<true>(), Flag<false>());
        else
            run(Flag<false>(), Flag<true>());
        tot_p[warp][lane] = pp;
        tot_h[warp][lane] = hh;
        tot_e[warp][lane] = ee;
        ok = __syncthreads_and(ok);                         // the runs' maps are there, the round before is done
        if (!ok)
            break;
        if (S == 2 && k + 1 < rounds)
            fetch(k + 1);
        if (warp == 1) {                                    // the states entering the runs
            float2 h = both(0.f);
            if (inside && some) {
                const float *cs = a.chunk_states + gated_chunk_row(a.n_seqs, seq, t0, j) * a.C + c0;
                h = make_float2(__ldg(cs), two ? __ldg(cs + 1) : 0.f);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                enter[w][lane] = h;
                h = fma2(tot_p[w][lane], h, tot_h[w][lane]);
            }
        }
        if (warp == 0) {
            float2 mine = s, next = s;                      // the E arriving at this block's chunk and at the next round
            if (R > 1) {
                GatedMsg m{both(1.f), both(0.f)};
#pragma unroll
                for (int w = W - 1; w >= 0; --w) {
                    m.h = fma2(tot_p[w][lane], m.h, tot_e[w][lane]);
                    m.p = mul2(m.p, tot_p[w][lane]);
                }
                exchange_send(ex, k, rank, R, lane, m);
                ok = ok && exchange_wait(ex, k, k > 0 ? late_cap : cap);
                __syncwarp();
                for (int r = R - 1; r >= 0; --r) {
                    if (r == rank)
                        mine = next;
                    next = fma2(ex.at(k, r, lane).p, next, ex.at(k, r, lane).h);
                }
            }
            if (!ok)
                mine = next = both(__int_as_float(0x7fc00000));
#pragma unroll
            for (int w = W - 1; w >= 0; --w) {              // the E arriving at the runs
                arrive[w][lane] = mine;
                mine = fma2(tot_p[w][lane], mine, tot_e[w][lane]);
            }
            s = R > 1 ? next : mine;
        }
        __syncthreads();
        float2 h = enter[warp][lane], E = arrive[warp][lane];
#pragma unroll
        for (int i = 0; i < L; ++i) {                       // hb[i]: b_i -> h_{i-1}
            const float2 before = h;
            h = fma2(dec[i], h, hb[i]);
            hb[i] = before;
        }
        const long long t = t0 + j * (long long)kGatedChunk + warp * L;
        T *ox = static_cast<T *>(a.grad_x) + t * a.gsx + c0;
        T *oa = static_cast<T *>(a.grad_ga) + t * a.gsga + c0;
        T *og = static_cast<T *>(a.grad_gx) + t * a.gsgx + c0;
        auto gradients = [&](auto whole, auto low) {
#pragma unroll
            for (int i = L - 1; i >= 0; --i)
                if (whole.value || i < cnt) {
                    const int at = (warp * L + i) * kGatedCh + 2 * lane;
                    const float2 g = add2(load_pair(bdy + at), E);
                    E = mul2(dec[i], g);
                    float2 r, gi;
                    gates2<low.value>(load_pair(bga + at), load_pair(bgx + at), r, gi);
                    const float2 v = mul2(rate, r);
                    const Decay d = decay_of(v);
                    const float2 ix = mul2(gi, load_pair(bx + at)), gm = mul2(g, d.m);
                    // d log a = g (a h - a^2 ix / m)
                    const float2 dla = mul2(mul2(g, d.a), fma2(mul2(d.a, d.im), make_float2(-ix.x, -ix.y), hb[i]));
                    part = fma2(dla, r, part);
                    if (inside) {
                        store_pair(ox + i * a.gsx, mul2(gm, gi), pairs, two);
                        store_pair(og + i * a.gsgx, mul2(gm, fma2(make_float2(-ix.x, -ix.y), gi, ix)), pairs, two);
                        store_pair(oa + i * a.gsga, mul2(dla, fma2(v, r, make_float2(-v.x, -v.y))), pairs, two);
                    }
                }
        };
        if (fast)
            gradients(Flag<true>(), Flag<false>());
        else
            gradients(Flag<false>(), Flag<true>());
        if (S == 1 && k + 1 < rounds) {
            __syncthreads();                                // the stage is read
            fetch(k + 1);
        }
    }
    ok = __syncthreads_and(ok);
    if (!ok) {                                              // a wait gave up: NaN, once the copies in flight have landed
        s = part = both(__int_as_float(0x7fc00000));
        const int from = chunk_of(k > 0 ? k - 1 : 0);
        gated_poison(static_cast<T *>(a.grad_x), a.gsx, t0, len, from, -R, cb * kGatedCh, a.C);
        gated_poison(static_cast<T *>(a.grad_ga), a.gsga, t0, len, from, -R, cb * kGatedCh, a.C);
        gated_poison(static_cast<T *>(a.grad_gx), a.gsgx, t0, len, from, -R, cb * kGatedCh, a.C);
        if (TMA && tid == 0)
            for (int i = 0; i < S; ++i)
                if (filled >> i & 1)
                    gated_wait(&full[i], (fill_parity >> i & 1) ^ 1, (int)tc::kSpinLimit);
        if (!TMA)
            cp_async_wait<0>();
        __syncthreads();
    }
    if (rank == 0 && warp == 0 && inside && a.grad_state0) {
        const bool resume = a.resume[seq] != 0;
        float *g = a.grad_state0 + (long long)seq * a.C + c0;
        g[0] = resume ? s.x : 0.f;
        if (two)
            g[1] = resume ? s.y : 0.f;
    }
    __syncthreads();
    tot_p[warp][lane] = part;
    __syncthreads();
    if (warp == 0 && inside) {
        float2 sum = both(0.f);
#pragma unroll
        for (int w = 0; w < W; ++w)
            sum = add2(sum, tot_p[w][lane]);
        float *to = a.lam_part + ((long long)seq * a.cluster + rank) * a.C + c0;
        to[0] = sum.x;
        if (two)
            to[1] = sum.y;
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
__global__ void __launch_bounds__(32 * kBackwardWarps, 2)
gated_scan_backward_kernel(const GatedArgs a, int pairs, int words, const __grid_constant__ GatedMap mx,
                           const __grid_constant__ GatedMap mga, const __grid_constant__ GatedMap mgx,
                           const __grid_constant__ GatedMap mdy)
{
    griddep_entry();
    if constexpr (LONGS) {
        __shared__ uint32_t masks[GatedLongs<kBackwardWarps>::kEach][kBackwardWarps];
        GatedLongs<kBackwardWarps> longs{masks};
        for (long long u = blockIdx.x;; u += gridDim.x) {
            const int seq = longs.find(a, u / a.cblocks);
            if (seq < 0)
                return;
            gated_walk_back<T, TMA, true>(a, seq, (int)(u % a.cblocks), 0, pairs, words, mx, mga, mgx, mdy);
        }
    } else {
        const int rank = blockIdx.x % a.cluster, job = blockIdx.x / a.cluster;
        gated_walk_back<T, TMA, false>(a, gated_job_seq(a, job / a.cblocks, threadIdx.x & 31), job % a.cblocks, rank, pairs,
                                       words, mx, mga, mgx, mdy);
    }
}

// ---- short sequences ----
// A thread owns two channels of one sequence.  From the last chunk to the first it
// steps h through the chunk, keeping the state before every fourth token, and then
// takes the fours from the last to the first: their decays and inputs again, and
// the gradients.
template <class T>
__global__ void __launch_bounds__(128)
gated_step_backward_kernel(const GatedArgs a, int pairs)
{
    griddep_entry();
    constexpr int B = 4, RUNS = kGatedChunk / B;
    const int c0 = (blockIdx.x * blockDim.x + threadIdx.x) * 2;
    if (c0 >= a.C)
        return;
    const bool two = c0 + 1 < a.C;
    const float2 rate = make_float2(a.decay_scale * softplus_f(__ldg(a.lam + c0)),
                                    two ? a.decay_scale * softplus_f(__ldg(a.lam + c0 + 1)) : 0.f);
    for (int seq = blockIdx.y; seq < a.n_seqs; seq += gridDim.y) {
        long long t0;
        const int len = gated_seq_len(a, seq, t0);
        float2 E = both(0.f), part = both(0.f);
        if (a.grad_state) {
            const float *g = a.grad_state + (long long)seq * a.C + c0;
            E = make_float2(g[0], two ? g[1] : 0.f);
        }
        if (len > a.step_most)                              // the walk has done it
            continue;
        for (int j = (len + kGatedChunk - 1) / kGatedChunk - 1; j >= 0; --j) {
            const long long tc = t0 + (long long)j * kGatedChunk;
            const int n = min(kGatedChunk, len - j * kGatedChunk), runs = (n + B - 1) / B;
            const float *cs = a.chunk_states + gated_chunk_row(a.n_seqs, seq, t0, j) * a.C + c0;
            float2 h = make_float2(__ldg(cs), two ? __ldg(cs + 1) : 0.f), entry[RUNS];
#pragma unroll 1
            for (int r = 0; r < runs; ++r) {
                entry[r] = h;
                if (r + 1 == runs)
                    break;
                float2 x[B], ga[B], gx[B];
#pragma unroll
                for (int k = 0; k < B; ++k) {
                    const long long t = tc + r * B + k;
                    x[k] = global_pair<T>(a.x, t * a.sx + c0, pairs, two);
                    ga[k] = global_pair<T>(a.gate_a, t * a.sga + c0, pairs, two);
                    gx[k] = global_pair<T>(a.gate_x, t * a.sgx + c0, pairs, two);
                }
#pragma unroll
                for (int k = 0; k < B; ++k) {
                    const Decay d = decay_of(mul2(rate, sigmoid2(ga[k])));
                    h = fma2(d.a, h, mul2(mul2(d.m, sigmoid2(gx[k])), x[k]));
                }
            }
#pragma unroll 1
            for (int r = runs - 1; r >= 0; --r) {
                const int cnt = min(B, n - r * B);
                float2 x[B], ga[B], gx[B], dy[B], before[B];
#pragma unroll
                for (int k = 0; k < B; ++k)
                    if (k < cnt) {
                        const long long t = tc + r * B + k;
                        x[k] = global_pair<T>(a.x, t * a.sx + c0, pairs, two);
                        ga[k] = global_pair<T>(a.gate_a, t * a.sga + c0, pairs, two);
                        gx[k] = global_pair<T>(a.gate_x, t * a.sgx + c0, pairs, two);
                        dy[k] = global_pair<T>(a.grad_y, t * a.sy + c0, pairs, two);
                    }
                h = entry[r];
                Decay d[B];
#pragma unroll
                for (int k = 0; k < B; ++k)
                    if (k < cnt) {
                        before[k] = h;
                        ga[k] = sigmoid2(ga[k]);
                        gx[k] = sigmoid2(gx[k]);
                        d[k] = decay_of(mul2(rate, ga[k]));
                        h = fma2(d[k].a, h, mul2(mul2(d[k].m, gx[k]), x[k]));
                    }
#pragma unroll
                for (int k = B - 1; k >= 0; --k)
                    if (k < cnt) {
                        const long long t = tc + r * B + k;
                        const float2 g = add2(dy[k], E), v = mul2(rate, ga[k]);
                        E = mul2(d[k].a, g);
                        const float2 ix = mul2(gx[k], x[k]), gm = mul2(g, d[k].m);
                        const float2 dla = mul2(E, fma2(mul2(d[k].a, d[k].im), make_float2(-ix.x, -ix.y), before[k]));
                        part = fma2(dla, ga[k], part);
                        store_pair(static_cast<T *>(a.grad_x) + t * a.gsx + c0, mul2(gm, gx[k]), pairs, two);
                        store_pair(static_cast<T *>(a.grad_gx) + t * a.gsgx + c0,
                                   mul2(gm, fma2(make_float2(-ix.x, -ix.y), gx[k], ix)), pairs, two);
                        store_pair(static_cast<T *>(a.grad_ga) + t * a.gsga + c0,
                                   mul2(dla, fma2(v, ga[k], make_float2(-v.x, -v.y))), pairs, two);
                    }
            }
        }
        if (a.grad_state0) {
            const bool resume = a.resume[seq] != 0;
            float *g = a.grad_state0 + (long long)seq * a.C + c0;
            g[0] = resume ? E.x : 0.f;
            if (two)
                g[1] = resume ? E.y : 0.f;
        }
        float *to = a.lam_part + (long long)seq * a.cluster * a.C + c0;    // (short sequences: one block each)
        to[0] = part.x;
        if (two)
            to[1] = part.y;
    }
}

// dlam from the blocks' sums, in a fixed order: a block of 8 warps owns 32
// channels, warp w adds rows w, w + 8, ...
__global__ void __launch_bounds__(256)
gated_lam_kernel(const GatedArgs a)
{
    griddep_entry();
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const int rows = a.n_seqs * a.cluster;
    float s = 0.f;
    if (c < a.C)
#pragma unroll 4
        for (int u = warp; u < rows; u += 8)
            s += a.lam_part[(long long)u * a.C + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < a.C) {
        s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            s += part[w][lane];
        a.grad_lam[c] = s * (-a.decay_scale * sigmoid_f(__ldg(a.lam + c)));
    }
}

// The walk over every sequence, or over the long ones of a call of short ones.
template <class T, bool LONGS>
cudaError_t launch_walk_back(const GatedArgs &a, bool pairs, int dtype, cudaStream_t stream)
{
    const unsigned blocks = LONGS ? gated_mixed_blocks(a) : gated_walk_blocks(a);
    const size_t smem = GatedBackward<T>::kSmem + gated_exchange_bytes(a.cluster);
    GatedMap mx, mga, mgx, mdy;
    if (gated_map(&mx, a.x, dtype, a.n_tokens, a.C, a.sx) && gated_map(&mga, a.gate_a, dtype, a.n_tokens, a.C, a.sga) &&
        gated_map(&mgx, a.gate_x, dtype, a.n_tokens, a.C, a.sgx) &&
        gated_map(&mdy, a.grad_y, dtype, a.n_tokens, a.C, a.sy))
        return launch_clusters(gated_scan_backward_kernel<T, true, LONGS>, a, blocks, kBackwardWarps, smem, stream, a,
                               pairs ? 1 : 0, 0, mx, mga, mgx, mdy);
    const bool words = gated_words(a.x, dtype, a.C, a.sx) && gated_words(a.gate_a, dtype, a.C, a.sga) &&
                       gated_words(a.gate_x, dtype, a.C, a.sgx) && gated_words(a.grad_y, dtype, a.C, a.sy);
    return launch_clusters(gated_scan_backward_kernel<T, false, LONGS>, a, blocks, kBackwardWarps, smem, stream, a,
                           pairs ? 1 : 0, words ? 1 : 0, mx, mga, mgx, mdy);
}

template <class T>
cudaError_t launch_backward(GatedArgs a, bool pairs, int dtype, cudaStream_t stream)
{
    cudaError_t e = cudaSuccess;
    if (!gated_short(a)) {
        e = launch_walk_back<T, false>(a, pairs, dtype, stream);
    } else {
        if (gated_mixed(a)) {
            a.step_most = kGatedStep;
            e = launch_walk_back<T, true>(a, pairs, dtype, stream);
            if (e != cudaSuccess)
                return e;
        }
        const bool in = ((a.sx | a.sga | a.sgx | a.sy) & 1) == 0 &&
                        ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.gate_a) |
                          reinterpret_cast<uintptr_t>(a.gate_x) | reinterpret_cast<uintptr_t>(a.grad_y)) %
                         (2 * sizeof(T))) == 0;
        const dim3 grid((unsigned)((a.C + 255) / 256), (unsigned)(a.n_seqs < 65535 ? a.n_seqs : 65535));
        e = launch_pdl(gated_step_backward_kernel<T>, grid, dim3(128), 0, stream, a, pairs && in ? 1 : 0);
    }
    return e != cudaSuccess ? e
                            : launch_pdl(gated_lam_kernel, dim3((unsigned)((a.C + 31) / 32)), dim3(256), 0, stream, a);
}

}  // namespace

cudaError_t launch_gated_scan_backward(GatedArgs a, int dtype, cudaStream_t stream)
{
    a.cblocks = (a.C + kGatedCh - 1) / kGatedCh;
    a.cluster = gated_cluster(a.n_seqs, a.n_tokens, a.C, false);
    a.fail_waits = debug_fail_waits();
    a.step_most = INT_MAX;
    const bool pairs = ((a.C | a.gsx | a.gsga | a.gsgx) & 1) == 0 &&
                       ((reinterpret_cast<uintptr_t>(a.grad_x) | reinterpret_cast<uintptr_t>(a.grad_ga) |
                         reinterpret_cast<uintptr_t>(a.grad_gx)) % (2 * dtype_size(dtype))) == 0;
    switch (dtype) {
    case kF32: return launch_backward<float>(a, pairs, dtype, stream);
    case kBF16: return launch_backward<__nv_bfloat16>(a, pairs, dtype, stream);
    case kF16: return launch_backward<__half>(a, pairs, dtype, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssm
