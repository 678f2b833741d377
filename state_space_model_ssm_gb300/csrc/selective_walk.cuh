// The walk over a unit's tokens that three passes of the selective scan share (formulas and the
// layout of a warp: selective_common.cuh):
//   kFull     the scan: states from the slot (or the segment's first state), outputs, saved states
//   kState    what a segment leaves from zero:        h <- a h + step x B
//   kCarry    what a segment's outputs' gradients hand to the one before, backwards in time:
//             e <- a (e + gp C),  gp = grad_y z sigmoid(z)
//
// Tokens go in chunks of 8.  A warp turns its channels' dt and x (or grad_y and z) into steps
// and inputs in shared memory, lanes along pairs of channels, walks the chunk with the states in
// registers, and turns the sums over states into outputs, lanes along channels again.  The next
// chunk's rows are loaded into registers before the walk.  A block's warps (neighbouring
// channels) share the chunk's B and C as fp32 rows in two buffers: one barrier a chunk.
#pragma once

#include "selective_common.cuh"

namespace ssm {

enum SelMode { kFull, kState, kCarry };

constexpr int kWalkL = 8;

template <int CH, int NP, int LN>
struct WalkLayout {
    static constexpr int WC = 32 / LN * CH, NN = NP * LN;
    static constexpr int kStage = SelStage<WC, kWalkL>::kTokens * WC;
    static constexpr int kWarp = 2 * kStage;                // floats: steps, inputs
    static constexpr int kRows = kWalkL * NN;               // of B or C
    static constexpr size_t kBytes = (size_t)(kSelWarps * kWarp + 4 * kRows) * sizeof(float);
};

// Three blocks an SM, 168 registers a thread: unbounded, kFull took 238 and 1 x 4096 x 4096 channels x 16 states
// (bf16) 180 us instead of 126.  Four states a lane, four blocks an SM: 156 us.  fp32 rows need twice the registers
// while staged and spill at three blocks (4 x 777 x 1001 channels: 80 us instead of 54).
template <class T, int CH, int NP, int LN, SelMode MODE>
__global__ void __launch_bounds__(32 * kSelWarps, CH * NP == 8 ? 5 : sizeof(T) == 4 && MODE == kFull ? 2 : 3)
sel_walk_kernel(const SelArgs a)
{
    griddep_entry();
    using Y = WalkLayout<CH, NP, LN>;
    constexpr int WC = Y::WC, NN = Y::NN, L = kWalkL;
    using S = SelStage<WC, L>;
    constexpr int M = S::M, KC = S::KC;
    extern __shared__ __align__(16) float sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane % LN, q = lane / LN, n0 = sub * NP;
    const int cblocks = a.groups * sel_group_blocks(a.channels, a.groups, WC), u = blockIdx.x / cblocks;
    const SelTile tile = sel_tile<WC>(a, blockIdx.x - u * cblocks, warp);
    SelUnit s;
    if (!sel_unit(a, u, s) || (MODE == kState && s.last) || (MODE == kCarry && s.k == 0))
        return;                                             // (the whole block)
    const int wc = tile.c1 - tile.c0;                       // channels of this warp that exist; 0: it only helps with B and C
    const bool vec = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
    const bool vec_c = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.chunk_states) & 15) == 0;
    const bool vec_a = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.A) & 15) == 0;
    const bool pad = a.N != NN, pairs = a.pairs != 0;
    float *step = sm + warp * Y::kWarp, *in = step + Y::kStage, *rows = sm + kSelWarps * Y::kWarp;

    float2 h[CH][NP / 2], A[CH][NP / 2];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = tile.c0 + q * CH + c;
        const bool there = q * CH + c < wc;
        read_states<NP>(A[c], a.A + (long long)ch * a.N, n0, a.N, vec_a, there);
#pragma unroll
        for (int j = 0; j < NP / 2; ++j)
            A[c][j] = mul2(A[c][j], twice(kLog2e));
        if (MODE != kFull)
            read_states<NP>(h[c], nullptr, n0, a.N, false, false);
        else if (s.cut)
            read_states<NP>(h[c], a.unit_state + ((long long)u * a.channels + ch) * a.N, n0, a.N, a.N % 4 == 0, there);
        else
            read_states<NP>(h[c], a.state + ((long long)s.seq * a.channels + ch) * a.N, n0, a.N, vec,
                            there && a.resume[s.seq] != 0);
    }
    float2 bias[KC], D[KC], total[KC];
    read_channels<KC, WC>(bias, a.bias, tile.c0, wc, lane);
    read_channels<KC, WC>(D, a.D, tile.c0, wc, lane);
#pragma unroll
    for (int k = 0; k < KC; ++k)
        total[k] = make_float2(0.f, 0.f);
    const T *x = static_cast<const T *>(MODE == kCarry ? a.grad_y : a.x) + tile.c0, *dt = static_cast<const T *>(a.dt) + tile.c0;
    const T *z = a.z ? static_cast<const T *>(a.z) + tile.c0 : nullptr;
    const long long sx = MODE == kCarry ? a.sgy : a.sx;
    T *y = MODE == kFull ? static_cast<T *>(a.y) + tile.c0 : nullptr;
    const T *B = static_cast<const T *>(MODE == kCarry ? a.C : a.B) + tile.g * a.N, *C = static_cast<const T *>(a.C) + tile.g * a.N;
    const long long sB = MODE == kCarry ? a.sC : a.sB;

    const int chunks = (s.end - s.begin + L - 1) / L;
    RawPair<T> rdt[M], rx[M], rz[M], xk[M];
    SelRows<T, NN, L> rB, rC;
    auto fetch = [&](int i) {
        const int b = s.begin + L * (MODE == kCarry ? chunks - 1 - i : i), cnt = min(L, s.end - b);
        const long long t0 = s.t0 + b;
        if (wc > 0) {
            load_places<T, WC, L>(rdt, 0, dt + t0 * a.sdt, a.sdt, cnt, wc, lane, pairs);
            load_places<T, WC, L>(rx, 0, x + t0 * sx, sx, cnt, wc, lane, pairs);
            if (MODE == kCarry && z)
                load_places<T, WC, L>(rz, 0, z + t0 * a.sz, a.sz, cnt, wc, lane, pairs);
        }
        rB.load(B + t0 * sB, sB, a.N, cnt);
        if (MODE == kFull)
            rC.load(C + t0 * a.sC, a.sC, a.N, cnt);
    };
    if (chunks > 0)
        fetch(0);
    for (int i = 0; i < chunks; ++i) {
        const int b = s.begin + L * (MODE == kCarry ? chunks - 1 - i : i), cnt = min(L, s.end - b);
        const long long t0 = s.t0 + b;
        float *Bs = rows + (i & 1) * 2 * Y::kRows, *Cs = Bs + Y::kRows;
        if (MODE == kFull && a.chunk_states && b % kSelChunk == 0) {
            float *cs = a.chunk_states + sel_chunk_row(a.n_seqs, s.seq, s.t0, b / kSelChunk) * a.channels * a.N;
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (q * CH + c < wc)
                    write_states<NP>(cs + (long long)(tile.c0 + q * CH + c) * a.N, h[c], n0, a.N, vec_c);
        }
        float2 finite = make_float2(0.f, 0.f);              // a NaN once anything is infinite or a NaN
        if (wc > 0) {
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int at = S::tok(m, lane) * WC + 2 * S::cp(m, lane);
                const float2 st = sel_step2(add2(pair_of<T>(rdt[m]), bias[m % KC]), a.softplus);
                float2 xv = pair_of<T>(rx[m]);
                if (MODE == kCarry && z) {
                    const float2 g = pair_of<T>(rz[m]);
                    xv = mul2(xv, mul2(g, sigmoid2(g)));
                }
                if (MODE != kCarry)
                    xv = mul2(st, xv);
                *reinterpret_cast<float2 *>(in + at) = xv;
                *reinterpret_cast<float2 *>(step + at) = st;
                if (MODE == kFull)
                    xk[m] = rx[m];
                else if (S::tok(m, lane) < cnt)
                    total[m % KC] = add2(total[m % KC], st);
            }
            if (MODE == kFull && z)
                load_places<T, WC, L>(rz, 0, z + t0 * a.sz, a.sz, cnt, wc, lane, pairs);
            if (pad)                                        // (a lane's own places)
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const int at = S::tok(m, lane) * WC + 2 * S::cp(m, lane);
                    finite = fma2(*reinterpret_cast<const float2 *>(in + at), twice(0.f),
                                  fma2(*reinterpret_cast<const float2 *>(step + at), twice(0.f), finite));
                }
        }
        const bool drop = pad && __any_sync(kFullMask, finite.x + finite.y != 0.f);
        rB.store(Bs, a.N);
        if (MODE == kFull)
            rC.store(Cs, a.N);
        __syncthreads();
        if (i + 1 < chunks)
            fetch(i + 1);
        if (wc == 0)
            continue;
#pragma unroll 1
        for (int i_t = 0; i_t < cnt; ++i_t) {
            const int t = MODE == kCarry ? cnt - 1 - i_t : i_t;
            float st[CH], uv[CH], p[CH];
            float2 Bv[NP / 2], Cv[NP / 2];
            load_floats<CH>(st, step + t * WC + q * CH);
            load_floats<CH>(uv, in + t * WC + q * CH);
            load_pairs<NP>(Bv, Bs + t * NN + n0);
            if (MODE == kFull)
                load_pairs<NP>(Cv, Cs + t * NN + n0);
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < NP / 2; ++j) {
                    const float2 decay = ex2_2(mul2(twice(st[c]), A[c][j]));
                    if (MODE == kCarry)
                        h[c][j] = mul2(decay, fma2(twice(uv[c]), Bv[j], h[c][j]));
                    else
                        h[c][j] = fma2(decay, h[c][j], mul2(twice(uv[c]), Bv[j]));
                }
            if (drop)                                       // (one branch a token: it is not known to be uniform)
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    drop_padding<NP>(h[c], n0, a.N);
            if (MODE == kFull)
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    float2 sum = mul2(h[c][0], Cv[0]);
#pragma unroll
                    for (int j = 1; j < NP / 2; ++j)
                        sum = fma2(h[c][j], Cv[j], sum);
                    p[c] = sum.x + sum.y;
                }
            if (MODE == kFull) {
                int at;
                bool mine;
                lanes_sum<CH, LN, 1>(p, sub, at, mine);
                __syncwarp();                               // the inputs of this token have been read
                if (mine)
#pragma unroll
                    for (int r = 0; r < (CH > LN ? CH / LN : 1); ++r)
                        in[t * WC + q * CH + at + r] = p[r];
            }
        }
        __syncwarp();
        if (MODE == kFull) {
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int t = S::tok(m, lane), c = 2 * S::cp(m, lane);
                float2 v = fma2(D[m % KC], pair_of<T>(xk[m]), *reinterpret_cast<const float2 *>(in + t * WC + c));
                if (z) {
                    const float2 g = pair_of<T>(rz[m]);
                    v = mul2(v, mul2(g, sigmoid2(g)));
                }
                if (t < cnt && c < wc)
                    store_pair<T>(y + (t0 + t) * a.sy + c, v, pairs, c + 1 < wc);
            }
            __syncwarp();
        }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = tile.c0 + q * CH + c;
        if (q * CH + c >= wc)
            continue;
        if (MODE != kFull)
            write_states<NP>(a.unit_state + ((long long)u * a.channels + ch) * a.N, h[c], n0, a.N, a.N % 4 == 0);
        else if (s.last)
            write_states<NP>(a.state + ((long long)s.seq * a.channels + ch) * a.N, h[c], n0, a.N, vec);
    }
    if (MODE != kFull) {
#pragma unroll
        for (int k = 0; k < KC; ++k) {                      // the lanes that hold the same pair
#pragma unroll
            for (int off = 16; off >= S::P; off /= 2) {
                total[k].x += __shfl_xor_sync(kFullMask, total[k].x, off);
                total[k].y += __shfl_xor_sync(kFullMask, total[k].y, off);
            }
            const int c = 2 * S::cp(k, lane);
            float *o = a.unit_step + (long long)u * a.channels + tile.c0 + c;
            if (lane < S::P && c < wc)
                o[0] = total[k].x;
            if (lane < S::P && c + 1 < wc)
                o[1] = total[k].y;
        }
    }
}

template <class T, int CH, int NP, int LN, SelMode MODE>
cudaError_t launch_walk(const SelArgs &a, int units, cudaStream_t st)
{
    using Y = WalkLayout<CH, NP, LN>;
    const auto kernel = sel_walk_kernel<T, CH, NP, LN, MODE>;
    const cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kernel), Y::kBytes);
    if (e != cudaSuccess)
        return e;
    const long long blocks = (long long)units * a.groups * sel_group_blocks(a.channels, a.groups, Y::WC);
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(32 * kSelWarps), Y::kBytes, st, a);
}

// By the states' number, with wide or narrow tiles (sel_narrow).
template <class T, SelMode MODE>
cudaError_t launch_walk_states(const SelArgs &a, int units, cudaStream_t st)
{
    if constexpr (MODE != kCarry) {
        if (a.narrow) {
            if (a.N <= 8) return launch_walk<T, 2, 4, 2, MODE>(a, units, st);
            if (a.N <= 16) return launch_walk<T, 2, 4, 4, MODE>(a, units, st);
            if (a.N <= 32) return launch_walk<T, 2, 4, 8, MODE>(a, units, st);
            if (a.N <= 64) return launch_walk<T, 2, 4, 16, MODE>(a, units, st);
            return launch_walk<T, 2, 4, 32, MODE>(a, units, st);
        }
    }
    if (a.N <= 8) return launch_walk<T, 4, 4, 2, MODE>(a, units, st);
    if (a.N <= 16) return launch_walk<T, 4, 8, 2, MODE>(a, units, st);
    if (a.N <= 32) return launch_walk<T, 4, 8, 4, MODE>(a, units, st);
    if (a.N <= 64) return launch_walk<T, 4, 8, 8, MODE>(a, units, st);
    return launch_walk<T, 4, 8, 16, MODE>(a, units, st);
}

}  // namespace ssm
