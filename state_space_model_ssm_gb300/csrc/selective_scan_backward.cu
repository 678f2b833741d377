// Selective scan with a decay for each channel and state, backward (sm_103a).
// Formulas and the layout of a warp: selective_common.cuh.  With gp = grad_y z sigmoid(z),
// the gradient e of a state after token t, a its decay and k = a h_{t-1} what the decay leaves:
//
//   e_t[c,n]  = gp_t[c] C_t[n] + a_{t+1}[c,n] e_{t+1}[c,n]      (+ grad_state after the last token)
//   grad_C[n] = sum_c gp h[c,n],         grad_B[n] = sum_c e[c,n] step x
//   grad_x    = D gp + step sum_n e B,   grad step = sum_n e (A k + x B),   grad_A = sum_t e step k
//   grad_z    = grad_y p s (1 + z (1 - s)), s = sigmoid(z)
//
// Per chunk of 16 tokens, from the state the forward pass saved, eight tokens at a time: the
// states are computed again with k kept in shared memory (one exponential more an element
// than keeping the decays too, half the memory), and with them the sums that need h; then the
// tokens are walked backwards.  A lane's share of a sum over states or channels goes to shared memory (exchanged
// between lanes for every token, the sums took a quarter of the instructions) and other threads add the
// shares up, over the block's warps too; sums over channel blocks and units are left to two small kernels.  Always
// in the same order.
//
// Units of time as in the forward pass: with segments, a pass before finds what each segment
// hands to the one in front of it.
#include "selective_walk.cuh"

namespace ssm {

namespace {

// The gradient that reaches each unit from behind, in place of what the unit hands on.  grid: (channels and states,
// shares of the sequences); a whole sequence takes grad_state itself.
__global__ void __launch_bounds__(256)
sel_carry_combine_kernel(const SelArgs a)
{
    griddep_entry();
    const long long width = (long long)a.channels * a.N, e = (long long)blockIdx.x * 256 + threadIdx.x;
    if (e >= width)
        return;
    const int c = (int)(e / a.N);
    const float A = a.A[e] * kLog2e;
    for (int seq = blockIdx.y; seq < a.n_seqs; seq += gridDim.y) {
        const int u0 = a.first[seq], u1 = a.first[seq + 1];
        if (u1 - u0 <= 1)
            continue;
        float g = a.grad_state ? a.grad_state[seq * width + e] : 0.f;
        for (int u = u1 - 1; u >= u0; u -= kCombineRun) {
            float own[kCombineRun], step[kCombineRun];
#pragma unroll
            for (int k = 0; k < kCombineRun; ++k) {
                const long long v = max(u - k, u0);
                own[k] = a.unit_state[v * width + e];
                step[k] = a.unit_step[v * a.channels + c];
            }
#pragma unroll
            for (int k = 0; k < kCombineRun; ++k) {
                if (u - k < u0)
                    break;
                a.unit_state[(u - k) * width + e] = g;
                g = sel_passed(g, step[k] * A, own[k]);     // (the first unit's values are not there, and not used)
            }
        }
    }
}

constexpr int kBackL = kSelChunk, kBackNP = 4, kKeepTokens = 8;

template <int LN>
struct BackLayout {                                         // floats of a warp, then of the block
    static constexpr int WC = 32 / LN * kSelCh, NN = kBackNP * LN;
    static constexpr int kRow = SelStage<WC, kBackL>::kTokens * WC;
    static constexpr int kSlot = 128;                       // four floats of every lane
    static constexpr int kKeep = kKeepTokens * 4 * kSlot;   // k of every token: four slots
    static constexpr int kWarp = kKeep + kKeepTokens * kSlot + 3 * kRow + kKeepTokens * WC;
    static constexpr int kRows = kBackL * NN;               // of B or C, last, each value twice: as the pair that multiplies two channels
    static constexpr size_t kBytes = ((size_t)kWarp * kSelWarps + 4 * kRows) * sizeof(float);
};

// Threads that share an output of a block's sums over channels.
template <int LN>
constexpr int kSumParts = 32 * kSelWarps / (kKeepTokens * LN) > 1 ? 32 * kSelWarps / (kKeepTokens * LN) : 1;

// Sums over a block's channels of what its lanes have put into slot `slot` of eight tokens (four states a lane):
// terms are the warps' lanes of one state, `kParts` threads of a warp share an output of four states.
template <int LN>
__device__ __forceinline__ float4 sum_slots(const float *first, int warp_stride, int token_stride, int out, int part)
{
    constexpr int Q = 32 / LN, kTerms = kSelWarps * Q, kParts = kSumParts<LN>, kEach = kTerms / kParts;
    const int t = out / LN, sub = out % LN;
    float2 lo = make_float2(0.f, 0.f), hi = lo;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int term = part * kEach + j, w = term / Q, q = term % Q;
        const float4 v = *reinterpret_cast<const float4 *>(first + w * warp_stride + t * token_stride + 4 * (q * LN + sub));
        lo = add2(lo, make_float2(v.x, v.y));
        hi = add2(hi, make_float2(v.z, v.w));
    }
    float r[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
    for (int off = kParts / 2; off >= 1; off /= 2)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r[e] += __shfl_xor_sync(kFullMask, r[e], off);
    return make_float4(r[0], r[1], r[2], r[3]);
}

// Sum over a channel's lanes of one slot, two channels (c even); lanes of different channels begin at different
// ones, so that they read different banks.
template <int LN>
__device__ __forceinline__ float2 sum_lanes(const float *slot, int c)
{
    const int q = c / 4;
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < LN; ++i)
        v = add2(v, *reinterpret_cast<const float2 *>(slot + 4 * (q * LN + ((i + q / 2) & (LN - 1))) + c % 4));
    return v;
}

// Two blocks an SM (1 x 4096 x 4096 channels x 16 states, bf16: 488 us).  Three of 168 registers with k of four tokens
// (546 to 590 us), k of four tokens in registers (625 us: more code, more barriers), two channels a lane with three
// blocks (594 us), a saved state every 8 tokens and no second walk (538 us) were slower.
template <class T, int LN>
__global__ void __launch_bounds__(32 * kSelWarps, LN == 32 ? 1 : 2)
sel_backward_kernel(const SelArgs a)
{
    griddep_entry();
    using Y = BackLayout<LN>;
    constexpr int CH = kSelCh, NP = kBackNP, WC = Y::WC, NN = Y::NN, L = kBackL, K = kKeepTokens;
    using S = SelStage<WC, L>;
    constexpr int M = S::M, KC = S::KC, H = M > 8 ? 8 : M;  // places loaded together
    constexpr int R = L / K, E = M >= R ? M / R : 1;        // places of K tokens (all of them where a place has more)
    constexpr int kOwn = CH > LN ? CH / LN : 1;             // sums over states that a lane ends with
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane % LN, q = lane / LN, n0 = sub * NP;
    const int u = blockIdx.x / a.cblocks, cblock = blockIdx.x - u * a.cblocks;
    const SelTile tile = sel_tile<WC>(a, cblock, warp);
    SelUnit s;
    if (!sel_unit(a, u, s))                                 // (the whole block)
        return;
    const int wc = tile.c1 - tile.c0;
    const bool pad = a.N != NN, pairs = a.pairs != 0;
    const bool vec_c = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.chunk_states) & 15) == 0;
    float *w = sm + warp * Y::kWarp;
    // Of eight tokens: k, in whose place a token's sums are put once it has been read (slot 0: sum_n e A k, slot 1:
    // sum_n e B, each of a lane's states and four channels; slot 2: sum_c e step x of its channels and four states);
    // sum_c gp h alike; p.  Of the chunk: step, step x, gp.
    float *keep = w, *sum_C = keep + Y::kKeep, *step = sum_C + K * Y::kSlot, *in = step + Y::kRow, *gs = in + Y::kRow;
    float *ps = gs + Y::kRow;
    float2 *Bs = reinterpret_cast<float2 *>(sm + kSelWarps * Y::kWarp), *Cs = Bs + Y::kRows;
    // Pairs of channels here (the walks pair states): the steps and inputs of two channels lie side by
    // side in shared memory, and a sum over states needs no last addition.
    constexpr int CP = CH / 2;
    float2 e[CP][NP], A[CP][NP], gA[CP][NP], h0[CP][NP];
    auto read_pair = [&](float2 (&v)[NP], const float *base, int cp, bool vec, bool given) {
        float2 r[2][NP / 2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = q * CH + 2 * cp + i;
            read_states<NP>(r[i], base + (long long)(tile.c0 + c) * a.N, n0, a.N, vec, given && c < wc);
        }
#pragma unroll
        for (int j = 0; j < NP / 2; ++j) {
            v[2 * j] = make_float2(r[0][j].x, r[1][j].x);
            v[2 * j + 1] = make_float2(r[0][j].y, r[1][j].y);
        }
    };
    auto write_pair = [&](float *base, const float2 (&v)[NP], int cp, bool vec) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = q * CH + 2 * cp + i;
            float2 r[NP / 2];
#pragma unroll
            for (int j = 0; j < NP / 2; ++j)
                r[j] = i == 0 ? make_float2(v[2 * j].x, v[2 * j + 1].x) : make_float2(v[2 * j].y, v[2 * j + 1].y);
            if (c < wc)
                write_states<NP>(base + (long long)(tile.c0 + c) * a.N, r, n0, a.N, vec);
        }
    };
    auto drop_padding = [&](float2 (&v)[NP]) {              // (see there)
#pragma unroll
        for (int n = 0; n < NP; ++n)
            v[n] = n0 + n < a.N ? v[n] : make_float2(0.f, 0.f);
    };
#pragma unroll
    for (int c = 0; c < CP; ++c) {
        read_pair(A[c], a.A, c, a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.A) & 15) == 0, true);
        if (s.cut)
            read_pair(e[c], a.unit_state + (long long)u * a.channels * a.N, c, a.N % 4 == 0, true);
        else
            read_pair(e[c], a.grad_state + (long long)s.seq * a.channels * a.N, c, false, a.grad_state != nullptr);
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            A[c][n] = mul2(A[c][n], twice(kLog2e));
            gA[c][n] = make_float2(0.f, 0.f);
        }
    }
    float2 bias[KC], D[KC], gD[KC], gbias[KC];
    read_channels<KC, WC>(bias, a.bias, tile.c0, wc, lane);
    read_channels<KC, WC>(D, a.D, tile.c0, wc, lane);
#pragma unroll
    for (int k = 0; k < KC; ++k)
        gD[k] = gbias[k] = make_float2(0.f, 0.f);
    const T *x = static_cast<const T *>(a.x) + tile.c0, *dt = static_cast<const T *>(a.dt) + tile.c0;
    const T *z = a.z ? static_cast<const T *>(a.z) + tile.c0 : nullptr, *gy = static_cast<const T *>(a.grad_y) + tile.c0;
    const T *B = static_cast<const T *>(a.B) + tile.g * a.N, *C = static_cast<const T *>(a.C) + tile.g * a.N;
    T *gx = static_cast<T *>(a.grad_x) + tile.c0, *gdt = static_cast<T *>(a.grad_dt) + tile.c0;
    T *gz = z ? static_cast<T *>(a.grad_z) + tile.c0 : nullptr;
    const long long row_n = (long long)a.groups * a.N;      // a row of the partial sums of grad_B and grad_C
    const long long part_row = (long long)(cblock % (a.cblocks / a.groups)) * a.n_tokens;

    for (int b = s.end > s.begin ? s.begin + (s.end - 1 - s.begin) / L * L : -1; b >= s.begin; b -= L) {
        const int cnt = min(L, s.end - b);
        const long long t0 = s.t0 + b;
        SelRows<T, NN, L> rB, rC;
        rB.load(B + t0 * a.sB, a.sB, a.N, cnt);
        rC.load(C + t0 * a.sC, a.sC, a.N, cnt);
        const float *cs = a.chunk_states + sel_chunk_row(a.n_seqs, s.seq, s.t0, b / L) * a.channels * a.N;
#pragma unroll
        for (int c = 0; c < CP; ++c)
            read_pair(h0[c], cs, c, vec_c, true);
        float2 finite = make_float2(0.f, 0.f);              // a NaN once anything is infinite or a NaN
        if (wc > 0) {
#pragma unroll
            for (int m0 = 0; m0 < M; m0 += H) {
                RawPair<T> rdt[H], rx[H], rg[H], rz[H];
                load_places<T, WC, L>(rdt, m0, dt + t0 * a.sdt, a.sdt, cnt, wc, lane, pairs);
                load_places<T, WC, L>(rx, m0, x + t0 * a.sx, a.sx, cnt, wc, lane, pairs);
                load_places<T, WC, L>(rg, m0, gy + t0 * a.sgy, a.sgy, cnt, wc, lane, pairs);
                if (z)
                    load_places<T, WC, L>(rz, m0, z + t0 * a.sz, a.sz, cnt, wc, lane, pairs);
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    const int m = m0 + k, t = S::tok(m, lane), c = 2 * S::cp(m, lane);
                    float2 st = sel_step2(add2(pair_of<T>(rdt[k]), bias[m % KC]), a.softplus);
                    float2 g = pair_of<T>(rg[k]), v = mul2(st, pair_of<T>(rx[k]));
                    if (z) {
                        const float2 zv = pair_of<T>(rz[k]);
                        g = mul2(g, mul2(zv, sigmoid2(zv)));
                    }
                    // what is not there takes no part in the sums over channels
                    const bool one = t < cnt && c < wc, two = t < cnt && c + 1 < wc;
                    *reinterpret_cast<float2 *>(step + t * WC + c) = make_float2(one ? st.x : 0.f, two ? st.y : 0.f);
                    *reinterpret_cast<float2 *>(in + t * WC + c) = make_float2(one ? v.x : 0.f, two ? v.y : 0.f);
                    *reinterpret_cast<float2 *>(gs + t * WC + c) = make_float2(one ? g.x : 0.f, two ? g.y : 0.f);
                }
            }
            if (pad)                                        // (a lane's own places)
#pragma unroll 1
                for (int m = 0; m < M; ++m) {
                    const float *p = step + S::tok(m, lane) * WC + 2 * S::cp(m, lane);
#pragma unroll
                    for (int r = 0; r < 3; ++r)
                        finite = fma2(*reinterpret_cast<const float2 *>(p + r * Y::kRow), twice(0.f), finite);
                }
        } else {
            for (int i = lane; i < 3 * Y::kRow; i += 32)
                step[i] = 0.f;
        }
        const bool drop = pad && __any_sync(kFullMask, finite.x + finite.y != 0.f);
        rB.store_twice(Bs, a.N);
        rC.store_twice(Cs, a.N);
        __syncthreads();
#pragma unroll 1
        for (int first = (cnt - 1) / K * K; first >= 0; first -= K) {
            const int stop = min(cnt, first + K);
            float2 h[CP][NP];
#pragma unroll
            for (int c = 0; c < CP; ++c)
#pragma unroll
                for (int n = 0; n < NP; ++n)
                    h[c][n] = h0[c][n];
#pragma unroll 1
            for (int t = 0; t < first; ++t) {               // up to the tokens whose k is kept
                float2 st[CP], uv[CP], Bv[NP];
                load_pairs<CH>(st, step + t * WC + q * CH);
                load_pairs<CH>(uv, in + t * WC + q * CH);
                load_pairs<2 * NP>(Bv, reinterpret_cast<const float *>(Bs + t * NN + n0));
#pragma unroll
                for (int c = 0; c < CP; ++c)
#pragma unroll
                    for (int n = 0; n < NP; ++n)
                        h[c][n] = fma2(ex2_2(mul2(st[c], A[c][n])), h[c][n], mul2(uv[c], Bv[n]));
            }
            // what the gate's gradient and the outputs read, loaded before the walks that come first
            const int m0 = M >= R ? first / K * E : 0;
            RawPair<T> rz[E], rx[E], rg[E], rdt[E];
            if (wc > 0) {
                load_places<T, WC, L>(rx, m0, x + t0 * a.sx, a.sx, cnt, wc, lane, pairs);
                if (z) {
                    load_places<T, WC, L>(rz, m0, z + t0 * a.sz, a.sz, cnt, wc, lane, pairs);
                    load_places<T, WC, L>(rg, m0, gy + t0 * a.sgy, a.sgy, cnt, wc, lane, pairs);
                }
            }
#pragma unroll 1
            for (int t = first; t < stop; ++t) {
                float2 st[CP], uv[CP], gv[CP], Bv[NP], Cv[NP], sum_c[NP];
                float p[CH];
                load_pairs<CH>(st, step + t * WC + q * CH);
                load_pairs<CH>(uv, in + t * WC + q * CH);
                load_pairs<CH>(gv, gs + t * WC + q * CH);
                load_pairs<2 * NP>(Bv, reinterpret_cast<const float *>(Bs + t * NN + n0));
                load_pairs<2 * NP>(Cv, reinterpret_cast<const float *>(Cs + t * NN + n0));
                float2 k[CP][NP];
#pragma unroll
                for (int c = 0; c < CP; ++c)
#pragma unroll
                    for (int n = 0; n < NP; ++n) {
                        k[c][n] = mul2(ex2_2(mul2(st[c], A[c][n])), h[c][n]);
                        h[c][n] = fma2(uv[c], Bv[n], k[c][n]);
                    }
                if (drop)                                   // (one branch a token: it is not known to be uniform)
#pragma unroll
                    for (int c = 0; c < CP; ++c) {
                        drop_padding(h[c]);
                        drop_padding(k[c]);
                    }
#pragma unroll
                for (int c = 0; c < CP; ++c) {
                    float2 sum;
#pragma unroll
                    for (int n = 0; n < NP; ++n) {
                        sum = n == 0 ? mul2(h[c][n], Cv[n]) : fma2(h[c][n], Cv[n], sum);
                        sum_c[n] = c == 0 ? mul2(gv[c], h[c][n]) : fma2(gv[c], h[c][n], sum_c[n]);
                    }
#pragma unroll
                    for (int n = 0; n < NP; n += 2)
                        *reinterpret_cast<float4 *>(keep + ((t - first) * 4 + 2 * c + n / 2) * Y::kSlot + 4 * lane) =
                            make_float4(k[c][n].x, k[c][n].y, k[c][n + 1].x, k[c][n + 1].y);
                    p[2 * c] = sum.x;
                    p[2 * c + 1] = sum.y;
                }
                *reinterpret_cast<float4 *>(sum_C + (t - first) * Y::kSlot + 4 * lane) =
                    make_float4(sum_c[0].x + sum_c[0].y, sum_c[1].x + sum_c[1].y, sum_c[2].x + sum_c[2].y, sum_c[3].x + sum_c[3].y);
                if (z) {
                    int at;
                    bool mine;
                    lanes_sum<CH, LN, 1>(p, lane, at, mine);
                    // (lanes that hold the same sum write the same value)
#pragma unroll
                    for (int r = 0; r < kOwn; ++r)
                        ps[(t - first) * WC + q * CH + at + r] = p[r];
                }
            }
            __syncwarp();
            if (z && wc > 0) {                              // the gate's gradient
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const int t = S::tok(m0 + k, lane), c = 2 * S::cp(m0 + k, lane);
                    if (t < first || t >= stop || c >= wc)
                        continue;
                    const float2 zv = pair_of<T>(rz[k]), sg = sigmoid2(zv);
                    const float2 p = fma2(D[k % KC], pair_of<T>(rx[k]), *reinterpret_cast<const float2 *>(ps + (t - first) * WC + c));
                    const float2 rest = make_float2(1.f - sg.x, 1.f - sg.y);
                    store_pair<T>(gz + (t0 + t) * a.sgz + c,
                                  mul2(mul2(pair_of<T>(rg[k]), p), fma2(mul2(zv, sg), rest, sg)), pairs, c + 1 < wc);
                }
            }
            if (wc > 0)
                load_places<T, WC, L>(rdt, m0, dt + t0 * a.sdt, a.sdt, cnt, wc, lane, pairs);
#pragma unroll 1
            for (int t = stop - 1; t >= first; --t) {
                float2 st[CP], uv[CP], gv[CP], Bv[NP], Cv[NP], sum_b[NP];
                float2 s1[CP], s2[CP];
                float *slots = keep + (t - first) * 4 * Y::kSlot + 4 * lane;
                load_pairs<CH>(st, step + t * WC + q * CH);
                load_pairs<CH>(uv, in + t * WC + q * CH);
                load_pairs<CH>(gv, gs + t * WC + q * CH);
                load_pairs<2 * NP>(Bv, reinterpret_cast<const float *>(Bs + t * NN + n0));
                load_pairs<2 * NP>(Cv, reinterpret_cast<const float *>(Cs + t * NN + n0));
                float2 k[CP][NP];
#pragma unroll
                for (int c = 0; c < CP; ++c) {
#pragma unroll
                    for (int n = 0; n < NP; n += 2) {
                        const float4 v = *reinterpret_cast<const float4 *>(slots + (2 * c + n / 2) * Y::kSlot);
                        k[c][n] = make_float2(v.x, v.y);
                        k[c][n + 1] = make_float2(v.z, v.w);
                    }
#pragma unroll
                    for (int n = 0; n < NP; ++n)
                        e[c][n] = fma2(gv[c], Cv[n], e[c][n]);
                }
                if (drop)
#pragma unroll
                    for (int c = 0; c < CP; ++c)
                        drop_padding(e[c]);
#pragma unroll
                for (int c = 0; c < CP; ++c) {
                    float2 wa, wb;
#pragma unroll
                    for (int n = 0; n < NP; ++n) {
                        const float2 v = mul2(e[c][n], k[c][n]);
                        gA[c][n] = fma2(st[c], v, gA[c][n]);
                        wa = n == 0 ? mul2(v, A[c][n]) : fma2(v, A[c][n], wa);
                        wb = n == 0 ? mul2(e[c][n], Bv[n]) : fma2(e[c][n], Bv[n], wb);
                        sum_b[n] = c == 0 ? mul2(uv[c], e[c][n]) : fma2(uv[c], e[c][n], sum_b[n]);
                        e[c][n] = mul2(ex2_2(mul2(st[c], A[c][n])), e[c][n]);
                    }
                    s1[c] = wa;
                    s2[c] = wb;
                }
                *reinterpret_cast<float4 *>(slots) = make_float4(s1[0].x, s1[0].y, s1[1].x, s1[1].y);
                *reinterpret_cast<float4 *>(slots + Y::kSlot) = make_float4(s2[0].x, s2[0].y, s2[1].x, s2[1].y);
                *reinterpret_cast<float4 *>(slots + 2 * Y::kSlot) =
                    make_float4(sum_b[0].x + sum_b[0].y, sum_b[1].x + sum_b[1].y, sum_b[2].x + sum_b[2].y, sum_b[3].x + sum_b[3].y);
            }
            __syncthreads();                                // every warp's sums are there
            constexpr int kParts = kSumParts<LN>;
#pragma unroll
            for (int i = tid; i < K * LN * kParts; i += 32 * kSelWarps) {
                const int out = i / kParts, part = i % kParts, t = first + out / LN, n = out % LN * NP;
                const float4 vb = sum_slots<LN>(sm + 2 * Y::kSlot, Y::kWarp, 4 * Y::kSlot, out, part);
                const float4 vc = sum_slots<LN>(sm + Y::kKeep, Y::kWarp, Y::kSlot, out, part);
                if (part == 0 && t < stop && n < a.N) {
                    const long long at = (part_row + t0 + t) * row_n + tile.g * a.N + n;
                    const float b4[4] = {vb.x, vb.y, vb.z, vb.w}, c4[4] = {vc.x, vc.y, vc.z, vc.w};
#pragma unroll
                    for (int e4 = 0; e4 < 4; ++e4)
                        if (n + e4 < a.N) {
                            a.part_B[at + e4] = b4[e4];
                            a.part_C[at + e4] = c4[e4];
                        }
                }
            }
            if (wc > 0) {
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const int t = S::tok(m0 + k, lane), c = 2 * S::cp(m0 + k, lane), i = t * WC + c;
                    if (t < first || t >= stop || c >= wc)
                        continue;
                    const float2 xv = pair_of<T>(rx[k]), gv = *reinterpret_cast<const float2 *>(gs + i);
                    const float2 st = *reinterpret_cast<const float2 *>(step + i);
                    const float2 sa = sum_lanes<LN>(keep + (t - first) * 4 * Y::kSlot, c);
                    const float2 eb = sum_lanes<LN>(keep + (t - first) * 4 * Y::kSlot + Y::kSlot, c);
                    const float2 g = mul2(fma2(sa, twice(kLn2), mul2(xv, eb)),
                                          sel_slope2(add2(pair_of<T>(rdt[k]), bias[k % KC]), a.softplus));
                    store_pair<T>(gx + (t0 + t) * a.sgx + c, fma2(D[k % KC], gv, mul2(st, eb)), pairs, c + 1 < wc);
                    store_pair<T>(gdt + (t0 + t) * a.sgdt + c, g, pairs, c + 1 < wc);
                    gD[k % KC] = fma2(gv, xv, gD[k % KC]);
                    gbias[k % KC] = add2(gbias[k % KC], g);
                }
            }
            __syncthreads();                                // ... and read
        }
    }
    const bool resumed = a.resume[s.seq] != 0;
#pragma unroll
    for (int c = 0; c < CP; ++c) {
        write_pair(a.part_A + (long long)u * a.channels * a.N, gA[c], c, a.N % 4 == 0);
        if (s.k == 0 && a.grad_state0) {
#pragma unroll
            for (int n = 0; n < NP; ++n)
                e[c][n] = resumed ? e[c][n] : make_float2(0.f, 0.f);
            write_pair(a.grad_state0 + (long long)s.seq * a.channels * a.N, e[c], c, false);
        }
    }
    // lanes that hold the same pair of channels
#pragma unroll
    for (int k = 0; k < KC; ++k) {
#pragma unroll
        for (int off = 16; off >= S::P; off /= 2) {
            gD[k].x += __shfl_xor_sync(kFullMask, gD[k].x, off);
            gD[k].y += __shfl_xor_sync(kFullMask, gD[k].y, off);
            gbias[k].x += __shfl_xor_sync(kFullMask, gbias[k].x, off);
            gbias[k].y += __shfl_xor_sync(kFullMask, gbias[k].y, off);
        }
        const int c = 2 * S::cp(k, lane);
        const long long at = (long long)u * a.channels + tile.c0 + c;
        if (lane < S::P && c < wc) {
            a.part_D[at] = gD[k].x;
            a.part_bias[at] = gbias[k].x;
        }
        if (lane < S::P && c + 1 < wc) {
            a.part_D[at + 1] = gD[k].y;
            a.part_bias[at + 1] = gbias[k].y;
        }
    }
}

// Sums over units (the parameters' gradients), elements i of `width`.
__global__ void __launch_bounds__(256)
sel_sum_units_kernel(const SelArgs a)
{
    griddep_entry();
    const int units = a.seg ? a.first[a.n_seqs] : a.n_seqs;
    const long long nA = (long long)a.channels * a.N, i = (long long)blockIdx.x * 256 + threadIdx.x;
    const float *src;
    float *dst;
    long long width, at = i;
    if (i < nA) {
        src = a.part_A; dst = a.grad_A; width = nA;
    } else if (i < nA + a.channels) {
        src = a.part_D; dst = a.grad_D; width = a.channels; at = i - nA;
    } else if (i < nA + 2 * a.channels) {
        src = a.part_bias; dst = a.grad_bias; width = a.channels; at = i - nA - a.channels;
    } else {
        return;
    }
    if (!dst)
        return;
    float v = 0.f;
    for (int u = 0; u < units; ++u)
        v += src[u * width + at];
    dst[at] = v;
}

// Whether a token belongs to a sequence is not known here: rows of none were never written, and the
// sequences are walked instead of the rows.  grid: (sequence, blocks of its values)
template <class T>
__global__ void __launch_bounds__(256)
sel_sum_channels_kernel(const SelArgs a, int blocks)
{
    griddep_entry();
    const int width = a.groups * a.N, per = a.cblocks / a.groups, seq = blockIdx.x / blocks;
    long long t0;
    const long long n = (long long)sel_seq_len(a, seq, t0) * width;
    T *gB = static_cast<T *>(a.grad_B), *gC = static_cast<T *>(a.grad_C);
    for (long long i = (long long)(blockIdx.x - seq * blocks) * 256 + threadIdx.x; i < n; i += (long long)blocks * 256) {
        const long long t = t0 + i / width;
        const int e = (int)(i % width);
        float vb = 0.f, vc = 0.f;
        for (int k = 0; k < per; ++k) {
            const long long at = ((long long)k * a.n_tokens + t) * width + e;
            vb += a.part_B[at];
            vc += a.part_C[at];
        }
        gB[t * a.sgB + e] = from_float<T>(vb);
        gC[t * a.sgC + e] = from_float<T>(vc);
    }
}

template <class T, int LN>
cudaError_t launch_shape(const SelArgs &a, cudaStream_t st)
{
    const auto kernel = sel_backward_kernel<T, LN>;
    constexpr size_t bytes = BackLayout<LN>::kBytes;
    const cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kernel), bytes);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kernel, dim3((unsigned)((long long)a.max_units * a.cblocks)), dim3(32 * kSelWarps), bytes, st, a);
}

template <class T>
cudaError_t launch_type(const SelArgs &a, cudaStream_t st)
{
    cudaError_t e = cudaSuccess;
    if (a.seg) {
        e = launch_walk_states<T, kCarry>(a, a.max_units, st);
        if (e != cudaSuccess)
            return e;
        e = launch_pdl(sel_carry_combine_kernel, sel_combine_grid(a), dim3(256), 0, st, a);
        if (e != cudaSuccess)
            return e;
    }
    // (up to 8 states as for 16: with two lanes a channel a block needs 139 KB and spills, and was half as fast)
    e = a.N <= 16 ? launch_shape<T, 4>(a, st) : a.N <= 32 ? launch_shape<T, 8>(a, st)
        : a.N <= 64 ? launch_shape<T, 16>(a, st) : launch_shape<T, 32>(a, st);
    if (e != cudaSuccess)
        return e;
    const long long n = (long long)a.channels * (a.N + 2);
    e = launch_pdl(sel_sum_units_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, a);
    if (e != cudaSuccess || a.n_tokens == 0)
        return e;
    const long long values = (long long)a.n_tokens * a.groups * a.N;
    long long blocks = values / a.n_seqs / 256 + 1;
    blocks = blocks > 1024 ? 1024 : blocks;
    return launch_pdl(sel_sum_channels_kernel<T>, dim3((unsigned)(blocks * a.n_seqs)), dim3(256), 0, st, a, (int)blocks);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Workspace {
    size_t units, first, state, step, A, D, bias, B, C, total;
};
Workspace layout(int n_seqs, int n_tokens, int channels, int N, int groups, int seg, int cblocks)
{
    const int units = sel_max_units(n_seqs, n_tokens, seg);
    const size_t rows = up256((size_t)(cblocks / groups) * n_tokens * groups * N * 4);
    Workspace w;
    w.units = 0;
    w.first = seg ? up256((size_t)units * sizeof(int2)) : 0;
    w.state = w.first + (seg ? up256(((size_t)n_seqs + 1) * 4) : 0);
    w.step = w.state + (seg ? up256((size_t)units * channels * N * 4) : 0);
    w.A = w.step + (seg ? up256((size_t)units * channels * 4) : 0);
    w.D = w.A + up256((size_t)units * channels * N * 4);
    w.bias = w.D + up256((size_t)units * channels * 4);
    w.B = w.bias + up256((size_t)units * channels * 4);
    w.C = w.B + rows;
    w.total = w.C + rows;
    return w;
}

}  // namespace

size_t sel_backward_workspace_bytes(int n_seqs, int n_tokens, int channels, int N, int groups)
{
    const SelShape s = sel_shape(channels, N, groups, true);
    return layout(n_seqs, n_tokens, channels, N, groups, sel_cut(n_seqs, n_tokens, channels, N, groups, true).seg, s.cblocks).total;
}

cudaError_t launch_selective_scan_backward(SelArgs a, int dtype, void *workspace, cudaStream_t st)
{
    const SelShape s = sel_shape(a.channels, a.N, a.groups, true);
    a.cblocks = s.cblocks;
    a.pairs = sel_pairs(a, dtype);
    const SelCut cut = sel_cut(a.n_seqs, a.n_tokens, a.channels, a.N, a.groups, true);
    a.seg = cut.seg;
    a.whole = cut.whole;
    a.max_units = sel_max_units(a.n_seqs, a.n_tokens, a.seg);
    unsigned char *w = static_cast<unsigned char *>(workspace);
    const Workspace l = layout(a.n_seqs, a.n_tokens, a.channels, a.N, a.groups, a.seg, a.cblocks);
    a.part_A = reinterpret_cast<float *>(w + l.A);
    a.part_D = reinterpret_cast<float *>(w + l.D);
    a.part_bias = reinterpret_cast<float *>(w + l.bias);
    a.part_B = reinterpret_cast<float *>(w + l.B);
    a.part_C = reinterpret_cast<float *>(w + l.C);
    if (a.seg) {
        int2 *table = reinterpret_cast<int2 *>(w + l.units);
        int *first = reinterpret_cast<int *>(w + l.first);
        a.unit_state = reinterpret_cast<float *>(w + l.state);
        a.unit_step = reinterpret_cast<float *>(w + l.step);
        const cudaError_t e = launch_sel_plan(a, table, first, st);
        if (e != cudaSuccess)
            return e;
        a.units = table;
        a.first = first;
    }
    switch (dtype) {
    case kF32: return launch_type<float>(a, st);
    case kBF16: return launch_type<__nv_bfloat16>(a, st);
    case kF16: return launch_type<__half>(a, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssm
