// Selective scan with a decay for each channel and state, backward (sm_103a).
// Formulas and the layout of a warp: selective_common.cuh.  With gp = grad_y z sigmoid(z),
// the gradient e of a state after token t, a its decay and k = a h_{t-1} what the decay leaves:
//
//   e_t[c,n]  = gp_t[c] C_t[n] + a_{t+1}[c,n] e_{t+1}[c,n]      (+ grad_state after the last token)
//   grad_C[n] = sum_c gp h[c,n],         grad_B[n] = sum_c e[c,n] step x
//   grad_x    = D gp + step sum_n e B,   grad step = sum_n e (A k + x B),   grad_A = sum_t e step k
//   grad_z    = grad_y p s (1 + z (1 - s)), s = sigmoid(z)
//
// Per chunk of 16 tokens, from the state the forward pass saved: the states are computed
// again with k kept in shared memory (one exponential more an element than keeping the
// decays too, half the memory), and with them the sums that need h; then the tokens are walked
// backwards.  Sums over states cross the LN lanes of a channel, sums over channels the
// lanes, then the block's warps in shared memory, then channel blocks in a second
// kernel: always in the same order.
//
// Units of time as in the forward pass: with segments, a pass before finds what each segment
// hands to the one in front of it.
#include "selective_common.cuh"

namespace ssm {

namespace {

constexpr int kBackCh = 2;                                  // channels of a lane

// e = exp(-step A)-weighted gradient that a unit hands to the one before it, from zero.
template <class T, int NP, int LN>
__global__ void __launch_bounds__(32 * kSelWarps)
sel_carry_kernel(const SelArgs a)
{
    griddep_entry();
    constexpr int CH = 4, WC = 32 / LN * CH, NN = NP * LN, L = kSelChunk, KC = WC > 32 ? WC / 32 : 1;
    __shared__ __align__(16) float s_step[kSelWarps][L * WC], s_g[kSelWarps][L * WC], s_C[2][L * NN];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane % LN, q = lane / LN, n0 = sub * NP;
    const int cblocks = a.groups * sel_group_blocks(a.channels, a.groups, WC), u = blockIdx.x / cblocks;
    const SelTile tile = sel_tile<WC>(a, blockIdx.x - u * cblocks, warp);
    SelUnit s;
    if (!sel_unit(a, u, s) || s.k == 0)                     // (the whole block)
        return;
    const int wc = tile.c1 - tile.c0;
    const bool pad = a.N != NN;
    float *step = s_step[warp], *gs = s_g[warp];
    float2 e[CH][NP / 2], A[CH][NP / 2];
    float total[CH], bias[KC];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        read_states<NP>(A[c], a.A + (long long)(tile.c0 + q * CH + c) * a.N, n0, a.N, false, q * CH + c < wc);
#pragma unroll
        for (int j = 0; j < NP / 2; ++j) {
            A[c][j] = make_float2(A[c][j].x * kLog2e, A[c][j].y * kLog2e);
            e[c][j] = make_float2(0.f, 0.f);
        }
        total[c] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        const int c = (lane + 32 * k) % WC;
        bias[k] = a.bias && c < wc ? __ldg(a.bias + tile.c0 + c) : 0.f;
    }
    const T *dt = static_cast<const T *>(a.dt) + tile.c0, *gy = static_cast<const T *>(a.grad_y) + tile.c0;
    const T *z = a.z ? static_cast<const T *>(a.z) + tile.c0 : nullptr;
    const T *C = static_cast<const T *>(a.C) + tile.g * a.N;
    for (int b = s.begin + (s.end - 1 - s.begin) / L * L; b >= s.begin; b -= L) {
        const int cnt = min(L, s.end - b);
        const long long t0 = s.t0 + b;
        float *Cs = s_C[b / L & 1];
#pragma unroll 4
        for (int m = 0; m < L * WC / 32; ++m) {
            const int i = lane + 32 * m, t = i / WC, c = i % WC;
            float st = 0.f, gv = 0.f, slope;
            if (t < cnt && c < wc) {
                st = sel_step(to_float(dt[(t0 + t) * a.sdt + c]) + bias[m % KC], a.softplus, slope);
                gv = to_float(gy[(t0 + t) * a.sgy + c]);
                if (z) {
                    const float g = to_float(z[(t0 + t) * a.sz + c]);
                    gv *= g * sigmoid_of(g);
                }
            }
            step[i] = st;
            gs[i] = gv;
        }
        stage_rows<T, NN>(Cs, C + t0 * a.sC, a.sC, a.N, cnt);
        __syncthreads();
        for (int t = cnt - 1; t >= 0; --t) {
            float st[CH], gv[CH];
            float2 Cv[NP / 2];
            load_floats<CH>(st, step + t * WC + q * CH);
            load_floats<CH>(gv, gs + t * WC + q * CH);
            load_pairs<NP>(Cv, Cs + t * NN + n0);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                total[c] += st[c];
#pragma unroll
                for (int j = 0; j < NP / 2; ++j)
                    e[c][j] = mul2(ex2_2(mul2(twice(st[c]), A[c][j])), fma2(twice(gv[c]), Cv[j], e[c][j]));
                if (pad)
                    drop_padding<NP>(e[c], n0, a.N);
            }
        }
        __syncwarp();
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = tile.c0 + q * CH + c;
        if (q * CH + c >= wc)
            continue;
        write_states<NP>(a.unit_state + ((long long)u * a.channels + ch) * a.N, e[c], n0, a.N, a.N % 4 == 0);
        if (sub == 0)
            a.unit_step[(long long)u * a.channels + ch] = total[c];
    }
}

// The gradient that reaches each unit from behind, in place of what the unit hands on.
__global__ void __launch_bounds__(256)
sel_carry_combine_kernel(const SelArgs a)
{
    griddep_entry();
    const long long width = (long long)a.channels * a.N, i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int seq = (int)(i / width);
    if (seq >= a.n_seqs)
        return;
    const long long e = i - seq * width;
    const int c = (int)(e / a.N), u0 = a.first[seq];
    const float A = a.A[e] * kLog2e;
    float g = a.grad_state ? a.grad_state[i] : 0.f;
    for (int u = a.first[seq + 1] - 1; u >= u0; --u) {
        float *p = a.unit_state + u * width + e;
        const float own = u > u0 ? *p : 0.f;
        *p = g;
        if (u > u0)
            g = fmaf(ex2(a.unit_step[(long long)u * a.channels + c] * A), g, own);
    }
}

template <int NP, int LN>
struct BackLayout {                                         // floats of a warp, then of the block
    static constexpr int CH = kBackCh, WC = 32 / LN * CH, NN = NP * LN, L = kSelChunk;
    static constexpr int kRow = L * WC;
    static constexpr int kKeep = L * 32 * CH * NP;          // k of every token: a lane's own values
    static constexpr int kSums = L * NN;                    // grad_B, grad_C of the warp's channels
    static constexpr int kWarp = kKeep + 5 * kRow + 2 * kSums;
    static constexpr size_t kBytes = ((size_t)kWarp * kSelWarps + 2 * kSums) * sizeof(float);   // B and C last
};

template <class T, int NP, int LN>
__global__ void __launch_bounds__(32 * kSelWarps)
sel_backward_kernel(const SelArgs a)
{
    griddep_entry();
    using Y = BackLayout<NP, LN>;
    constexpr int CH = Y::CH, WC = Y::WC, NN = Y::NN, L = kSelChunk, KC = WC > 32 ? WC / 32 : 1;
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane % LN, q = lane / LN, n0 = sub * NP;
    const int u = blockIdx.x / a.cblocks, cblock = blockIdx.x - u * a.cblocks;
    const SelTile tile = sel_tile<WC>(a, cblock, warp);
    SelUnit s;
    if (!sel_unit(a, u, s))                                 // (the whole block)
        return;
    const int wc = tile.c1 - tile.c0;
    const bool pad = a.N != NN;
    const bool vec_c = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.chunk_states) & 15) == 0;
    float *w = sm + warp * Y::kWarp;
    float *keep = w, *step = keep + Y::kKeep, *in = step + Y::kRow, *gs = in + Y::kRow, *sa = gs + Y::kRow, *eb = sa + Y::kRow;
    float *sB = eb + Y::kRow, *sC = sB + Y::kSums, *Bs = sm + kSelWarps * Y::kWarp, *Cs = Bs + Y::kSums;
    float2 e[CH][NP / 2], A[CH][NP / 2], gA[CH][NP / 2];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = tile.c0 + q * CH + c;
        const bool there = q * CH + c < wc;
        read_states<NP>(A[c], a.A + (long long)ch * a.N, n0, a.N, false, there);
        if (a.seg)
            read_states<NP>(e[c], a.unit_state + ((long long)u * a.channels + ch) * a.N, n0, a.N, a.N % 4 == 0, there);
        else
            read_states<NP>(e[c], a.grad_state + ((long long)s.seq * a.channels + ch) * a.N, n0, a.N, false,
                            there && a.grad_state != nullptr);
#pragma unroll
        for (int j = 0; j < NP / 2; ++j) {
            A[c][j] = make_float2(A[c][j].x * kLog2e, A[c][j].y * kLog2e);
            gA[c][j] = make_float2(0.f, 0.f);
        }
    }
    float bias[KC], D[KC], gD[KC], gbias[KC];
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        const int c = (lane + 32 * k) % WC;
        bias[k] = a.bias && c < wc ? __ldg(a.bias + tile.c0 + c) : 0.f;
        D[k] = a.D && c < wc ? __ldg(a.D + tile.c0 + c) : 0.f;
        gD[k] = gbias[k] = 0.f;
    }
    const T *x = static_cast<const T *>(a.x) + tile.c0, *dt = static_cast<const T *>(a.dt) + tile.c0;
    const T *z = a.z ? static_cast<const T *>(a.z) + tile.c0 : nullptr, *gy = static_cast<const T *>(a.grad_y) + tile.c0;
    const T *B = static_cast<const T *>(a.B) + tile.g * a.N, *C = static_cast<const T *>(a.C) + tile.g * a.N;
    T *gx = static_cast<T *>(a.grad_x) + tile.c0, *gdt = static_cast<T *>(a.grad_dt) + tile.c0;
    T *gz = z ? static_cast<T *>(a.grad_z) + tile.c0 : nullptr;
    const long long row_n = (long long)a.groups * a.N;      // a row of the partial sums of grad_B and grad_C

    for (int b = s.end > s.begin ? s.begin + (s.end - 1 - s.begin) / L * L : -1; b >= s.begin; b -= L) {
        const int cnt = min(L, s.end - b);
        const long long t0 = s.t0 + b;
#pragma unroll 4
        for (int m = 0; m < L * WC / 32; ++m) {
            const int i = lane + 32 * m, t = i / WC, c = i % WC;
            float st = 0.f, xv = 0.f, gv = 0.f, slope;
            if (t < cnt && c < wc) {
                st = sel_step(to_float(dt[(t0 + t) * a.sdt + c]) + bias[m % KC], a.softplus, slope);
                xv = to_float(x[(t0 + t) * a.sx + c]);
                gv = to_float(gy[(t0 + t) * a.sgy + c]);
                if (z) {
                    const float g = to_float(z[(t0 + t) * a.sz + c]);
                    gv *= g * sigmoid_of(g);
                }
            }
            step[i] = st;
            in[i] = st * xv;
            gs[i] = gv;
        }
        stage_rows<T, NN>(Bs, B + t0 * a.sB, a.sB, a.N, cnt);
        stage_rows<T, NN>(Cs, C + t0 * a.sC, a.sC, a.N, cnt);
        float2 h[CH][NP / 2];
        const float *cs = a.chunk_states + sel_chunk_row(a.n_seqs, s.seq, s.t0, b / L) * a.channels * a.N;
#pragma unroll
        for (int c = 0; c < CH; ++c)
            read_states<NP>(h[c], cs + (long long)(tile.c0 + q * CH + c) * a.N, n0, a.N, vec_c, q * CH + c < wc);
        __syncthreads();
        for (int t = 0; t < cnt; ++t) {
            float st[CH], uv[CH], gv[CH], p[CH], gc[NP];
            float2 Bv[NP / 2], Cv[NP / 2], sum_c[NP / 2];
            load_floats<CH>(st, step + t * WC + q * CH);
            load_floats<CH>(uv, in + t * WC + q * CH);
            load_floats<CH>(gv, gs + t * WC + q * CH);
            load_pairs<NP>(Bv, Bs + t * NN + n0);
            load_pairs<NP>(Cv, Cs + t * NN + n0);
#pragma unroll
            for (int j = 0; j < NP / 2; ++j)
                sum_c[j] = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float2 sum = make_float2(0.f, 0.f), k[NP / 2];
#pragma unroll
                for (int j = 0; j < NP / 2; ++j) {
                    k[j] = mul2(ex2_2(mul2(twice(st[c]), A[c][j])), h[c][j]);
                    h[c][j] = fma2(twice(uv[c]), Bv[j], k[j]);
                }
                if (pad)
                    drop_padding<NP>(h[c], n0, a.N);
#pragma unroll
                for (int j = 0; j < NP / 2; ++j) {
                    sum = fma2(h[c][j], Cv[j], sum);
                    sum_c[j] = fma2(twice(gv[c]), h[c][j], sum_c[j]);
                }
#pragma unroll
                for (int j = 0; j < NP / 2; j += 2)
                    *reinterpret_cast<float4 *>(keep + ((t * CH + c) * (NP / 4) + j / 2) * 128 + 4 * lane) =
                        make_float4(k[j].x, k[j].y, k[j + 1].x, k[j + 1].y);
                p[c] = sum.x + sum.y;
            }
#pragma unroll
            for (int j = 0; j < NP / 2; ++j) {
                gc[2 * j] = sum_c[j].x;
                gc[2 * j + 1] = sum_c[j].y;
            }
            int at;
            bool mine;
            if (z) {
                lanes_sum<CH, LN, 1>(p, lane, at, mine);
                if (mine)
#pragma unroll
                    for (int r = 0; r < (CH > LN ? CH / LN : 1); ++r)
                        sa[t * WC + q * CH + at + r] = p[r];
            }
            lanes_sum<NP, 32 / LN, LN>(gc, lane, at, mine);
            constexpr int kLeft = NP * LN > 32 ? NP * LN / 32 : 1;
            if (mine)
#pragma unroll
                for (int r = 0; r < kLeft; ++r)
                    sC[t * NN + n0 + at + r] = gc[r];
        }
        __syncwarp();
        if (z) {
#pragma unroll 4
            for (int m = 0; m < L * WC / 32; ++m) {
                const int i = lane + 32 * m, t = i / WC, c = i % WC;
                if (t < cnt && c < wc) {
                    const float g = to_float(z[(t0 + t) * a.sz + c]), sg = sigmoid_of(g);
                    const float p = fmaf(D[m % KC], to_float(x[(t0 + t) * a.sx + c]), sa[i]);
                    gz[(t0 + t) * a.sgz + c] = from_float<T>(to_float(gy[(t0 + t) * a.sgy + c]) * p * fmaf(g * sg, 1.f - sg, sg));
                }
            }
            __syncwarp();
        }
        for (int t = cnt - 1; t >= 0; --t) {
            float st[CH], uv[CH], gv[CH], s1[CH], s2[CH], gb[NP];
            float2 Bv[NP / 2], Cv[NP / 2], sum_b[NP / 2];
            load_floats<CH>(st, step + t * WC + q * CH);
            load_floats<CH>(uv, in + t * WC + q * CH);
            load_floats<CH>(gv, gs + t * WC + q * CH);
            load_pairs<NP>(Bv, Bs + t * NN + n0);
            load_pairs<NP>(Cv, Cs + t * NN + n0);
#pragma unroll
            for (int j = 0; j < NP / 2; ++j)
                sum_b[j] = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float2 k[NP / 2], wa = make_float2(0.f, 0.f), wb = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < NP / 2; j += 2) {
                    const float4 v = *reinterpret_cast<const float4 *>(keep + ((t * CH + c) * (NP / 4) + j / 2) * 128 + 4 * lane);
                    k[j] = make_float2(v.x, v.y);
                    k[j + 1] = make_float2(v.z, v.w);
                }
#pragma unroll
                for (int j = 0; j < NP / 2; ++j)
                    e[c][j] = fma2(twice(gv[c]), Cv[j], e[c][j]);
                if (pad) {
                    drop_padding<NP>(e[c], n0, a.N);
                    drop_padding<NP>(k, n0, a.N);
                }
#pragma unroll
                for (int j = 0; j < NP / 2; ++j) {
                    const float2 v = mul2(e[c][j], k[j]);
                    gA[c][j] = fma2(twice(st[c]), v, gA[c][j]);
                    wa = fma2(v, A[c][j], wa);
                    wb = fma2(e[c][j], Bv[j], wb);
                    sum_b[j] = fma2(twice(uv[c]), e[c][j], sum_b[j]);
                    e[c][j] = mul2(ex2_2(mul2(twice(st[c]), A[c][j])), e[c][j]);
                }
                s1[c] = wa.x + wa.y;
                s2[c] = wb.x + wb.y;
            }
#pragma unroll
            for (int j = 0; j < NP / 2; ++j) {
                gb[2 * j] = sum_b[j].x;
                gb[2 * j + 1] = sum_b[j].y;
            }
            int at;
            bool mine;
            lanes_sum<CH, LN, 1>(s1, lane, at, mine);
            lanes_sum<CH, LN, 1>(s2, lane, at, mine);
            if (mine)
#pragma unroll
                for (int r = 0; r < (CH > LN ? CH / LN : 1); ++r) {
                    sa[t * WC + q * CH + at + r] = s1[r];
                    eb[t * WC + q * CH + at + r] = s2[r];
                }
            lanes_sum<NP, 32 / LN, LN>(gb, lane, at, mine);
            constexpr int kLeft = NP * LN > 32 ? NP * LN / 32 : 1;
            if (mine)
#pragma unroll
                for (int r = 0; r < kLeft; ++r)
                    sB[t * NN + n0 + at + r] = gb[r];
        }
        __syncthreads();                                    // every warp's sums over its channels are there
        for (int i = tid; i < cnt * NN; i += 32 * kSelWarps) {
            const int t = i / NN, n = i % NN;
            if (n < a.N) {
                float vb = 0.f, vc = 0.f;
#pragma unroll
                for (int k = 0; k < kSelWarps; ++k) {
                    const float *o = sm + k * Y::kWarp + (sB - w);
                    vb += o[i];
                    vc += o[i + Y::kSums];
                }
                const long long at = ((long long)(cblock % (a.cblocks / a.groups)) * a.n_tokens + t0 + t) * row_n + tile.g * a.N + n;
                a.part_B[at] = vb;
                a.part_C[at] = vc;
            }
        }
#pragma unroll 4
        for (int m = 0; m < L * WC / 32; ++m) {
            const int i = lane + 32 * m, t = i / WC, c = i % WC;
            if (t < cnt && c < wc) {
                const float xv = to_float(x[(t0 + t) * a.sx + c]), gv = gs[i], st = step[i];
                float slope;
                sel_step(to_float(dt[(t0 + t) * a.sdt + c]) + bias[m % KC], a.softplus, slope);
                const float g = fmaf(sa[i], kLn2, xv * eb[i]) * slope;
                gx[(t0 + t) * a.sgx + c] = from_float<T>(fmaf(D[m % KC], gv, st * eb[i]));
                gdt[(t0 + t) * a.sgdt + c] = from_float<T>(g);
                gD[m % KC] = fmaf(gv, xv, gD[m % KC]);
                gbias[m % KC] += g;
            }
        }
        __syncthreads();                                    // ... and read
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = tile.c0 + q * CH + c;
        if (q * CH + c >= wc)
            continue;
        write_states<NP>(a.part_A + ((long long)u * a.channels + ch) * a.N, gA[c], n0, a.N, a.N % 4 == 0);
        if (s.k == 0 && a.grad_state0) {
            const bool resumed = a.resume[s.seq] != 0;
#pragma unroll
            for (int j = 0; j < NP / 2; ++j)
                e[c][j] = resumed ? e[c][j] : make_float2(0.f, 0.f);
            write_states<NP>(a.grad_state0 + ((long long)s.seq * a.channels + ch) * a.N, e[c], n0, a.N, false);
        }
    }
    // lanes that hold the same channel
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        if constexpr (WC < 32) {
#pragma unroll
            for (int off = 16; off >= WC; off /= 2) {
                gD[k] += __shfl_xor_sync(kFullMask, gD[k], off);
                gbias[k] += __shfl_xor_sync(kFullMask, gbias[k], off);
            }
        }
        const int c = (lane + 32 * k) % WC;
        if (c < wc && lane + 32 * k < (WC < 32 ? WC : 32 * KC)) {
            a.part_D[(long long)u * a.channels + tile.c0 + c] = gD[k];
            a.part_bias[(long long)u * a.channels + tile.c0 + c] = gbias[k];
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

template <class T, int NP, int LN>
cudaError_t launch_shape(const SelArgs &a, cudaStream_t st)
{
    const dim3 block(32 * kSelWarps);
    cudaError_t e;
    if (a.seg) {
        const int cblocks = a.groups * sel_group_blocks(a.channels, a.groups, 32 / LN * 4);
        e = launch_pdl(sel_carry_kernel<T, NP, LN>, dim3((unsigned)((long long)a.max_units * cblocks)), block, 0, st, a);
        if (e != cudaSuccess)
            return e;
        const long long n = (long long)a.n_seqs * a.channels * a.N;
        e = launch_pdl(sel_carry_combine_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, a);
        if (e != cudaSuccess)
            return e;
    }
    const auto kernel = sel_backward_kernel<T, NP, LN>;
    constexpr size_t bytes = BackLayout<NP, LN>::kBytes;
    e = set_dynamic_smem(reinterpret_cast<const void *>(kernel), bytes);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kernel, dim3((unsigned)((long long)a.max_units * a.cblocks)), block, bytes, st, a);
}

template <class T>
cudaError_t launch_type(const SelArgs &a, cudaStream_t st)
{
    cudaError_t e = a.N <= 8     ? launch_shape<T, 4, 2>(a, st)
                    : a.N <= 16  ? launch_shape<T, 4, 4>(a, st)
                    : a.N <= 32  ? launch_shape<T, 4, 8>(a, st)
                    : a.N <= 64  ? launch_shape<T, 4, 16>(a, st)
                                 : launch_shape<T, 4, 32>(a, st);
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
    return layout(n_seqs, n_tokens, channels, N, groups, sel_segment(n_seqs, n_tokens, s, true), s.cblocks).total;
}

cudaError_t launch_selective_scan_backward(SelArgs a, int dtype, void *workspace, cudaStream_t st)
{
    const SelShape s = sel_shape(a.channels, a.N, a.groups, true);
    a.cblocks = s.cblocks;
    a.seg = sel_segment(a.n_seqs, a.n_tokens, s, true);
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
