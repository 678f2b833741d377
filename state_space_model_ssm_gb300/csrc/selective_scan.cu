// Selective scan with a decay for each channel and state, forward (sm_103a).
// Formulas and the layout of a warp: selective_common.cuh.
//
// sel_scan_kernel walks a unit's tokens in chunks of 16: the warp turns dt and x of its
// channels into steps and inputs in shared memory (lanes along channels), walks the
// chunk's tokens with the states in registers, and turns the sums over states into
// outputs (lanes along channels again).  A block's warps share the chunk's B and C, in two
// buffers: one barrier a chunk.
#include "selective_common.cuh"

namespace ssm {

namespace {

template <class T, int NP, int LN, int CH, bool STATE_ONLY>
__global__ void __launch_bounds__(32 * kSelWarps)
sel_scan_kernel(const SelArgs a)
{
    griddep_entry();
    constexpr int WC = 32 / LN * CH, NN = NP * LN, L = kSelChunk, KC = WC > 32 ? WC / 32 : 1;
    __shared__ __align__(16) float s_step[kSelWarps][L * WC], s_in[kSelWarps][L * WC];
    extern __shared__ __align__(16) float s_rows[];         // [2][B, C][L * NN]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane % LN, q = lane / LN, n0 = sub * NP;
    const int u = blockIdx.x / a.cblocks;
    const SelTile tile = sel_tile<WC>(a, blockIdx.x - u * a.cblocks, warp);
    SelUnit s;
    if (!sel_unit(a, u, s) || (STATE_ONLY && s.last))       // (the whole block)
        return;
    const int wc = tile.c1 - tile.c0;                       // channels of this warp that exist
    const bool vec = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
    const bool vec_c = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.chunk_states) & 15) == 0;
    const bool pad = a.N != NN;
    float *step = s_step[warp], *in = s_in[warp];

    float2 h[CH][NP / 2], A[CH][NP / 2];
    float total[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = tile.c0 + q * CH + c;
        const bool there = q * CH + c < wc;
        read_states<NP>(A[c], a.A + (long long)ch * a.N, n0, a.N, false, there);
#pragma unroll
        for (int j = 0; j < NP / 2; ++j)
            A[c][j] = make_float2(A[c][j].x * kLog2e, A[c][j].y * kLog2e);
        if (STATE_ONLY)
            read_states<NP>(h[c], nullptr, n0, a.N, false, false);
        else if (a.seg)
            read_states<NP>(h[c], a.unit_state + ((long long)u * a.channels + ch) * a.N, n0, a.N, a.N % 4 == 0, there);
        else
            read_states<NP>(h[c], a.state + ((long long)s.seq * a.channels + ch) * a.N, n0, a.N, vec,
                            there && a.resume[s.seq] != 0);
        total[c] = 0.f;
    }
    // this lane's channels while staging
    float bias[KC], D[KC];
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        const int c = (lane + 32 * k) % WC;
        bias[k] = a.bias && c < wc ? __ldg(a.bias + tile.c0 + c) : 0.f;
        D[k] = a.D && c < wc ? __ldg(a.D + tile.c0 + c) : 0.f;
    }
    const T *x = static_cast<const T *>(a.x) + tile.c0, *dt = static_cast<const T *>(a.dt) + tile.c0;
    const T *z = a.z ? static_cast<const T *>(a.z) + tile.c0 : nullptr;
    T *y = STATE_ONLY ? nullptr : static_cast<T *>(a.y) + tile.c0;
    const T *B = static_cast<const T *>(a.B) + tile.g * a.N, *C = static_cast<const T *>(a.C) + tile.g * a.N;

    for (int b = s.begin; b < s.end; b += L) {
        const int cnt = min(L, s.end - b);
        const long long t0 = s.t0 + b;
        float *Bs = s_rows + (b / L & 1) * 2 * L * NN, *Cs = Bs + L * NN;
        if (!STATE_ONLY && a.chunk_states) {
            float *cs = a.chunk_states + sel_chunk_row(a.n_seqs, s.seq, s.t0, b / L) * a.channels * a.N;
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (q * CH + c < wc)
                    write_states<NP>(cs + (long long)(tile.c0 + q * CH + c) * a.N, h[c], n0, a.N, vec_c);
        }
#pragma unroll 4
        for (int m = 0; m < L * WC / 32; ++m) {
            const int i = lane + 32 * m, t = i / WC, c = i % WC;
            float st = 0.f, xv = 0.f, slope;
            if (t < cnt && c < wc) {
                st = sel_step(to_float(dt[(t0 + t) * a.sdt + c]) + bias[m % KC], a.softplus, slope);
                xv = to_float(x[(t0 + t) * a.sx + c]);
            }
            step[i] = st;
            in[i] = st * xv;
        }
        stage_rows<T, NN>(Bs, B + t0 * a.sB, a.sB, a.N, cnt);
        if (!STATE_ONLY)
            stage_rows<T, NN>(Cs, C + t0 * a.sC, a.sC, a.N, cnt);
        __syncthreads();
        for (int t = 0; t < cnt; ++t) {
            float st[CH], uv[CH], p[CH];
            float2 Bv[NP / 2], Cv[NP / 2];
            load_floats<CH>(st, step + t * WC + q * CH);
            load_floats<CH>(uv, in + t * WC + q * CH);
            load_pairs<NP>(Bv, Bs + t * NN + n0);
            if (!STATE_ONLY)
                load_pairs<NP>(Cv, Cs + t * NN + n0);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float2 sum = make_float2(0.f, 0.f);
                if (STATE_ONLY)
                    total[c] += st[c];
#pragma unroll
                for (int j = 0; j < NP / 2; ++j) {
                    const float2 decay = ex2_2(mul2(twice(st[c]), A[c][j]));
                    h[c][j] = fma2(decay, h[c][j], mul2(twice(uv[c]), Bv[j]));
                }
                if (pad)
                    drop_padding<NP>(h[c], n0, a.N);
                if (!STATE_ONLY)
#pragma unroll
                    for (int j = 0; j < NP / 2; ++j)
                        sum = fma2(h[c][j], Cv[j], sum);
                p[c] = sum.x + sum.y;
            }
            if (!STATE_ONLY) {
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
        if (!STATE_ONLY) {
#pragma unroll 4
            for (int m = 0; m < L * WC / 32; ++m) {
                const int i = lane + 32 * m, t = i / WC, c = i % WC;
                if (t < cnt && c < wc) {
                    float v = in[i];
                    if (a.D)
                        v = fmaf(D[m % KC], to_float(x[(t0 + t) * a.sx + c]), v);
                    if (z) {
                        const float g = to_float(z[(t0 + t) * a.sz + c]);
                        v *= g * sigmoid_of(g);
                    }
                    y[(t0 + t) * a.sy + c] = from_float<T>(v);
                }
            }
            __syncwarp();
        }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = tile.c0 + q * CH + c;
        if (q * CH + c >= wc)
            continue;
        if (STATE_ONLY) {
            write_states<NP>(a.unit_state + ((long long)u * a.channels + ch) * a.N, h[c], n0, a.N, a.N % 4 == 0);
            if (sub == 0)
                a.unit_step[(long long)u * a.channels + ch] = total[c];
        } else if (s.last) {
            write_states<NP>(a.state + ((long long)s.seq * a.channels + ch) * a.N, h[c], n0, a.N, vec);
        }
    }
}

// Units of every sequence: as many segments as its tokens take, one at least.
__global__ void __launch_bounds__(1024)
sel_plan_kernel(const SelArgs a, int2 *units, int *first)
{
    griddep_entry();
    __shared__ int sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int base = 0;
    for (int s0 = 0; s0 < a.n_seqs; s0 += 1024) {
        const int seq = s0 + tid;
        long long t0;
        const int mine = seq < a.n_seqs ? max(1, (sel_seq_len(a, seq, t0) + a.seg - 1) / a.seg) : 0;
        int incl = mine;
        for (int off = 1; off < 32; off *= 2) {
            const int v = __shfl_up_sync(kFullMask, incl, off);
            if (lane >= off)
                incl += v;
        }
        if (lane == 31)
            sums[warp] = incl;
        __syncthreads();
        int before = base, all = 0;
        for (int w = 0; w < 32; ++w) {
            before += w < warp ? sums[w] : 0;
            all += sums[w];
        }
        const int at = before + incl - mine;
        if (seq < a.n_seqs) {
            first[seq] = min(at, a.max_units);
            for (int k = 0; k < mine && at + k < a.max_units; ++k)   // (ranges that overlap could take more)
                units[at + k] = make_int2(seq, k);
        }
        base += all;
        __syncthreads();
    }
    if (tid == 0)
        first[a.n_seqs] = min(base, a.max_units);
}

// The state entering each unit, in place of the unit's state from zero.
__global__ void __launch_bounds__(256)
sel_combine_kernel(const SelArgs a)
{
    griddep_entry();
    const long long width = (long long)a.channels * a.N, i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int seq = (int)(i / width);
    if (seq >= a.n_seqs)
        return;
    const long long e = i - seq * width;
    const int c = (int)(e / a.N), u1 = a.first[seq + 1];
    const float A = a.A[e] * kLog2e;
    float h = a.resume[seq] != 0 ? a.state[i] : 0.f;
    for (int u = a.first[seq]; u < u1; ++u) {
        float *p = a.unit_state + u * width + e;
        const float own = u + 1 < u1 ? *p : 0.f;
        *p = h;
        if (u + 1 < u1)
            h = fmaf(ex2(a.unit_step[(long long)u * a.channels + c] * A), h, own);
    }
}

template <class T, int NP, int LN>
cudaError_t launch_shape(const SelArgs &a, int units, cudaStream_t st)
{
    const dim3 grid((unsigned)((long long)units * a.cblocks)), block(32 * kSelWarps);
    constexpr size_t bytes = 4 * kSelChunk * NP * LN * sizeof(float);
    if (a.seg) {
        cudaError_t e = launch_pdl(sel_scan_kernel<T, NP, LN, 4, true>, grid, block, bytes, st, a);
        if (e != cudaSuccess)
            return e;
        const long long n = (long long)a.n_seqs * a.channels * a.N;
        e = launch_pdl(sel_combine_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, a);
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(sel_scan_kernel<T, NP, LN, 4, false>, grid, block, bytes, st, a);
}

template <class T>
cudaError_t launch_type(const SelArgs &a, int units, cudaStream_t st)
{
    if (a.N <= 8) return launch_shape<T, 4, 2>(a, units, st);
    if (a.N <= 16) return launch_shape<T, 4, 4>(a, units, st);
    if (a.N <= 32) return launch_shape<T, 4, 8>(a, units, st);
    if (a.N <= 64) return launch_shape<T, 4, 16>(a, units, st);
    return launch_shape<T, 4, 32>(a, units, st);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

long long sel_chunk_rows(long long n_seqs, long long n_tokens) { return n_seqs + n_tokens / kSelChunk + 1; }

SelShape sel_shape(int channels, int N, int groups, bool backward)
{
    const int lanes = N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32;
    SelShape s;
    s.wc = 32 / lanes * (backward ? 2 : 4);
    s.cblocks = groups * sel_group_blocks(channels, groups, s.wc);
    s.tiles = groups * ((channels / groups + s.wc - 1) / s.wc);
    return s;
}

int sel_segment(int n_seqs, int n_tokens, const SelShape &s, bool backward)
{
    // warps that walk whole sequences, against what keeps the device busy
    const long long want = kSms * (backward ? 8 : 16), walk = (long long)n_seqs * s.tiles;
    if (walk >= want || n_tokens < 128 || n_tokens / n_seqs < 64)
        return 0;
    long long seg = (long long)n_tokens * s.tiles / want / kSelChunk * kSelChunk;
    return (int)(seg < 64 ? 64 : seg);
}

int sel_max_units(int n_seqs, int n_tokens, int seg) { return seg ? n_seqs + n_tokens / seg : n_seqs; }

cudaError_t launch_sel_plan(const SelArgs &a, int2 *units, int *first, cudaStream_t st)
{
    return launch_pdl(sel_plan_kernel, dim3(1), dim3(1024), 0, st, a, units, first);
}

namespace {
struct Workspace {
    size_t units, first, state, step, total;
};
Workspace layout(int n_seqs, int channels, int N, int units)
{
    Workspace w;
    w.units = 0;
    w.first = up256((size_t)units * sizeof(int2));
    w.state = w.first + up256(((size_t)n_seqs + 1) * 4);
    w.step = w.state + up256((size_t)units * channels * N * 4);
    w.total = w.step + up256((size_t)units * channels * 4);
    return w;
}
}  // namespace

size_t sel_scan_workspace_bytes(int n_seqs, int n_tokens, int channels, int N, int groups)
{
    const int seg = sel_segment(n_seqs, n_tokens, sel_shape(channels, N, groups, false), false);
    return seg ? layout(n_seqs, channels, N, sel_max_units(n_seqs, n_tokens, seg)).total : 0;
}

cudaError_t launch_selective_scan(SelArgs a, int dtype, void *workspace, cudaStream_t st)
{
    const SelShape s = sel_shape(a.channels, a.N, a.groups, false);
    a.cblocks = s.cblocks;
    a.seg = sel_segment(a.n_seqs, a.n_tokens, s, false);
    const int units = sel_max_units(a.n_seqs, a.n_tokens, a.seg);
    a.max_units = units;
    if (a.seg) {
        unsigned char *w = static_cast<unsigned char *>(workspace);
        const Workspace l = layout(a.n_seqs, a.channels, a.N, units);
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
    case kF32: return launch_type<float>(a, units, st);
    case kBF16: return launch_type<__nv_bfloat16>(a, units, st);
    case kF16: return launch_type<__half>(a, units, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssm
