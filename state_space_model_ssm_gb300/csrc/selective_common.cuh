// Shared parts of the selective scan with a decay for each channel and state
// (selective_scan.cu, selective_scan_backward.cu).
//
//   v = dt + dt_bias, step = v, or softplus(v) = v > 20 ? v : log1p(exp(v))
//   h[c,n] <- exp(step[c] A[c,n]) h[c,n] + step[c] x[c] B[g,n]
//   p[c] = sum_n h[c,n] C[g,n] + D[c] x[c],   y[c] = p[c] z[c] sigmoid(z[c])
//
// Every state has its own decay, so there is no matrix form: the work is one
// exponential and about five multiplications an element (token, channel, state).
// A warp owns a tile of channels with all their states: LN lanes share CH channels
// and each holds NP of their states, so a lane has CH x NP independent recurrences
// in registers.  What a lane reads from shared memory for a token (CH steps and inputs,
// NP values of B and of C) serves all of them: with single channels a lane
// the reads of B and C cost more than the arithmetic.  Two states go into one packed fp32
// instruction; the exponential is the hardware's 2^x of the rounded product
// step * (A log2(e)), within 2 ulp and 2^-24 of its argument.
//
// Time: a unit is a sequence, or, of a sequence so long that others would have to wait for it, a
// segment of `seg` tokens.  Of those a pass before composes each segment's state from zero, and a
// small one walks the segments.  The lengths are on the device, so a plan made there says which
// sequences are cut; the host says from which length on.
#pragma once

#include "packed.cuh"

namespace ssm {

constexpr int kSelChunk = 16;             // tokens for each of which training saves a state
constexpr int kSelCh = 4;                 // channels of a lane (two in the walks of small calls)
constexpr int kSelWarps = 4;              // warps of a block: neighbouring channel tiles of one unit
constexpr int kSelMaxState = 128;
constexpr int kCombineRun = 8;            // units whose loads the combining kernels issue together

struct SelArgs {
    float *state;
    const void *x, *dt, *z, *B, *C;
    const float *A, *D, *bias;
    void *y;
    const int32_t *starts, *lens, *resume;
    int n_seqs, n_tokens, channels, N, groups, softplus;
    long long sx, sdt, sz, sB, sC, sy;
    float *chunk_states;
    int seg, whole;                       // tokens of a segment (0: units are sequences); of the longest sequence left whole
    const int2 *units;                    // (sequence, segment)
    const int *first;                     // [n_seqs + 1]: a sequence's first unit; the last entry: how many there are
    float *unit_state, *unit_step;        // [units][channels][N], [units][channels]
    // backward
    const void *grad_y;
    const float *grad_state;
    long long sgy, sgx, sgdt, sgz, sgB, sgC;
    void *grad_x, *grad_dt, *grad_z, *grad_B, *grad_C;
    float *grad_A, *grad_D, *grad_bias, *grad_state0;
    float *part_A, *part_D, *part_bias;   // [units][channels][N], [units][channels] twice
    float *part_B, *part_C;               // [channel blocks][n_tokens][groups N]
    int max_units, cblocks;
    int pairs, narrow;                    // two channels of every row are one aligned word; tiles of the walks
};

// Row of chunk_states for chunk j of a sequence that starts at token t0: the first chunk's by
// the sequence, the others' by their position.  n_seqs + n_tokens / 16 + 1 rows.
__host__ __device__ __forceinline__ long long sel_chunk_row(int n_seqs, int seq, long long t0, int j)
{
    return j == 0 ? seq : n_seqs + t0 / kSelChunk + j;
}

// A sequence's token range; one that is not inside the packed rows counts as empty.
__device__ __forceinline__ int sel_seq_len(const SelArgs &a, int seq, long long &t0)
{
    t0 = a.starts[seq];
    const long long len = a.lens[seq];
    if (t0 >= 0 && len > 0 && t0 + len <= a.n_tokens)
        return (int)len;
    t0 = 0;
    return 0;
}

// A unit: tokens [begin, end) of sequence seq, whose first token is t0.
struct SelUnit {
    int seq, k, begin, end, len;
    long long t0;
    bool last, cut;                       // the last of its sequence; one of several
};

__device__ __forceinline__ bool sel_unit(const SelArgs &a, int u, SelUnit &s)
{
    s.seq = u;
    s.k = 0;
    if (a.seg) {
        if (u >= a.first[a.n_seqs])
            return false;
        const int2 v = a.units[u];
        s.seq = v.x;
        s.k = v.y;
    }
    s.len = sel_seq_len(a, s.seq, s.t0);
    s.cut = a.seg && a.first[s.seq + 1] - a.first[s.seq] > 1;
    s.begin = s.cut ? a.seg * s.k : 0;
    s.end = s.cut ? min(s.len, s.begin + a.seg) : s.len;
    s.last = s.end == s.len;
    return true;
}

// Channel tiles: WC channels of one group; a block has kSelWarps neighbours of one group.
struct SelTile {
    int c0, c1, g;                        // channels [c0, c1), at most WC of them
};

__host__ __device__ __forceinline__ int sel_group_blocks(int channels, int groups, int wc)
{
    return (channels / groups + wc * kSelWarps - 1) / (wc * kSelWarps);
}

template <int WC>
__device__ __forceinline__ SelTile sel_tile(const SelArgs &a, int cblock, int warp)
{
    const int per = sel_group_blocks(a.channels, a.groups, WC), cg = a.channels / a.groups;
    SelTile t;
    t.g = cblock / per;
    const int in_group = ((cblock - t.g * per) * kSelWarps + warp) * WC;
    t.c0 = t.g * cg + min(in_group, cg);
    t.c1 = t.g * cg + min(in_group + WC, cg);
    return t;
}

// ---- arithmetic ----

__device__ __forceinline__ float2 ex2_2(float2 v) { return make_float2(ex2(v.x), ex2(v.y)); }

// The discretised step of two values.  softplus(v) = max(v, 0) + log1p(e) with e = exp(-|v|), and
// log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3: the series 2 s (1 + s^2/3 + s^4/5 + ...) to s^14
// leaves (1/9)^8 / 17 < 2^-29 of it, and keeps the relative accuracy of small e, which a
// logarithm of 1 + e would lose.  All together within (3|v| + 18) 2^-24 of the step.
__device__ __forceinline__ float2 sel_step2(float2 v, bool softplus)
{
    if (!softplus)
        return v;
    const float2 e = make_float2(ex2(-fabsf(v.x) * kLog2e), ex2(-fabsf(v.y) * kLog2e));
    const float2 s = mul2(e, rcp2(add2(e, twice(2.f)))), q = mul2(s, s);
    float2 r = fma2(q, twice(1.f / 15), twice(1.f / 13));
    r = fma2(q, r, twice(1.f / 11));
    r = fma2(q, r, twice(1.f / 9));
    r = fma2(q, r, twice(1.f / 7));
    r = fma2(q, r, twice(1.f / 5));
    r = fma2(q, r, twice(1.f / 3));
    const float2 s2 = add2(s, s);
    r = fma2(mul2(s2, q), r, s2);
    return make_float2(v.x > 20.f ? v.x : fmaxf(v.x, 0.f) + r.x, v.y > 20.f ? v.y : fmaxf(v.y, 0.f) + r.y);
}

// Its derivative by v: 1 above the threshold, else sigmoid(v).
__device__ __forceinline__ float2 sel_slope2(float2 v, bool softplus)
{
    if (!softplus)
        return twice(1.f);
    const float2 s = rcp2(make_float2(1.f + ex2(-v.x * kLog2e), 1.f + ex2(-v.y * kLog2e)));
    return make_float2(v.x > 20.f ? 1.f : s.x, v.y > 20.f ? 1.f : s.y);
}

// A state h behind a whole segment: 2^x h + own, x the sum of its tokens' exponents.  2^x alone can overflow where the
// product does not, and where h is 0 (decays that grow: A above 0, or negative steps), so it goes in two
// factors that are never infinite; between -126 and 127 the second is 1.  From 2^254 on the product overflows for
// every normal h, below 2^-252 it is nothing beside own.  A zero stays zero, an infinity infinite, as token by
// token; a step that is no number is in own already.
__device__ __forceinline__ float sel_passed(float h, float x, float own)
{
    const float first = fminf(fmaxf(x, -126.f), 127.f), second = fminf(fmaxf(x - first, -126.f), 127.f);
    return fmaf(h * ex2(second), ex2(first), own);
}

// How a warp stages pairs of channels of up to L tokens: place m of a lane is token tok(m), pair cp(m).
template <int WC, int L>
struct SelStage {
    static constexpr int P = WC / 2, KC = P >= 32 ? P / 32 : 1, TI = P >= 32 ? 1 : 32 / P;
    static constexpr int M = L * P / 32 > 0 ? L * P / 32 : 1, kTokens = L > TI ? L : TI;   // (places past L are staged and not used)
    static_assert(kTokens % TI == 0, "whole places");
    static __device__ __forceinline__ int tok(int m, int lane) { return P >= 32 ? m / KC : m * TI + lane / P; }
    static __device__ __forceinline__ int cp(int m, int lane) { return P >= 32 ? lane + 32 * (m % KC) : lane % P; }
};

// Places [m0, m0 + CNT) of cnt tokens' rows at `p` (the tile's first channel), all loads together: places past
// the last token or channel read the last one's (their values are not used).  `pairs`: two
// channels of a row are one aligned word.
template <class T, int WC, int L, int CNT>
__device__ __forceinline__ void load_places(RawPair<T> (&r)[CNT], int m0, const T *p, long long stride, int cnt, int wc, int lane,
                                            bool pairs)
{
    using S = SelStage<WC, L>;
    if (pairs) {
#pragma unroll
        for (int m = 0; m < CNT; ++m)
            r[m] = load_pair(p + min(S::tok(m0 + m, lane), cnt - 1) * stride + min(2 * S::cp(m0 + m, lane), wc - 2));
    } else {
#pragma unroll
        for (int m = 0; m < CNT; ++m) {
            const T *q = p + min(S::tok(m0 + m, lane), cnt - 1) * stride;
            const int c = 2 * S::cp(m0 + m, lane);
            r[m] = join_pair<T>(q[min(c, wc - 1)], q[min(c + 1, wc - 1)]);
        }
    }
}

template <class T>
__device__ __forceinline__ void store_pair(T *p, float2 v, bool pairs, bool second)
{
    if (pairs) {
        store_word(p, v);
    } else {
        p[0] = from_float<T>(v.x);
        if (second)
            p[1] = from_float<T>(v.y);
    }
}

// Parameters of a lane's channel pairs (zeros past the tile's channels).
template <int KC, int WC>
__device__ __forceinline__ void read_channels(float2 (&v)[KC], const float *p, int c0, int wc, int lane)
{
    using S = SelStage<WC, 16>;
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        const int c = 2 * S::cp(k, lane);
        v[k] = make_float2(p && c < wc ? __ldg(p + c0 + c) : 0.f, p && c + 1 < wc ? __ldg(p + c0 + c + 1) : 0.f);
    }
}

// CNT sums over LANES lanes STRIDE apart, each of the lanes ending with max(1, CNT / LANES) of
// them in v[0..]: as long as there are two values to a lane, a lane keeps half and sends
// the other.  `at`: which value v[0] is; `mine`: whether this lane is the first of
// those that hold the same.
template <int CNT, int LANES, int STRIDE>
__device__ __forceinline__ void lanes_sum(float (&v)[CNT], int lane, int &at, bool &mine)
{
    const int l = lane / STRIDE;
    at = 0;
    mine = true;
    int width = CNT;
#pragma unroll
    for (int off = LANES / 2; off >= 1; off /= 2) {
        const bool up = (l & off) != 0;
        if (width > 1) {
            width /= 2;
#pragma unroll
            for (int m = 0; m < CNT / 2; ++m)
                if (m < width) {
                    const float keep = up ? v[m + width] : v[m], send = up ? v[m] : v[m + width];
                    v[m] = keep + __shfl_xor_sync(kFullMask, send, off * STRIDE);
                }
            at += up ? width : 0;
        } else {
            v[0] += __shfl_xor_sync(kFullMask, v[0], off * STRIDE);
            mine = mine && !up;
        }
    }
}

// CH consecutive floats of shared memory.
template <int CH>
__device__ __forceinline__ void load_floats(float (&v)[CH], const float *p)
{
    if constexpr (CH % 4 == 0) {
#pragma unroll
        for (int i = 0; i < CH; i += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p + i);
            v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
        }
    } else if constexpr (CH % 2 == 0) {
#pragma unroll
        for (int i = 0; i < CH; i += 2) {
            const float2 q = *reinterpret_cast<const float2 *>(p + i);
            v[i] = q.x; v[i + 1] = q.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i)
            v[i] = p[i];
    }
}

template <int NP>
__device__ __forceinline__ void load_pairs(float2 (&v)[NP / 2], const float *p)
{
#pragma unroll
    for (int i = 0; i < NP / 4; ++i) {
        const float4 q = *reinterpret_cast<const float4 *>(p + 4 * i);
        v[2 * i] = make_float2(q.x, q.y);
        v[2 * i + 1] = make_float2(q.z, q.w);
    }
}

// A lane's NP states of one channel out of a row of N (and back): four at a time where rows allow.
template <int NP>
__device__ __forceinline__ void read_states(float2 (&v)[NP / 2], const float *row, int n0, int N, bool vec, bool there)
{
#pragma unroll
    for (int i = 0; i < NP; i += 4) {
        float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
        if (there && vec) {
            if (n0 + i < N)
                q = *reinterpret_cast<const float4 *>(row + n0 + i);
        } else if (there) {
            if (n0 + i < N) q.x = row[n0 + i];
            if (n0 + i + 1 < N) q.y = row[n0 + i + 1];
            if (n0 + i + 2 < N) q.z = row[n0 + i + 2];
            if (n0 + i + 3 < N) q.w = row[n0 + i + 3];
        }
        v[i / 2] = make_float2(q.x, q.y);
        v[i / 2 + 1] = make_float2(q.z, q.w);
    }
}

template <int NP>
__device__ __forceinline__ void write_states(float *row, const float2 (&v)[NP / 2], int n0, int N, bool vec)
{
#pragma unroll
    for (int i = 0; i < NP; i += 4) {
        const float4 q = make_float4(v[i / 2].x, v[i / 2].y, v[i / 2 + 1].x, v[i / 2 + 1].y);
        if (vec) {
            if (n0 + i < N)
                *reinterpret_cast<float4 *>(row + n0 + i) = q;
        } else {
            if (n0 + i < N) row[n0 + i] = q.x;
            if (n0 + i + 1 < N) row[n0 + i + 1] = q.y;
            if (n0 + i + 2 < N) row[n0 + i + 2] = q.z;
            if (n0 + i + 3 < N) row[n0 + i + 3] = q.w;
        }
    }
}

// States past the last one are zero, and stay so while steps and inputs are finite.  In a chunk where one is not
// they are set back after every token: 0 times infinity would make them NaN, and their zeros of C would not
// take that out of a sum.
template <int NP>
__device__ __forceinline__ void drop_padding(float2 (&v)[NP / 2], int n0, int N)
{
#pragma unroll
    for (int j = 0; j < NP / 2; ++j)
        v[j] = make_float2(n0 + 2 * j < N ? v[j].x : 0.f, n0 + 2 * j + 1 < N ? v[j].y : 0.f);
}

// L rows of N values of B or C by the block's threads: loads into registers, and later as fp32 rows of NN
// with zeros past N.
template <class T, int NN, int L>
struct SelRows {
    static constexpr int kEach = L * NN / (32 * kSelWarps) > 0 ? L * NN / (32 * kSelWarps) : 1;
    T v[kEach];
    __device__ __forceinline__ void load(const T *src, long long stride, int N, int cnt)
    {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int e = threadIdx.x + 32 * kSelWarps * i, t = e / NN, n = e % NN;
            v[i] = src[min(t, cnt - 1) * stride + min(n, N - 1)];
        }
    }
    __device__ __forceinline__ void store(float *dst, int N) const
    {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int e = threadIdx.x + 32 * kSelWarps * i, n = e % NN;
            if (L * NN >= 32 * kSelWarps || e < L * NN)
                dst[e] = n < N ? to_float(v[i]) : 0.f;
        }
    }
    __device__ __forceinline__ void store_twice(float2 *dst, int N) const
    {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int e = threadIdx.x + 32 * kSelWarps * i, n = e % NN;
            if (L * NN >= 32 * kSelWarps || e < L * NN)
                dst[e] = twice(n < N ? to_float(v[i]) : 0.f);
        }
    }
};

// Launches: host side of both passes (selective_scan.cu).
struct SelShape {
    int wc, cblocks, tiles;               // channels of a warp; blocks of channels; warps of channels
};
SelShape sel_shape(int channels, int N, int groups, bool backward);
// Tokens of a segment (0: units are sequences) and of the longest sequence that is left whole.
struct SelCut {
    int seg, whole;
};
SelCut sel_cut(int n_seqs, int n_tokens, int channels, int N, int groups, bool backward);
bool sel_narrow(int n_seqs, int n_tokens, int units, int tiles);
bool sel_pairs(const SelArgs &a, int dtype);
dim3 sel_combine_grid(const SelArgs &a);
int sel_max_units(int n_seqs, int n_tokens, int seg);
long long sel_chunk_rows(long long n_seqs, long long n_tokens);
cudaError_t launch_sel_plan(const SelArgs &a, int2 *units, int *first, cudaStream_t st);   // a.max_units bounds it
size_t sel_scan_workspace_bytes(int n_seqs, int n_tokens, int channels, int N, int groups);
cudaError_t launch_selective_scan(SelArgs a, int dtype, void *workspace, cudaStream_t st);
size_t sel_backward_workspace_bytes(int n_seqs, int n_tokens, int channels, int N, int groups);
cudaError_t launch_selective_scan_backward(SelArgs a, int dtype, void *workspace, cudaStream_t st);

}  // namespace ssm
