// Short causal convolution (depthwise, kernel 1..8) with SiLU on 16- or 32-bit rows with
// strides, forward and backward (sm_103a).  For a sequence, s is the stream of its slot's
// K - 1 inputs (zeros when fresh) followed by its tokens:
//
//   v[t,c] = bias[c] + sum_u w[c,u] s[t+u],   out = v sigmoid(v), or v;   slot <- the last K - 1 of s
//
// and with gv = grad_out times the derivative at v:
//
//   grad s[j,c] = sum_u w[c,u] gv[j-u,c]  (+ the slot's gradient for the last K - 1),
//   grad w[c,u] = sum_t gv[t,c] s[t+u,c],   grad bias = sum_t gv
//
// Bytes bound both, if the arithmetic is packed: a thread owns two channels (neighbours where
// rows allow 4-byte words of 16-bit types, 8-byte words of fp32; else two 128 apart, so that single
// elements are still read side by side) over a span of a sequence's tokens, keeps the window of
// inputs (and, backward, K unfinished sums of grad s) in registers as packed pairs, and loads
// the next run of eight tokens while it works on one.  A row is read once but for K - 1 rows of halo a
// span.  Backward recomputes v from the window.  Only the first span of a sequence reads its
// slot, so it writes it too.  The sums over tokens of grad w and grad bias leave as one row a
// span and are added in a second kernel in a fixed order.
#include <type_traits>

#include "packed.cuh"

namespace ssm {

namespace {

constexpr int kThreads = 128;
constexpr int kRun = 8;                       // tokens whose loads are issued together
constexpr int kPair = 2;                      // channels of a thread

struct ConvArgs {
    const void *x;
    const float *w, *bias;
    float *state;                             // forward: slots, in/out
    void *out;
    const int32_t *starts, *lens, *resume;
    int n_seqs, n_tokens, C, silu, span, units, cblocks;
    long long sx, so;
    // backward
    const void *grad_out;
    const float *state0, *grad_state;         // slots before the call, gradient of those after it
    void *grad_x;
    float *grad_w, *grad_bias, *grad_state0, *part;      // part [units][K + 1][C]
    long long sgo, sgx;
};

__device__ __forceinline__ int seq_len(const ConvArgs &a, int seq, long long &t0)
{
    t0 = a.starts[seq];
    const long long len = a.lens[seq];
    if (t0 >= 0 && len > 0 && t0 + len <= a.n_tokens)
        return (int)len;
    t0 = 0;
    return 0;
}

// The u-th span of all sequences (each has one at least): its sequence and place in it; false past
// the last.  Every warp finds it by itself.
__device__ __forceinline__ bool find_span(const ConvArgs &a, int u, int &seq, int &k)
{
    k = 0;
    seq = u;
    if (a.units == a.n_seqs)                                // no sequence is longer than a span
        return u < a.n_seqs;
    const int lane = threadIdx.x & 31;
    constexpr int kEach = 4;                                // groups of 32 sequences whose lengths are loaded together
    int base = 0;
    for (int s0 = 0; s0 < a.n_seqs; s0 += 32 * kEach) {
        int spans[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int s = s0 + 32 * j + lane;
            long long t0;
            spans[j] = s < a.n_seqs ? max(1, (seq_len(a, s, t0) + a.span - 1) / a.span) : 0;
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int all = __reduce_add_sync(kFullMask, spans[j]);
            if (u >= base + all) {
                base += all;
                continue;
            }
            int incl = spans[j];
#pragma unroll
            for (int off = 1; off < 32; off *= 2) {
                const int v = __shfl_up_sync(kFullMask, incl, off);
                if (lane >= off)
                    incl += v;
            }
            const int l = __ffs(__ballot_sync(kFullMask, u < base + incl)) - 1;
            seq = s0 + 32 * j + l;
            k = u - base - __shfl_sync(kFullMask, incl - spans[j], l);
            return true;
        }
    }
    return false;
}

// A thread's two channels: neighbours, or kThreads apart.
template <bool PAIRS>
struct Channels {
    int c;                                                  // the first
    bool first, second;                                     // whether they exist
    __device__ __forceinline__ Channels(int cblock, int C)
    {
        c = cblock * kPair * kThreads + (PAIRS ? kPair : 1) * threadIdx.x;
        first = c < C;
        second = c + step() < C;
    }
    static __device__ __forceinline__ constexpr int step() { return PAIRS ? 1 : kThreads; }
    __device__ __forceinline__ float2 read(const float *p, long long each) const      // p[c * each], zeros where there is none
    {
        return make_float2(first ? p[c * each] : 0.f, second ? p[(c + step()) * each] : 0.f);
    }
    __device__ __forceinline__ void write(float *p, long long each, float2 v) const
    {
        if (first) p[c * each] = v.x;
        if (second) p[(c + step()) * each] = v.y;
    }
    // of a row of T: loads stay inside the row (a channel that is not there reads the first)
    template <class T>
    __device__ __forceinline__ RawPair<T> load(const T *row) const
    {
        if constexpr (PAIRS)
            return load_pair(row + c);
        else
            return join_pair<T>(row[c], row[second ? c + kThreads : c]);
    }
    template <class T>
    __device__ __forceinline__ void store(T *row, float2 v) const
    {
        if constexpr (PAIRS) {
            store_word(row + c, v);
        } else {
            row[c] = from_float<T>(v.x);
            if (second)
                row[c + kThreads] = from_float<T>(v.y);
        }
    }
};

// The window in front of token `begin`: slot entries (zeros for a fresh sequence, whose slot is not read)
// or, in later spans, tokens (a span is longer than the window).
template <class T, int K, class Ch>
__device__ __forceinline__ void first_window(float2 (&win)[K > 1 ? K - 1 : 1], const float *slots, const T *x, const ConvArgs &a,
                                             const Ch &ch, int seq, int begin)
{
#pragma unroll
    for (int u = 0; u < K - 1; ++u)
        win[u] = make_float2(0.f, 0.f);
    if (K == 1)
        return;
    if (begin > 0) {
#pragma unroll
        for (int u = 0; u < K - 1; ++u)
            win[u] = pair_of<T>(ch.load(x + (long long)(begin - (K - 1) + u) * a.sx));
    } else if (slots && a.resume[seq] != 0) {
#pragma unroll
        for (int u = 0; u < K - 1; ++u)
            win[u] = ch.read(slots + (long long)seq * a.C * (K - 1) + u, K - 1);
    }
}

// v of a token, and the window moved on to it.
template <int K>
__device__ __forceinline__ float2 taps(const float2 (&w)[K], float2 bias, float2 (&win)[K > 1 ? K - 1 : 1], float2 now)
{
    float2 v = fma2(w[K - 1], now, bias);
#pragma unroll
    for (int u = 0; u < K - 1; ++u)
        v = fma2(w[u], win[u], v);
#pragma unroll
    for (int u = 0; u + 1 < K - 1; ++u)
        win[u] = win[u + 1];
    if (K > 1)
        win[K > 1 ? K - 2 : 0] = now;
    return v;
}

template <class T, bool PAIRS, int K>
__global__ void __launch_bounds__(kThreads)
causal_conv_kernel(const ConvArgs a)
{
    griddep_entry();
    const int unit = blockIdx.x / a.cblocks;
    const Channels<PAIRS> ch(blockIdx.x - unit * a.cblocks, a.C);
    int seq, k;
    if (!find_span(a, unit, seq, k) || !ch.first)
        return;
    long long t0;
    const int len = seq_len(a, seq, t0), begin = k * a.span, end = min(len, begin + a.span);
    float2 w[K], win[K > 1 ? K - 1 : 1];
#pragma unroll
    for (int u = 0; u < K; ++u)
        w[u] = ch.read(a.w + u, K);
    const float2 bias = a.bias ? ch.read(a.bias, 1) : make_float2(0.f, 0.f);
    const T *x = static_cast<const T *>(a.x) + t0 * a.sx;
    T *out = static_cast<T *>(a.out) + t0 * a.so;
    RawPair<T> next[kRun];
    auto fetch = [&](int b) {
#pragma unroll
        for (int r = 0; r < kRun; ++r)
            next[r] = ch.load(x + (long long)min(b + r, end - 1) * a.sx);
    };
    if (begin < end)
        fetch(begin);
    first_window<T, K>(win, a.state, x, a, ch, seq, begin);
    if (K > 1 && k == 0) {                                  // the stream's last K - 1: of the tokens, or still of the slot
        float *slot = a.state + (long long)seq * a.C * (K - 1);
#pragma unroll
        for (int u = 0; u < K - 1; ++u) {
            const int t = len - (K - 1) + u;                // token, or slot entry t + K - 1
            float2 v = make_float2(0.f, 0.f);
            if (t >= 0)
                v = pair_of<T>(ch.load(x + t * a.sx));
            else
#pragma unroll
                for (int e = 0; e < K - 1; ++e)
                    v = e == t + K - 1 ? win[e] : v;
            ch.write(slot + u, K - 1, v);
        }
    }
    auto run = [&](int b, auto whole) {                     // whole: every token of the run is in the span
        RawPair<T> in[kRun];
#pragma unroll
        for (int r = 0; r < kRun; ++r)
            in[r] = next[r];
        if (b + kRun < end)
            fetch(b + kRun);
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            const float2 v = taps<K>(w, bias, win, pair_of<T>(in[r]));
            if (decltype(whole)::value || b + r < end)
                ch.store(out + (long long)(b + r) * a.so, a.silu ? mul2(v, sigmoid2(v)) : v);
        }
    };
    int b = begin;
    for (; b + kRun <= end; b += kRun)
        run(b, std::true_type());
    if (b < end)
        run(b, std::false_type());
}

template <class T, bool PAIRS, int K>
__global__ void __launch_bounds__(kThreads)
causal_conv_backward_kernel(const ConvArgs a)
{
    griddep_entry();
    const int unit = blockIdx.x / a.cblocks;
    const Channels<PAIRS> ch(blockIdx.x - unit * a.cblocks, a.C);
    int seq, k;
    if (!find_span(a, unit, seq, k) || !ch.first)
        return;
    long long t0;
    const int len = seq_len(a, seq, t0), begin = k * a.span, end = min(len, begin + a.span);
    const float2 zero = make_float2(0.f, 0.f);
    float2 w[K], gw[K], gb = zero, win[K > 1 ? K - 1 : 1];
    float2 sum[K];                                          // unfinished gradients of stream entries t .. t + K - 1
#pragma unroll
    for (int u = 0; u < K; ++u) {
        w[u] = ch.read(a.w + u, K);
        gw[u] = sum[u] = zero;
    }
    const float2 bias = a.bias ? ch.read(a.bias, 1) : zero;
    const T *x = static_cast<const T *>(a.x) + t0 * a.sx, *go = static_cast<const T *>(a.grad_out) + t0 * a.sgo;
    T *gx = static_cast<T *>(a.grad_x) + t0 * a.sgx;
    const long long slot = (long long)seq * a.C * (K - 1);
    const bool resumed = K > 1 && a.grad_state0 && a.resume[seq] != 0;
    const int stop = end + K - 1;                           // the last entries need the tokens behind the span
    RawPair<T> next_x[kRun], next_g[kRun];
    auto fetch = [&](int b) {
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            const long long t = min(b + r, min(stop, len) - 1);
            next_x[r] = ch.load(x + t * a.sx);
            next_g[r] = ch.load(go + t * a.sgo);
        }
    };
    if (begin < end)
        fetch(begin);
    first_window<T, K>(win, a.state0, x, a, ch, seq, begin);
    // whole: every token of the run is in the span, and behind its first K - 1
    auto run = [&](int b, auto whole) {
        constexpr bool W = decltype(whole)::value;
        RawPair<T> in[kRun], g[kRun];
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            in[r] = next_x[r];
            g[r] = next_g[r];
        }
        if (b + kRun < stop && b + kRun < len)
            fetch(b + kRun);
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            const int t = b + r;
            if (W || (t < stop && t < len)) {
                const float2 now = pair_of<T>(in[r]);
                float2 before[K > 1 ? K - 1 : 1], gv = pair_of<T>(g[r]);
#pragma unroll
                for (int u = 0; u < K - 1; ++u)
                    before[u] = win[u];
                const float2 v = taps<K>(w, bias, win, now);
                if (a.silu) {
                    const float2 s = sigmoid2(v);
                    gv = mul2(gv, fma2(mul2(v, s), make_float2(1.f - s.x, 1.f - s.y), s));
                }
                if (W || t < end) {
                    gb = add2(gb, gv);
#pragma unroll
                    for (int u = 0; u < K - 1; ++u)
                        gw[u] = fma2(gv, before[u], gw[u]);
                    gw[K - 1] = fma2(gv, now, gw[K - 1]);
                }
#pragma unroll
                for (int u = 0; u < K; ++u)
                    sum[u] = fma2(w[u], gv, sum[u]);
            }
            // stream entry t is complete: token t - (K - 1), or entry t of the slot
            if (W) {
                ch.store(gx + (long long)(t - (K - 1)) * a.sgx, sum[0]);
            } else if (t < stop && (t >= begin + K - 1 || k == 0)) {
                float2 done = sum[0];
                if (K > 1 && t >= len && a.grad_state)
                    done = add2(done, ch.read(a.grad_state + slot + t - len, K - 1));
                if (t >= K - 1)
                    ch.store(gx + (long long)(t - (K - 1)) * a.sgx, done);
                else if (a.grad_state0)
                    ch.write(a.grad_state0 + slot + t, K - 1, resumed ? done : zero);
            }
#pragma unroll
            for (int u = 0; u + 1 < K; ++u)
                sum[u] = sum[u + 1];
            sum[K - 1] = zero;
        }
    };
    static_assert(kRun >= K - 1, "the run behind the first is behind the window");
    for (int b = begin; b < stop; b += kRun) {
        if (b > begin && b + kRun <= end)
            run(b, std::true_type());
        else
            run(b, std::false_type());
    }
    float *part = a.part + (long long)unit * (K + 1) * a.C;
#pragma unroll
    for (int u = 0; u < K; ++u)
        ch.write(part + (long long)u * a.C, 1, gw[u]);
    ch.write(part + (long long)K * a.C, 1, gb);
}

// grad w and grad bias: 32 channels of one tap a block, the spans over 8 lanes of threads.
__global__ void __launch_bounds__(256)
causal_conv_sum_kernel(const ConvArgs a, int K)
{
    griddep_entry();
    __shared__ float sums[8][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), u = blockIdx.y, lane = threadIdx.x >> 5;
    // spans that exist: find_span gives the sequence of the last one
    int units = a.n_seqs;
    if (a.units != a.n_seqs) {
        int n = 0;
        for (int s = threadIdx.x & 31; s < a.n_seqs; s += 32) {
            long long t0;
            n += max(1, (seq_len(a, s, t0) + a.span - 1) / a.span);
        }
#pragma unroll
        for (int off = 16; off >= 1; off /= 2)
            n += __shfl_xor_sync(kFullMask, n, off);
        units = min(n, a.units);
    }
    float v = 0.f;
    if (c < a.C)
        for (int i = lane; i < units; i += 8)
            v += a.part[((long long)i * (K + 1) + u) * a.C + c];
    sums[lane][threadIdx.x & 31] = v;
    __syncthreads();
    if (lane == 0 && c < a.C) {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            v += sums[i][threadIdx.x];
        if (u < K)
            a.grad_w[(long long)c * K + u] = v;
        else if (a.grad_bias)
            a.grad_bias[c] = v;
    }
}

template <class T, bool PAIRS, int K>
cudaError_t launch_kernel(ConvArgs a, bool backward, cudaStream_t st)
{
    a.cblocks = (a.C + kPair * kThreads - 1) / (kPair * kThreads);
    const dim3 grid((unsigned)((long long)a.units * a.cblocks)), block(kThreads);
    if (!backward)
        return launch_pdl(causal_conv_kernel<T, PAIRS, K>, grid, block, 0, st, a);
    const cudaError_t e = launch_pdl(causal_conv_backward_kernel<T, PAIRS, K>, grid, block, 0, st, a);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(causal_conv_sum_kernel, dim3((a.C + 31) / 32, K + 1), dim3(256), 0, st, a, K);
}

template <class T, bool PAIRS>
cudaError_t launch_taps(const ConvArgs &a, int K, bool backward, cudaStream_t st)
{
    switch (K) {
    case 1: return launch_kernel<T, PAIRS, 1>(a, backward, st);
    case 2: return launch_kernel<T, PAIRS, 2>(a, backward, st);
    case 3: return launch_kernel<T, PAIRS, 3>(a, backward, st);
    case 4: return launch_kernel<T, PAIRS, 4>(a, backward, st);
    case 5: return launch_kernel<T, PAIRS, 5>(a, backward, st);
    case 6: return launch_kernel<T, PAIRS, 6>(a, backward, st);
    case 7: return launch_kernel<T, PAIRS, 7>(a, backward, st);
    case 8: return launch_kernel<T, PAIRS, 8>(a, backward, st);
    default: return cudaErrorInvalidValue;
    }
}

template <class T>
cudaError_t launch_type(const ConvArgs &a, int K, bool backward, cudaStream_t st)
{
    auto even = [&](const void *p, long long stride) {
        return (reinterpret_cast<uintptr_t>(p) % (2 * sizeof(T))) == 0 && stride % 2 == 0;
    };
    bool pairs = a.C % 2 == 0 && even(a.x, a.sx);
    pairs = pairs && (backward ? even(a.grad_out, a.sgo) && even(a.grad_x, a.sgx) : even(a.out, a.so));
    return pairs ? launch_taps<T, true>(a, K, backward, st) : launch_taps<T, false>(a, K, backward, st);
}

// Tokens of a span: about two rounds of resident threads, whole runs.
int span_of(int n_tokens, int channels)
{
    const long long each = (long long)n_tokens * ((channels + kPair - 1) / kPair) / (kSms * 1280);
    return (int)(each < 32 ? 32 : each > 512 ? 512 : (each + kRun - 1) / kRun * kRun);
}

int units_of(int n_seqs, int n_tokens, int span) { return n_tokens <= span ? n_seqs : n_seqs + n_tokens / span; }

}  // namespace

size_t causal_conv_backward_workspace_bytes(int n_seqs, int n_tokens, int channels, int K)
{
    return (size_t)units_of(n_seqs, n_tokens, span_of(n_tokens, channels)) * (K + 1) * channels * sizeof(float);
}

long long causal_conv_blocks(int n_seqs, int n_tokens, int channels)
{
    return (long long)units_of(n_seqs, n_tokens, span_of(n_tokens, channels)) * ((channels + kPair * kThreads - 1LL) / (kPair * kThreads));
}

cudaError_t launch_causal_conv(const CausalConv &c, bool backward, cudaStream_t st)
{
    ConvArgs a{};
    a.x = c.x; a.w = c.w; a.bias = c.bias; a.state = c.state; a.out = c.out;
    a.starts = c.starts; a.lens = c.lens; a.resume = c.resume;
    a.n_seqs = c.n_seqs; a.n_tokens = c.n_tokens; a.C = c.channels; a.silu = c.silu; a.sx = c.sx; a.so = c.so;
    a.grad_out = c.grad_out; a.state0 = c.state0; a.grad_state = c.grad_state; a.grad_x = c.grad_x;
    a.grad_w = c.grad_w; a.grad_bias = c.grad_bias; a.grad_state0 = c.grad_state0; a.part = c.part;
    a.sgo = c.sgo; a.sgx = c.sgx;
    a.span = span_of(c.n_tokens, c.channels);
    a.units = units_of(c.n_seqs, c.n_tokens, a.span);
    switch (c.dtype) {
    case kF32: return launch_type<float>(a, c.K, backward, st);
    case kBF16: return launch_type<__nv_bfloat16>(a, c.K, backward, st);
    case kF16: return launch_type<__half>(a, c.K, backward, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssm
