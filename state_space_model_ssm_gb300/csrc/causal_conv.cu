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
// Bytes bound both: a thread owns V neighbouring channels over a span of a sequence's tokens
// and keeps the window of inputs (and, backward, K unfinished sums of grad s) in registers, so
// a row is read once but for K - 1 rows of halo a span.  Backward recomputes v from the
// window.  Loads of a run of tokens are issued together.  Only the first span of a sequence
// reads its slot, so it writes it too.  The sums over tokens of grad w and grad bias leave as
// one row a span and are added in a second kernel in a fixed order.
#include "layer_common.cuh"

namespace ssm {

namespace {

constexpr int kThreads = 128;
constexpr int kRun = 8;                       // tokens whose loads are issued together

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

__device__ __forceinline__ float sigmoid_of(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

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
    int base = 0;
    for (int s0 = 0; s0 < a.n_seqs; s0 += 32) {
        long long t0;
        const int mine = s0 + lane < a.n_seqs ? max(1, (seq_len(a, s0 + lane, t0) + a.span - 1) / a.span) : 0;
        int incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
            const int v = __shfl_up_sync(kFullMask, incl, off);
            if (lane >= off)
                incl += v;
        }
        const unsigned m = __ballot_sync(kFullMask, u < base + incl);
        if (m) {
            const int l = __ffs(m) - 1;
            seq = s0 + l;
            k = u - base - __shfl_sync(kFullMask, incl - mine, l);
            return true;
        }
        base += __shfl_sync(kFullMask, incl, 31);
    }
    return false;
}

// V channels' K - 1 slot entries.
template <int V, int K>
__device__ __forceinline__ void read_slot(float (&s)[K > 1 ? K - 1 : 1][V], const float *p)
{
    if constexpr (K > 1) {
        float v[V * (K - 1)];
        if constexpr (V == 4) {
#pragma unroll
            for (int i = 0; i < K - 1; ++i) {
                const float4 q = reinterpret_cast<const float4 *>(p)[i];
                v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V * (K - 1); ++i)
                v[i] = p[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int u = 0; u < K - 1; ++u)
                s[u][i] = v[i * (K - 1) + u];
    }
}

template <int V, int K>
__device__ __forceinline__ void write_slot(float *p, const float (&s)[K > 1 ? K - 1 : 1][V])
{
    if constexpr (K > 1) {
        float v[V * (K - 1)];
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int u = 0; u < K - 1; ++u)
                v[i * (K - 1) + u] = s[u][i];
        if constexpr (V == 4) {
#pragma unroll
            for (int i = 0; i < K - 1; ++i)
                reinterpret_cast<float4 *>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < V * (K - 1); ++i)
                p[i] = v[i];
        }
    }
}

// The slot's entries as inputs: zeros for a fresh sequence (whose slot is not read).
template <int V, int K>
__device__ __forceinline__ void first_window(float (&win)[K > 1 ? K - 1 : 1][V], const float *slots, const ConvArgs &a,
                                             int seq, int c0)
{
#pragma unroll
    for (int u = 0; u < (K > 1 ? K - 1 : 1); ++u)
#pragma unroll
        for (int i = 0; i < V; ++i)
            win[u][i] = 0.f;
    if (K > 1 && slots && a.resume[seq] != 0)
        read_slot<V, K>(win, slots + ((long long)seq * a.C + c0) * (K - 1));
}

template <class T, int V, int K>
__global__ void __launch_bounds__(kThreads)
causal_conv_kernel(const ConvArgs a)
{
    griddep_entry();
    const int unit = blockIdx.x / a.cblocks, c0 = ((blockIdx.x - unit * a.cblocks) * kThreads + threadIdx.x) * V;
    int seq, k;
    if (!find_span(a, unit, seq, k) || c0 >= a.C)
        return;
    long long t0;
    const int len = seq_len(a, seq, t0), begin = k * a.span, end = min(len, begin + a.span);
    float w[K][V], bias[V], win[K > 1 ? K - 1 : 1][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int u = 0; u < K; ++u)
            w[u][i] = __ldg(a.w + (long long)(c0 + i) * K + u);
        bias[i] = a.bias ? __ldg(a.bias + c0 + i) : 0.f;
    }
    const T *x = static_cast<const T *>(a.x) + t0 * a.sx + c0;
    T *out = static_cast<T *>(a.out) + t0 * a.so + c0;
    if (k == 0) {
        first_window<V, K>(win, a.state, a, seq, c0);
        if constexpr (K > 1) {                              // the stream's last K - 1: of the tokens, or still of the slot
            float last[K - 1][V];
#pragma unroll
            for (int u = 0; u < K - 1; ++u) {
                const int t = len - (K - 1) + u;            // token, or slot entry t + K - 1
                if (t >= 0) {
                    const Vec<T, V> v = load_vec<T, V>(x + t * a.sx);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        last[u][i] = to_float(v.v[i]);
                } else {
#pragma unroll
                    for (int e = 0; e < K - 1; ++e)
                        if (e == t + K - 1)
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                last[u][i] = win[e][i];
                }
            }
            write_slot<V, K>(a.state + ((long long)seq * a.C + c0) * (K - 1), last);
        }
    } else {
#pragma unroll
        for (int u = 0; u < K - 1; ++u) {                   // (a span is longer than the window)
            const Vec<T, V> v = load_vec<T, V>(x + (long long)(begin - (K - 1) + u) * a.sx);
#pragma unroll
            for (int i = 0; i < V; ++i)
                win[u][i] = to_float(v.v[i]);
        }
    }
    for (int b = begin; b < end; b += kRun) {
        Vec<T, V> in[kRun];
#pragma unroll
        for (int r = 0; r < kRun; ++r)
            if (b + r < end)
                in[r] = load_vec<T, V>(x + (long long)(b + r) * a.sx);
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            if (b + r >= end)
                break;
            Vec<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float now = to_float(in[r].v[i]);
                float v = fmaf(w[K - 1][i], now, bias[i]);
#pragma unroll
                for (int u = 0; u < K - 1; ++u)
                    v = fmaf(w[u][i], win[u][i], v);
#pragma unroll
                for (int u = 0; u + 1 < K - 1; ++u)
                    win[u][i] = win[u + 1][i];
                if (K > 1)
                    win[K > 1 ? K - 2 : 0][i] = now;
                o.v[i] = from_float<T>(a.silu ? v * sigmoid_of(v) : v);
            }
            store_vec<T, V>(out + (long long)(b + r) * a.so, o);
        }
    }
}

template <class T, int V, int K>
__global__ void __launch_bounds__(kThreads)
causal_conv_backward_kernel(const ConvArgs a)
{
    griddep_entry();
    const int unit = blockIdx.x / a.cblocks, c0 = ((blockIdx.x - unit * a.cblocks) * kThreads + threadIdx.x) * V;
    int seq, k;
    if (!find_span(a, unit, seq, k) || c0 >= a.C)
        return;
    long long t0;
    const int len = seq_len(a, seq, t0), begin = k * a.span, end = min(len, begin + a.span);
    float w[K][V], bias[V], gw[K][V], gb[V], win[K > 1 ? K - 1 : 1][V];
    float sum[K][V];                                        // unfinished gradients of stream entries t .. t + K - 1
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int u = 0; u < K; ++u) {
            w[u][i] = __ldg(a.w + (long long)(c0 + i) * K + u);
            gw[u][i] = sum[u][i] = 0.f;
        }
        bias[i] = a.bias ? __ldg(a.bias + c0 + i) : 0.f;
        gb[i] = 0.f;
    }
    const T *x = static_cast<const T *>(a.x) + t0 * a.sx + c0, *go = static_cast<const T *>(a.grad_out) + t0 * a.sgo + c0;
    T *gx = static_cast<T *>(a.grad_x) + t0 * a.sgx + c0;
    if (k == 0) {
        first_window<V, K>(win, a.state0, a, seq, c0);
    } else {
#pragma unroll
        for (int u = 0; u < K - 1; ++u) {
            const Vec<T, V> v = load_vec<T, V>(x + (long long)(begin - (K - 1) + u) * a.sx);
#pragma unroll
            for (int i = 0; i < V; ++i)
                win[u][i] = to_float(v.v[i]);
        }
    }
    const long long slot = ((long long)seq * a.C + c0) * (K - 1);
    const bool resumed = a.grad_state0 && a.resume[seq] != 0;
    const int stop = end + K - 1;                           // the last entries need the tokens behind the span
    for (int b = begin; b < stop; b += kRun) {
        Vec<T, V> in[kRun], g[kRun];
#pragma unroll
        for (int r = 0; r < kRun; ++r)
            if (b + r < stop && b + r < len) {
                in[r] = load_vec<T, V>(x + (long long)(b + r) * a.sx);
                g[r] = load_vec<T, V>(go + (long long)(b + r) * a.sgo);
            }
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            const int t = b + r;
            if (t >= stop)
                break;
            if (t < len) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float now = to_float(in[r].v[i]);
                    float v = fmaf(w[K - 1][i], now, bias[i]), gv = to_float(g[r].v[i]);
#pragma unroll
                    for (int u = 0; u < K - 1; ++u)
                        v = fmaf(w[u][i], win[u][i], v);
                    if (a.silu) {
                        const float s = sigmoid_of(v);
                        gv *= fmaf(v * s, 1.f - s, s);
                    }
                    if (t < end) {
                        gb[i] += gv;
#pragma unroll
                        for (int u = 0; u < K - 1; ++u)
                            gw[u][i] = fmaf(gv, win[u][i], gw[u][i]);
                        gw[K - 1][i] = fmaf(gv, now, gw[K - 1][i]);
                    }
#pragma unroll
                    for (int u = 0; u < K; ++u)
                        sum[u][i] = fmaf(w[u][i], gv, sum[u][i]);
#pragma unroll
                    for (int u = 0; u + 1 < K - 1; ++u)
                        win[u][i] = win[u + 1][i];
                    if (K > 1)
                        win[K > 1 ? K - 2 : 0][i] = now;
                }
            }
            // stream entry t is complete: token t - (K - 1), or entry t of the slot
            if (t >= begin + K - 1 || k == 0) {
                float done[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    done[i] = sum[0][i];
                    if (K > 1 && t >= len && a.grad_state)
                        done[i] += a.grad_state[slot + i * (K - 1) + t - len];
                }
                if (t >= K - 1) {
                    Vec<T, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        o.v[i] = from_float<T>(done[i]);
                    store_vec<T, V>(gx + (long long)(t - (K - 1)) * a.sgx, o);
                } else if (a.grad_state0) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        a.grad_state0[slot + i * (K - 1) + t] = resumed ? done[i] : 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int u = 0; u + 1 < K; ++u)
                    sum[u][i] = sum[u + 1][i];
                sum[K - 1][i] = 0.f;
            }
        }
    }
    float *part = a.part + (long long)unit * (K + 1) * a.C + c0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int u = 0; u < K; ++u)
            part[(long long)u * a.C + i] = gw[u][i];
        part[(long long)K * a.C + i] = gb[i];
    }
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

template <class T, int V, int K>
cudaError_t launch_kernel(ConvArgs a, bool backward, cudaStream_t st)
{
    a.cblocks = (a.C + kThreads * V - 1) / (kThreads * V);
    const dim3 grid((unsigned)((long long)a.units * a.cblocks)), block(kThreads);
    if (!backward)
        return launch_pdl(causal_conv_kernel<T, V, K>, grid, block, 0, st, a);
    const cudaError_t e = launch_pdl(causal_conv_backward_kernel<T, V, K>, grid, block, 0, st, a);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(causal_conv_sum_kernel, dim3((a.C + 31) / 32, K + 1), dim3(256), 0, st, a, K);
}

template <class T, int V>
cudaError_t launch_taps(const ConvArgs &a, int K, bool backward, cudaStream_t st)
{
    switch (K) {
    case 1: return launch_kernel<T, V, 1>(a, backward, st);
    case 2: return launch_kernel<T, V, 2>(a, backward, st);
    case 3: return launch_kernel<T, V, 3>(a, backward, st);
    case 4: return launch_kernel<T, V, 4>(a, backward, st);
    case 5: return launch_kernel<T, V, 5>(a, backward, st);
    case 6: return launch_kernel<T, V, 6>(a, backward, st);
    case 7: return launch_kernel<T, V, 7>(a, backward, st);
    case 8: return launch_kernel<T, V, 8>(a, backward, st);
    default: return cudaErrorInvalidValue;
    }
}

template <class T>
cudaError_t launch_type(const ConvArgs &a, int K, bool backward, cudaStream_t st)
{
    // four channels a thread where every row and slot allows it
    const uintptr_t rows = sizeof(T) * 4;
    auto fits = [&](const void *p, long long stride) {
        return (reinterpret_cast<uintptr_t>(p) % rows) == 0 && stride * (long long)sizeof(T) % (long long)rows == 0;
    };
    bool wide = a.C % 4 == 0 && (reinterpret_cast<uintptr_t>(backward ? a.state0 : a.state) & 15) == 0 && fits(a.x, a.sx);
    wide = wide && (backward ? fits(a.grad_out, a.sgo) && fits(a.grad_x, a.sgx) : fits(a.out, a.so));
    return wide ? launch_taps<T, 4>(a, K, backward, st) : launch_taps<T, 1>(a, K, backward, st);
}

// Tokens of a span: threads of about one wave, whole runs.
int span_of(int n_tokens, int channels)
{
    const long long each = (long long)n_tokens * ((channels + 3) / 4) / (kSms * 1024);
    return (int)(each < 32 ? 32 : each > 256 ? 256 : (each + kRun - 1) / kRun * kRun);
}

int units_of(int n_seqs, int n_tokens, int span) { return n_tokens <= span ? n_seqs : n_seqs + n_tokens / span; }

}  // namespace

size_t causal_conv_backward_workspace_bytes(int n_seqs, int n_tokens, int channels, int K)
{
    return (size_t)units_of(n_seqs, n_tokens, span_of(n_tokens, channels)) * (K + 1) * channels * sizeof(float);
}

long long causal_conv_blocks(int n_seqs, int n_tokens, int channels)
{
    return (long long)units_of(n_seqs, n_tokens, span_of(n_tokens, channels)) * ((channels + kThreads - 1LL) / kThreads);
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
