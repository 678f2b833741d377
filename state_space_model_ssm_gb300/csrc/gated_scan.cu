// Forward kernels of the gated linear recurrence (sm_103a); the mathematics and
// the passing of state between time chunks are in gated_common.cuh.
#include "gated_common.cuh"

namespace ssm {

namespace {

// ---- one token a sequence (decode), or any lengths token by token ----
// A thread owns V channels of one sequence and steps through its tokens.
template <class T, int V>
__global__ void __launch_bounds__(128)
gated_step_kernel(const GatedArgs a)
{
    griddep_entry();
    const int c0 = (blockIdx.x * blockDim.x + threadIdx.x) * V;
    if (c0 >= a.C)
        return;
    float rate[V];
#pragma unroll
    for (int q = 0; q < V; ++q)
        rate[q] = a.decay_scale * softplus_f(__ldg(a.lam + c0 + q));
    for (int seq = blockIdx.y; seq < a.n_seqs; seq += gridDim.y) {
        long long t0;
        const int len = gated_seq_len(a, seq, t0);
        float *slot = a.state + (long long)seq * a.C + c0;
        float h[V];
        const bool resume = a.resume[seq] != 0;
#pragma unroll
        for (int q = 0; q < V; ++q)
            h[q] = resume ? slot[q] : 0.f;
        for (int t = 0; t < len; ++t) {
            const Vec<T, V> x = load_vec<T, V>(static_cast<const T *>(a.x) + (t0 + t) * a.sx + c0);
            const Vec<T, V> ga = load_vec<T, V>(static_cast<const T *>(a.gate_a) + (t0 + t) * a.sga + c0);
            const Vec<T, V> gx = load_vec<T, V>(static_cast<const T *>(a.gate_x) + (t0 + t) * a.sgx + c0);
            Vec<T, V> y;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const Decay d = decay_of(rate[q] * sigmoid_f(to_float(ga.v[q])));
                h[q] = fmaf(d.a, h[q], d.m * sigmoid_f(to_float(gx.v[q])) * to_float(x.v[q]));
                y.v[q] = from_float<T>(h[q]);
            }
            store_vec<T, V>(static_cast<T *>(a.y) + (t0 + t) * a.sy + c0, y);
        }
#pragma unroll
        for (int q = 0; q < V; ++q)
            slot[q] = h[q];
    }
}

// ---- plan: the units of the batch, cleared flags ----
// Block 0 lists the (sequence, chunk) units; the others clear the flags.
__global__ void __launch_bounds__(1024)
gated_plan_kernel(const GatedArgs a)
{
    griddep_entry();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    if (blockIdx.x > 0) {
        const long long n = (long long)a.max_units * a.cblocks;
        for (long long i = (long long)(blockIdx.x - 1) * blockDim.x + tid; i < n; i += (long long)(gridDim.x - 1) * blockDim.x)
            a.flags[i] = 0;
        return;
    }
    __shared__ int warp_tot[32];
    __shared__ int carry;
    if (tid == 0)
        carry = 0;
    __syncthreads();
    for (int base = 0; base < a.n_seqs; base += blockDim.x) {
        const int i = base + tid;
        int cnt = 0;
        if (i < a.n_seqs) {
            long long t0;
            cnt = max(1, (gated_seq_len(a, i, t0) + kGatedChunk - 1) / kGatedChunk);   // an empty sequence keeps its slot's rule
        }
        int incl = cnt;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(kFullMask, incl, off);
            if (lane >= off)
                incl += v;
        }
        if (lane == 31)
            warp_tot[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            int wt = lane < nw ? warp_tot[lane] : 0;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_up_sync(kFullMask, wt, off);
                if (lane >= off)
                    wt += v;
            }
            if (lane < nw)
                warp_tot[lane] = wt;
        }
        __syncthreads();
        const int first = carry + (warp ? warp_tot[warp - 1] : 0) + incl - cnt;
        const int total = warp_tot[nw - 1];
        if (i < a.n_seqs)
            a.unit_base[i] = min(first, a.max_units);
        // the units of this round's sequences, a warp's 32 sequences one after another, its lanes over the chunks
        for (int k = 0; k < 32; ++k) {
            const int f = __shfl_sync(kFullMask, first, k), n = __shfl_sync(kFullMask, cnt, k);
            for (int j = lane; j < n; j += 32)
                if (f + j < a.max_units)
                    a.units[f + j] = make_int2(base + warp * 32 + k, j);
        }
        __syncthreads();
        if (tid == 0)
            carry += total;
        __syncthreads();
    }
    if (tid == 0) {
        a.unit_base[a.n_seqs] = min(carry, a.max_units);
        a.control[0] = min(carry, a.max_units);
        a.control[1] = 0;
        a.control[2] = 0;
    }
}

// ---- chunked kernel ----
// Block: kGatedWarps warps; warp w holds tokens w L .. w L + L - 1 of the chunk
// for the block's 32 V channels (lane: V channels).
template <class T, int V>
__global__ void __launch_bounds__(32 * kGatedWarps)
gated_scan_kernel(const GatedArgs a)
{
    griddep_entry();
    constexpr int L = kGatedLen, W = kGatedWarps;
    __shared__ float tot_p[W][32 * V], tot_h[W][32 * V], enter[32 * V];
    __shared__ int ticket;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0)
        ticket = atomicAdd(a.control + 1, 1);
    __syncthreads();
    const int u = ticket / a.cblocks, cb = ticket - u * a.cblocks;
    if (u >= a.control[0])
        return;
    const int2 unit = a.units[u];
    const int seq = unit.x, first = a.unit_base[seq];
    long long t0;
    const int len = gated_seq_len(a, seq, t0);
    const int c0 = (cb * 32 + lane) * V;
    const bool inside = c0 < a.C;
    const int tw = unit.y * kGatedChunk + warp * L;        // this warp's first token of the sequence
    const int cnt = min(L, len - tw);                      // its tokens (may be <= 0)
    float rate[V];
#pragma unroll
    for (int q = 0; q < V; ++q)
        rate[q] = inside ? a.decay_scale * softplus_f(__ldg(a.lam + c0 + q)) : 0.f;

    // every load first
    Vec<T, V> x[L], ga[L], gx[L];
#pragma unroll
    for (int k = 0; k < L; ++k)
        if (inside && k < cnt) {
            const long long t = t0 + tw + k;
            x[k] = load_vec<T, V>(static_cast<const T *>(a.x) + t * a.sx + c0);
            ga[k] = load_vec<T, V>(static_cast<const T *>(a.gate_a) + t * a.sga + c0);
            gx[k] = load_vec<T, V>(static_cast<const T *>(a.gate_x) + t * a.sgx + c0);
        }
    // the run from zero: h[k] and the product of decays p[k] up to token k
    float h[L][V], p[L][V];
#pragma unroll
    for (int q = 0; q < V; ++q) {
        float hh = 0.f, pp = 1.f;
#pragma unroll
        for (int k = 0; k < L; ++k) {
            if (inside && k < cnt) {
                const Decay d = decay_of(rate[q] * sigmoid_f(to_float(ga[k].v[q])));
                hh = fmaf(d.a, hh, d.m * sigmoid_f(to_float(gx[k].v[q])) * to_float(x[k].v[q]));
                pp *= d.a;
            }
            h[k][q] = hh;
            p[k][q] = pp;
        }
        tot_p[warp][lane * V + q] = pp;
        tot_h[warp][lane * V + q] = hh;
    }
    __syncthreads();
    if (warp == 0) {
        float P[V], H[V], s[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            P[q] = 1.f;
            H[q] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                H[q] = fmaf(tot_p[w][lane * V + q], H[q], tot_h[w][lane * V + q]);
                P[q] *= tot_p[w][lane * V + q];
            }
            s[q] = 0.f;
        }
        const long long at = (long long)u * a.C + c0;
        int *flag = a.flags + (long long)u * a.cblocks + cb;
        bool ok = true;
        if (u == first) {
            if (inside && a.resume[seq] != 0)
#pragma unroll
                for (int q = 0; q < V; ++q)
                    s[q] = a.state[(long long)seq * a.C + c0 + q];
        } else {
            if (inside)
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    __stcg(a.agg_p + at + q, P[q]);
                    __stcg(a.agg_h + at + q, H[q]);
                }
            __threadfence();
            __syncwarp();
            if (lane == 0)
                st_release(flag, 1);
            ok = gated_gather<V>(a, u, -1, first, cb, c0, lane, s);
            if (!ok) {
                a.control[2] = 1;
#pragma unroll
                for (int q = 0; q < V; ++q)
                    s[q] = __int_as_float(0x7fc00000);
            }
        }
        const bool last = u + 1 == a.unit_base[seq + 1];
        if (inside)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float o = fmaf(P[q], s[q], H[q]);
                if (last)
                    a.state[(long long)seq * a.C + c0 + q] = o;
                else
                    __stcg(a.out_state + at + q, o);
                if (a.chunk_states)
                    a.chunk_states[at + q] = s[q];
            }
        if (!last) {
            __threadfence();
            __syncwarp();
            if (lane == 0)
                st_release(flag, 2);
        }
#pragma unroll
        for (int q = 0; q < V; ++q)
            enter[lane * V + q] = s[q];
    }
    __syncthreads();
    float s[V];
#pragma unroll
    for (int q = 0; q < V; ++q) {
        s[q] = enter[lane * V + q];
        for (int w = 0; w < warp; ++w)
            s[q] = fmaf(tot_p[w][lane * V + q], s[q], tot_h[w][lane * V + q]);
    }
#pragma unroll
    for (int k = 0; k < L; ++k)
        if (inside && k < cnt) {
            Vec<T, V> y;
#pragma unroll
            for (int q = 0; q < V; ++q)
                y.v[q] = from_float<T>(fmaf(p[k][q], s[q], h[k][q]));
            store_vec<T, V>(static_cast<T *>(a.y) + (t0 + tw + k) * a.sy + c0, y);
        }
}

template <class T, int V>
cudaError_t launch_forward(const GatedArgs &a, cudaStream_t stream)
{
    if (a.n_tokens == a.n_seqs && !a.chunk_states) {
        const dim3 grid((unsigned)((a.C + 128 * V - 1) / (128 * V)), (unsigned)(a.n_seqs < 65535 ? a.n_seqs : 65535));
        return launch_pdl(gated_step_kernel<T, V>, grid, dim3(128), 0, stream, a);
    }
    cudaError_t e = launch_gated_plan(a, stream);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(gated_scan_kernel<T, V>, dim3((unsigned)((long long)a.max_units * a.cblocks)),
                      dim3(32 * kGatedWarps), 0, stream, a);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

long long gated_max_units(long long n_seqs, long long n_tokens) { return n_seqs + n_tokens / kGatedChunk; }

// Workspace: control, unit table, flags (for blocks of 32 channels), and three
// fp32 rows of C a unit.
size_t gated_workspace_bytes(int n_seqs, int n_tokens, int C)
{
    const size_t u = (size_t)gated_max_units(n_seqs, n_tokens), cb = ((size_t)C + 31) / 32;
    return 256 + up256(u * sizeof(int2)) + up256(((size_t)n_seqs + 1) * 4) + up256(u * cb * 4) +
           3 * up256(u * (size_t)C * 4);
}

void gated_carve(GatedArgs &a, void *workspace)
{
    const size_t u = (size_t)a.max_units, cb = ((size_t)a.C + 31) / 32;
    char *w = static_cast<char *>(workspace);
    auto take = [&](size_t bytes) {
        char *p = w;
        w += up256(bytes);
        return p;
    };
    a.control = reinterpret_cast<int *>(take(256));
    a.units = reinterpret_cast<int2 *>(take(u * sizeof(int2)));
    a.unit_base = reinterpret_cast<int *>(take(((size_t)a.n_seqs + 1) * 4));
    a.flags = reinterpret_cast<int *>(take(u * cb * 4));
    a.agg_p = reinterpret_cast<float *>(take(u * (size_t)a.C * 4));
    a.agg_h = reinterpret_cast<float *>(take(u * (size_t)a.C * 4));
    a.out_state = reinterpret_cast<float *>(take(u * (size_t)a.C * 4));
    a.lam_part = nullptr;
}

bool gated_pairs(const GatedArgs &a, int dtype, bool backward)
{
    const uintptr_t pair = 2 * dtype_size(dtype);
    long long odd = a.C | a.sx | a.sga | a.sgx | a.sy;
    uintptr_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.gate_a) |
                  reinterpret_cast<uintptr_t>(a.gate_x) | reinterpret_cast<uintptr_t>(backward ? a.grad_y : a.y);
    if (backward) {
        odd |= a.gsx | a.gsga | a.gsgx;
        p |= reinterpret_cast<uintptr_t>(a.grad_x) | reinterpret_cast<uintptr_t>(a.grad_ga) |
             reinterpret_cast<uintptr_t>(a.grad_gx);
    }
    return (odd & 1) == 0 && p % pair == 0;
}

cudaError_t launch_gated_plan(const GatedArgs &a, cudaStream_t stream)
{
    const long long words = (long long)a.max_units * a.cblocks;
    const long long extra = (words + 8 * 1024 - 1) / (8 * 1024);
    return launch_pdl(gated_plan_kernel, dim3(1 + (unsigned)(extra < 128 ? extra : 128)), dim3(1024), 0, stream, a);
}

cudaError_t launch_gated_scan(GatedArgs a, int dtype, void *workspace, cudaStream_t stream)
{
    const bool pairs = gated_pairs(a, dtype, false);
    a.max_units = (int)gated_max_units(a.n_seqs, a.n_tokens);
    a.cblocks = (a.C + (pairs ? 63 : 31)) / (pairs ? 64 : 32);
    gated_carve(a, workspace);
    switch (dtype) {
    case kF32: return pairs ? launch_forward<float, 2>(a, stream) : launch_forward<float, 1>(a, stream);
    case kBF16: return pairs ? launch_forward<__nv_bfloat16, 2>(a, stream) : launch_forward<__nv_bfloat16, 1>(a, stream);
    case kF16: return pairs ? launch_forward<__half, 2>(a, stream) : launch_forward<__half, 1>(a, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssm
