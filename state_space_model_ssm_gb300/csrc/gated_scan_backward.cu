// Backward kernel of the gated linear recurrence (sm_103a); the mathematics of
// the forward pass and the time chunks are in gated_common.cuh.
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
// thread's tokens gives P, H and E, a block needs the state entering its chunk
// (saved by the forward pass, fp32: h is recomputed in registers instead of
// read back rounded) and the E leaving the chunk after it, which it obtains as
// the forward kernel obtains its state, from the last chunk to the first.
#include "gated_common.cuh"

namespace ssm {

namespace {

template <class T, int V>
__global__ void __launch_bounds__(32 * kGatedWarps)
gated_scan_backward_kernel(const GatedArgs a)
{
    griddep_entry();
    constexpr int L = kGatedLen, W = kGatedWarps;
    __shared__ float tot_p[W][32 * V], tot_h[W][32 * V], tot_e[W][32 * V], arrive[32 * V];
    __shared__ int ticket;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0)
        ticket = atomicAdd(a.control + 1, 1);
    __syncthreads();
    const int back = ticket / a.cblocks, cb = ticket - back * a.cblocks;
    const int u = a.control[0] - 1 - back;                 // the last chunks first
    if (u < 0)
        return;
    const int2 unit = a.units[u];
    const int seq = unit.x, first = a.unit_base[seq], last = a.unit_base[seq + 1] - 1;
    long long t0;
    const int len = gated_seq_len(a, seq, t0);
    const int c0 = (cb * 32 + lane) * V;
    const bool inside = c0 < a.C;
    const int tw = unit.y * kGatedChunk + warp * L;
    const int cnt = min(L, len - tw);
    const long long at = (long long)u * a.C + c0;
    float rate[V], hin[V];
#pragma unroll
    for (int q = 0; q < V; ++q) {
        rate[q] = inside ? a.decay_scale * softplus_f(__ldg(a.lam + c0 + q)) : 0.f;
        hin[q] = inside ? __ldg(a.chunk_states + at + q) : 0.f;
    }
    Vec<T, V> x[L], ga[L], gx[L], dy[L];
#pragma unroll
    for (int k = 0; k < L; ++k)
        if (inside && k < cnt) {
            const long long t = t0 + tw + k;
            x[k] = load_vec<T, V>(static_cast<const T *>(a.x) + t * a.sx + c0);
            ga[k] = load_vec<T, V>(static_cast<const T *>(a.gate_a) + t * a.sga + c0);
            gx[k] = load_vec<T, V>(static_cast<const T *>(a.gate_x) + t * a.sgx + c0);
            dy[k] = load_vec<T, V>(static_cast<const T *>(a.grad_y) + t * a.sy + c0);
        }
    // decays a[k] and inputs b[k] of the run; its maps of h and of E
    float dec[L][V], hb[L][V];
#pragma unroll
    for (int q = 0; q < V; ++q) {
        float hh = 0.f, pp = 1.f, ee = 0.f;
#pragma unroll
        for (int k = 0; k < L; ++k) {
            dec[k][q] = 1.f;
            hb[k][q] = 0.f;
            if (inside && k < cnt) {
                const Decay d = decay_of(rate[q] * sigmoid_f(to_float(ga[k].v[q])));
                const float b = d.m * sigmoid_f(to_float(gx[k].v[q])) * to_float(x[k].v[q]);
                hh = fmaf(d.a, hh, b);
                pp *= d.a;
                ee = fmaf(pp, to_float(dy[k].v[q]), ee);
                dec[k][q] = d.a;
                hb[k][q] = b;
            }
        }
        tot_p[warp][lane * V + q] = pp;
        tot_h[warp][lane * V + q] = hh;
        tot_e[warp][lane * V + q] = ee;
    }
    __syncthreads();
    if (warp == 0) {
        float P[V], E[V], s[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            P[q] = 1.f;
            E[q] = 0.f;
#pragma unroll
            for (int w = W - 1; w >= 0; --w) {
                E[q] = fmaf(tot_p[w][lane * V + q], E[q], tot_e[w][lane * V + q]);
                P[q] *= tot_p[w][lane * V + q];
            }
            s[q] = 0.f;
        }
        int *flag = a.flags + (long long)u * a.cblocks + cb;
        if (u == last) {
            if (inside && a.grad_state)
#pragma unroll
                for (int q = 0; q < V; ++q)
                    s[q] = a.grad_state[(long long)seq * a.C + c0 + q];
        } else {
            if (inside)
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    __stcg(a.agg_p + at + q, P[q]);
                    __stcg(a.agg_h + at + q, E[q]);
                }
            __threadfence();
            __syncwarp();
            if (lane == 0)
                st_release(flag, 1);
            if (!gated_gather<V>(a, u, 1, last, cb, c0, lane, s)) {
                a.control[2] = 1;
#pragma unroll
                for (int q = 0; q < V; ++q)
                    s[q] = __int_as_float(0x7fc00000);
            }
        }
        if (u == first) {
            if (inside && a.grad_state0)
#pragma unroll
                for (int q = 0; q < V; ++q)
                    a.grad_state0[(long long)seq * a.C + c0 + q] =
                        a.resume[seq] != 0 ? fmaf(P[q], s[q], E[q]) : 0.f;
        } else {
            if (inside)
#pragma unroll
                for (int q = 0; q < V; ++q)
                    __stcg(a.out_state + at + q, fmaf(P[q], s[q], E[q]));
            __threadfence();
            __syncwarp();
            if (lane == 0)
                st_release(flag, 2);
        }
#pragma unroll
        for (int q = 0; q < V; ++q)
            arrive[lane * V + q] = s[q];
    }
    __syncthreads();
    float E[V], part[V];
#pragma unroll
    for (int q = 0; q < V; ++q) {
        float h = hin[q];
        for (int w = 0; w < warp; ++w)
            h = fmaf(tot_p[w][lane * V + q], h, tot_h[w][lane * V + q]);
#pragma unroll
        for (int k = 0; k < L; ++k) {                      // hb[k]: b_k -> h_{k-1}
            const float before = h;
            h = fmaf(dec[k][q], h, hb[k][q]);
            hb[k][q] = before;
        }
        E[q] = arrive[lane * V + q];
        for (int w = W - 1; w > warp; --w)
            E[q] = fmaf(tot_p[w][lane * V + q], E[q], tot_e[w][lane * V + q]);
        part[q] = 0.f;
    }
#pragma unroll
    for (int k = L - 1; k >= 0; --k)
        if (inside && k < cnt) {
            Vec<T, V> ox, oa, og;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float g = to_float(dy[k].v[q]) + E[q];
                const float e = dec[k][q];
                E[q] = e * g;
                const float r = sigmoid_f(to_float(ga[k].v[q])), i = sigmoid_f(to_float(gx[k].v[q]));
                const float v = rate[q] * r;
                const Decay d = decay_of(v);
                const float ix = i * to_float(x[k].v[q]);
                const float dla = g * (e * hb[k][q] - e * e * d.im * ix);
                part[q] = fmaf(dla, r, part[q]);
                ox.v[q] = from_float<T>(g * d.m * i);
                og.v[q] = from_float<T>(g * d.m * ix * (1.f - i));
                oa.v[q] = from_float<T>(-dla * v * (1.f - r));
            }
            const long long t = t0 + tw + k;
            store_vec<T, V>(static_cast<T *>(a.grad_x) + t * a.gsx + c0, ox);
            store_vec<T, V>(static_cast<T *>(a.grad_ga) + t * a.gsga + c0, oa);
            store_vec<T, V>(static_cast<T *>(a.grad_gx) + t * a.gsgx + c0, og);
        }
    __syncthreads();                                       // tot_p is read no more
#pragma unroll
    for (int q = 0; q < V; ++q)
        tot_p[warp][lane * V + q] = part[q];
    __syncthreads();
    if (warp == 0 && inside)
#pragma unroll
        for (int q = 0; q < V; ++q) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w)
                s += tot_p[w][lane * V + q];
            a.lam_part[at + q] = s;
        }
}

// dlam from the units' sums, in a fixed order: a block of 8 warps owns 32
// channels, warp w adds units w, w + 8, ...
__global__ void __launch_bounds__(256)
gated_lam_kernel(const GatedArgs a)
{
    griddep_entry();
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const int units = a.control[0];
    float s = 0.f;
    if (c < a.C)
        for (int u = warp; u < units; u += 8)
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

template <class T, int V>
cudaError_t launch_backward(const GatedArgs &a, cudaStream_t stream)
{
    cudaError_t e = launch_gated_plan(a, stream);
    if (e == cudaSuccess)
        e = launch_pdl(gated_scan_backward_kernel<T, V>, dim3((unsigned)((long long)a.max_units * a.cblocks)),
                       dim3(32 * kGatedWarps), 0, stream, a);
    if (e == cudaSuccess)
        e = launch_pdl(gated_lam_kernel, dim3((unsigned)((a.C + 31) / 32)), dim3(256), 0, stream, a);
    return e;
}

}  // namespace

cudaError_t launch_gated_scan_backward(GatedArgs a, int dtype, void *workspace, cudaStream_t stream)
{
    const bool pairs = gated_pairs(a, dtype, true);
    a.max_units = (int)gated_max_units(a.n_seqs, a.n_tokens);
    a.cblocks = (a.C + (pairs ? 63 : 31)) / (pairs ? 64 : 32);
    gated_carve(a, workspace);
    a.lam_part = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                           gated_workspace_bytes(a.n_seqs, a.n_tokens, a.C));
    switch (dtype) {
    case kF32: return pairs ? launch_backward<float, 2>(a, stream) : launch_backward<float, 1>(a, stream);
    case kBF16: return pairs ? launch_backward<__nv_bfloat16, 2>(a, stream) : launch_backward<__nv_bfloat16, 1>(a, stream);
    case kF16: return pairs ? launch_backward<__half, 2>(a, stream) : launch_backward<__half, 1>(a, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssm
