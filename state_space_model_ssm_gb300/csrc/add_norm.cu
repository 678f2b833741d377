// RMS norm with the residual's addition, its 8-bit output, its gradient, and the
// row quantiser (sm_103a).  Per row of D elements:
//
//   h = x + residual, rounded to the residual's type (the residual stream as the
//       next layer reads it; the norm is of that value)
//   inv = 1 / sqrt(mean(h^2) + eps),  y = h inv w
//   8 bits: v = h w,  f = min(127 / max|v|, FLT_MAX),  code = rint(v f),  scale = inv / f
//
// so code * scale ~ h inv w.  The norm's inv is the same for the whole row and
// cancels out of the codes, so the sum of squares and the largest |v| come from
// one reduction and the row is read once; the codes depend on no order of
// summation (a product, a maximum, a quotient and a rounding, each exact or
// rounded once).  A row of zeros has f = FLT_MAX and codes 0; a row with a NaN or
// an infinity has scale NaN, so its values are NaN.  The quantiser is the same
// with v = x and inv = 1.
//
// Gradient, with n = h inv and s = mean(n w gy):
//   grad_in = grad_h + inv (w gy - n s),  grad_w = sum over rows of gy n
#include <cfloat>

#include "layer_common.cuh"

namespace ssm {

namespace {

constexpr int kNormThreads = 512;         // most threads of a block
constexpr int kNormOut = 0, kNormCodes = 1, kCodesOnly = 2;

struct NormArgs {
    const void *x, *residual;
    const float *w;
    float eps;
    void *h, *y;
    int8_t *codes;
    float *scales;
    int rows, D;
    long long sx, sr, sh, sy;       // row strides (elements) of x, residual, h and y / codes
};

// V weights (the weight is only 4-byte aligned for certain; its rows are read
// again by every block, from the caches).
template <int V>
__device__ __forceinline__ Vec<float, V> load_weight(const float *w)
{
    Vec<float, V> r;
#pragma unroll
    for (int q = 0; q < V; ++q)
        r.v[q] = __ldg(w + q);
    return r;
}

// Sums of a and maxima of b over the row's threads (blockDim.x of them), the
// same in every thread.  red: 2 x 32 floats a row of the block.
__device__ __forceinline__ void row_reduce(float &a, float &b, float *red)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        a += __shfl_xor_sync(kFullMask, a, o);
        b = fmaxf(b, __shfl_xor_sync(kFullMask, b, o));
    }
    const int nw = blockDim.x >> 5;
    if (nw == 1)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
        red[warp] = a;
        red[32 + warp] = b;
    }
    __syncthreads();
    a = lane < nw ? red[lane] : 0.f;
    b = lane < nw ? red[32 + lane] : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        a += __shfl_xor_sync(kFullMask, a, o);
        b = fmaxf(b, __shfl_xor_sync(kFullMask, b, o));
    }
}

// threadIdx.x walks a row (vector j of a thread: j * blockDim.x + threadIdx.x),
// threadIdx.y the rows of the block (more than one only with one warp a row).
template <class TX, class TR, int V, int NV, int MODE>
__global__ void __launch_bounds__(kNormThreads) add_norm_kernel(const NormArgs a)
{
    griddep_entry();
    __shared__ float red[64];
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= a.rows)
        return;
    const TX *x = static_cast<const TX *>(a.x) + row * a.sx;
    Vec<TX, V> xv[NV];
    Vec<TR, V> rv[NV];
    const int nvec = a.D / V;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = j * blockDim.x + threadIdx.x;
        if (c < nvec)
            xv[j] = load_vec<TX, V>(x + (long long)c * V);
    }
    const bool add = MODE != kCodesOnly && a.residual != nullptr;
    if (add) {
        const TR *r = static_cast<const TR *>(a.residual) + row * a.sr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < nvec)
                rv[j] = load_vec<TR, V>(r + (long long)c * V);
        }
    }
    float v[NV][V];                                        // h, or h w for the codes
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = j * blockDim.x + threadIdx.x;
        if (c < nvec) {
            Vec<float, V> w;
            if (MODE == kNormCodes)
                w = load_weight<V>(a.w + (long long)c * V);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                float h = to_float(xv[j].v[q]);
                if (add) {
                    rv[j].v[q] = from_float<TR>(h + to_float(rv[j].v[q]));
                    h = to_float(rv[j].v[q]);
                }
                ss = fmaf(h, h, ss);
                v[j][q] = MODE == kNormCodes ? __fmul_rn(h, w.v[q]) : h;
                if (MODE != kNormOut)
                    top = fmaxf(top, fabsf(v[j][q]));
            }
            if (add && a.h)
                store_vec<TR, V>(static_cast<TR *>(a.h) + row * a.sh + (long long)c * V, rv[j]);
        }
    }
    row_reduce(ss, top, red);
    const float inv = 1.f / sqrtf(ss / (float)a.D + a.eps);
    if (MODE == kNormOut) {
        TX *y = static_cast<TX *>(a.y) + row * a.sy;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < nvec) {
                Vec<TX, V> o;
                const Vec<float, V> w = load_weight<V>(a.w + (long long)c * V);
#pragma unroll
                for (int q = 0; q < V; ++q)
                    o.v[q] = from_float<TX>(v[j][q] * inv * w.v[q]);
                store_vec<TX, V>(y + (long long)c * V, o);
            }
        }
        return;
    }
    const float f = fminf(__fdiv_rn(127.f, top), FLT_MAX);
    int8_t *codes = a.codes + row * a.sy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = j * blockDim.x + threadIdx.x;
        if (c < nvec) {
            Vec<int8_t, V> o;
#pragma unroll
            for (int q = 0; q < V; ++q)
                o.v[q] = (int8_t)__float2int_rn(__fmul_rn(v[j][q], f));
            store_vec<int8_t, V>(codes + (long long)c * V, o);
        }
    }
    if (threadIdx.x == 0) {
        // a NaN among the values does not reach the maximum, but it does reach the sum
        const float one = MODE == kCodesOnly ? (ss == ss ? 1.f : ss) : inv;
        a.scales[row] = top <= FLT_MAX ? one / f : __int_as_float(0x7fc00000);
    }
}

// ---- gradient ----

struct NormGradArgs {
    const void *gy, *h, *gh;
    const float *w;
    float eps;
    void *gin;
    float *gw, *part;
    int rows, D;
    long long sgy, sh, sgh, sgi;
};

// A block walks rows blockIdx.x * blockDim.y + threadIdx.y, ... and keeps its
// columns' share of grad_w in registers; its sum goes to row blockIdx.x of part.
template <class TY, class TR, int V, int NV>
__global__ void __launch_bounds__(V == 8 ? 256 : kNormThreads) add_norm_backward_kernel(const NormGradArgs a)
{
    griddep_entry();
    __shared__ float red[2][64];
    const int nvec = a.D / V;
    Vec<float, V> w[NV];
    float gw[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = j * blockDim.x + threadIdx.x;
#pragma unroll
        for (int q = 0; q < V; ++q) {
            w[j].v[q] = c < nvec ? __ldg(a.w + (long long)c * V + q) : 0.f;
            gw[j][q] = 0.f;
        }
    }
    int flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const TY *gy = static_cast<const TY *>(a.gy) + row * a.sgy;
        const TR *h = static_cast<const TR *>(a.h) + row * a.sh;
        Vec<TY, V> g[NV];
        Vec<TR, V> hv[NV], gh[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < nvec) {
                g[j] = load_vec<TY, V>(gy + (long long)c * V);
                hv[j] = load_vec<TR, V>(h + (long long)c * V);
                if (a.gh)
                    gh[j] = load_vec<TR, V>(static_cast<const TR *>(a.gh) + row * a.sgh + (long long)c * V);
            }
        }
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < nvec)
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float hf = to_float(hv[j].v[q]);
                    ss = fmaf(hf, hf, ss);
                    dot = fmaf(to_float(g[j].v[q]) * w[j].v[q], hf, dot);
                }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            ss += __shfl_xor_sync(kFullMask, ss, o);
            dot += __shfl_xor_sync(kFullMask, dot, o);
        }
        const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
        if (nw > 1) {
            if (lane == 0) {
                red[flip][threadIdx.x >> 5] = ss;
                red[flip][32 + (threadIdx.x >> 5)] = dot;
            }
            __syncthreads();                               // the other buffer is free again after the next one
            ss = lane < nw ? red[flip][lane] : 0.f;
            dot = lane < nw ? red[flip][32 + lane] : 0.f;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
                ss += __shfl_xor_sync(kFullMask, ss, o);
                dot += __shfl_xor_sync(kFullMask, dot, o);
            }
        }
        const float inv = 1.f / sqrtf(ss / (float)a.D + a.eps);
        const float s = dot * inv / (float)a.D;            // mean(n w gy)
        TR *gin = static_cast<TR *>(a.gin) + row * a.sgi;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < nvec) {
                Vec<TR, V> o;
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float n = to_float(hv[j].v[q]) * inv, gq = to_float(g[j].v[q]);
                    float d = inv * fmaf(-n, s, gq * w[j].v[q]);
                    if (a.gh)
                        d += to_float(gh[j].v[q]);
                    o.v[q] = from_float<TR>(d);
                    gw[j][q] = fmaf(gq, n, gw[j][q]);
                }
                store_vec<TR, V>(gin + (long long)c * V, o);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = j * blockDim.x + threadIdx.x;
        if (c < nvec)
#pragma unroll
            for (int q = 0; q < V; ++q)
                a.part[(long long)blockIdx.x * a.D + (long long)c * V + q] = gw[j][q];
    }
}

// grad_w from the blocks' sums in a fixed order: 8 warps a block of 32 columns.
__global__ void __launch_bounds__(256)
norm_weight_kernel(const float *part, int nparts, int D, float *gw)
{
    griddep_entry();
    __shared__ float sum[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < D)
        for (int k = warp; k < nparts; k += 8)
            s += part[(long long)k * D + c];
    sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < D) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s += sum[k][lane];
        gw[c] = s;
    }
}

// Threads a row and vectors a thread.  The widest row (16384) fits: 32 scalars x
// 512 threads, 8 vectors of 4 x 512, 8 vectors of 8 x 256.
struct RowShape {
    int threads, nv;
};

RowShape row_shape(int nvec, int most)
{
    RowShape s{32, 1};
    while (s.nv < most && (nvec + s.nv - 1) / s.nv > 256)
        s.nv *= 2;
    const int t = (nvec + s.nv - 1) / s.nv;
    s.threads = (t + 31) / 32 * 32;
    return s;
}

template <class TX, class TR, int V, int MODE>
cudaError_t launch_norm_v(const NormArgs &a, cudaStream_t st)
{
    const RowShape s = row_shape(a.D / V, V == 1 ? 32 : 8);
    const int rows = s.threads == 32 ? 4 : 1;
    const dim3 grid((unsigned)((a.rows + rows - 1) / rows)), block(s.threads, rows);
    if (s.threads > kNormThreads)
        return cudaErrorInvalidValue;
    switch (s.nv) {
    case 1: return launch_pdl(add_norm_kernel<TX, TR, V, 1, MODE>, grid, block, 0, st, a);
    case 2: return launch_pdl(add_norm_kernel<TX, TR, V, 2, MODE>, grid, block, 0, st, a);
    case 4: return launch_pdl(add_norm_kernel<TX, TR, V, 4, MODE>, grid, block, 0, st, a);
    case 8: return launch_pdl(add_norm_kernel<TX, TR, V, 8, MODE>, grid, block, 0, st, a);
    default: break;
    }
    if constexpr (V == 1) {
        if (s.nv == 16)
            return launch_pdl(add_norm_kernel<TX, TR, V, 16, MODE>, grid, block, 0, st, a);
        return launch_pdl(add_norm_kernel<TX, TR, V, 32, MODE>, grid, block, 0, st, a);
    }
    return cudaErrorInvalidValue;
}

template <class TX, class TR, int MODE>
cudaError_t launch_norm_t(const NormArgs &a, cudaStream_t st)
{
    constexpr int V = sizeof(TX) == 2 && sizeof(TR) == 2 ? 8 : 4;
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y);
    const uintptr_t r = reinterpret_cast<uintptr_t>(a.residual) | reinterpret_cast<uintptr_t>(a.h);
    const long long strides = a.D | a.sx | a.sr | a.sh | a.sy;
    const bool vec = strides % V == 0 && p % (V * sizeof(TX)) == 0 && r % (V * sizeof(TR)) == 0 &&
                     reinterpret_cast<uintptr_t>(a.codes) % V == 0;
    return vec ? launch_norm_v<TX, TR, V, MODE>(a, st) : launch_norm_v<TX, TR, 1, MODE>(a, st);
}

template <int MODE>
cudaError_t launch_norm(const NormArgs &a, int dx, int dr, cudaStream_t st)
{
    if (dx == kF32)
        return launch_norm_t<float, float, MODE>(a, st);
    if (dx == kBF16)
        return dr == kF32 ? launch_norm_t<__nv_bfloat16, float, MODE>(a, st)
                          : launch_norm_t<__nv_bfloat16, __nv_bfloat16, MODE>(a, st);
    return dr == kF32 ? launch_norm_t<__half, float, MODE>(a, st) : launch_norm_t<__half, __half, MODE>(a, st);
}

template <class TY, class TR, int V>
cudaError_t launch_norm_grad_v(const NormGradArgs &a, int nparts, cudaStream_t st)
{
    const RowShape s = row_shape(a.D / V, V == 1 ? 32 : 8);
    const dim3 grid((unsigned)nparts), block(s.threads);
    if (s.threads > kNormThreads)
        return cudaErrorInvalidValue;
    switch (s.nv) {
    case 1: return launch_pdl(add_norm_backward_kernel<TY, TR, V, 1>, grid, block, 0, st, a);
    case 2: return launch_pdl(add_norm_backward_kernel<TY, TR, V, 2>, grid, block, 0, st, a);
    case 4: return launch_pdl(add_norm_backward_kernel<TY, TR, V, 4>, grid, block, 0, st, a);
    case 8: return launch_pdl(add_norm_backward_kernel<TY, TR, V, 8>, grid, block, 0, st, a);
    default: break;
    }
    if constexpr (V == 1) {
        if (s.nv == 16)
            return launch_pdl(add_norm_backward_kernel<TY, TR, V, 16>, grid, block, 0, st, a);
        return launch_pdl(add_norm_backward_kernel<TY, TR, V, 32>, grid, block, 0, st, a);
    }
    return cudaErrorInvalidValue;
}

template <class TY, class TR>
cudaError_t launch_norm_grad_t(const NormGradArgs &a, int nparts, cudaStream_t st)
{
    constexpr int V = sizeof(TY) == 2 && sizeof(TR) == 2 ? 8 : 4;
    const uintptr_t r = reinterpret_cast<uintptr_t>(a.h) | reinterpret_cast<uintptr_t>(a.gh) |
                        reinterpret_cast<uintptr_t>(a.gin);
    const long long strides = a.D | a.sgy | a.sh | a.sgh | a.sgi;
    const bool vec = strides % V == 0 && reinterpret_cast<uintptr_t>(a.gy) % (V * sizeof(TY)) == 0 &&
                     r % (V * sizeof(TR)) == 0;
    return vec ? launch_norm_grad_v<TY, TR, V>(a, nparts, st) : launch_norm_grad_v<TY, TR, 1>(a, nparts, st);
}

}  // namespace

cudaError_t launch_add_norm(const void *x, const void *residual, const float *w, float eps, void *h, void *y,
                            int8_t *codes, float *scales, int rows, int D, int dx, int dr, long long sx,
                            long long sr, long long sh, long long sy, cudaStream_t st)
{
    NormArgs a{x, residual, w, eps, h, y, codes, scales, rows, D, sx, residual ? sr : 0, h ? sh : 0, sy};
    if (!w)
        return launch_norm<kCodesOnly>(a, dx, dx, st);
    return codes ? launch_norm<kNormCodes>(a, dx, dr, st) : launch_norm<kNormOut>(a, dx, dr, st);
}

int add_norm_parts(int rows) { return rows < 304 ? (rows < 1 ? 1 : rows) : 304; }

cudaError_t launch_add_norm_backward(const void *gy, const void *h, const void *gh, const float *w, float eps,
                                     void *gin, float *gw, float *part, int rows, int D, int dy, int dr,
                                     long long sgy, long long sh, long long sgh, long long sgi, cudaStream_t st)
{
    NormGradArgs a{gy, h, gh, w, eps, gin, gw, part, rows, D, sgy, sh, gh ? sgh : 0, sgi};
    const int nparts = add_norm_parts(rows);
    cudaError_t e;
    if (dy == kF32)
        e = launch_norm_grad_t<float, float>(a, nparts, st);
    else if (dy == kBF16)
        e = dr == kF32 ? launch_norm_grad_t<__nv_bfloat16, float>(a, nparts, st)
                       : launch_norm_grad_t<__nv_bfloat16, __nv_bfloat16>(a, nparts, st);
    else
        e = dr == kF32 ? launch_norm_grad_t<__half, float>(a, nparts, st)
                       : launch_norm_grad_t<__half, __half>(a, nparts, st);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(norm_weight_kernel, dim3((unsigned)((D + 31) / 32)), dim3(256), 0, st, (const float *)part,
                      nparts, D, gw);
}

}  // namespace ssm
