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
// an infinity in h or v has codes 0 and scale NaN, so its values are NaN (an infinite
// or NaN h makes v infinite or NaN whatever the weight, so only v is looked at: a NaN
// counts as an infinite maximum).  The quantiser is the same with v = x and inv = 1.
//
// Gradient, with n = h inv and s = mean(n w gy):
//   grad_in = grad_h + inv (w gy - n s),  grad_w = sum over rows of gy n
#include <cfloat>

#include "layer_common.cuh"

namespace ssm {

namespace {

// Most threads of a block: 256 slots a pass and one for the offset, but 16384 fp32
// values are 4097 slots of 4, 8 a thread.
constexpr int norm_threads(int V, int NV) { return V == 4 && NV == 8 ? 544 : 288; }
constexpr int kGradThreads = 544;         // the gradient's: rows over 512 threads before a second slot a thread
constexpr int kNormOut = 0, kNormCodes = 1, kCodesOnly = 2;

// A row is walked in slots of V elements; slot c begins at element c V - m.  How the
// rows lie is a compile-time matter (no access is chosen at run time between a
// vector and its elements except at a row's two ends):
//   kAligned   every row of every tensor begins and ends on a boundary of V elements
//              (16 bytes of 16-bit types, 16 or 8 beside an fp32 residual): m = 0
//   kAlike     rows begin anywhere, but all tensors' rows alike: m is the row's offset
//              from the boundary before it, a slot inside the row is one access, and
//              the ones at its ends go element by element
//   kElements  anything else: m = 0, element by element
// kAlike costs about 1.5 times kAligned and a third of kElements (quantising
// 4108 x 6145 fp16: 28 us against 81).
constexpr int kAligned = 0, kAlike = 1, kElements = 2;

template <class T, int V>
__device__ __forceinline__ int slot_offset(const T *row) { return (int)(reinterpret_cast<uintptr_t>(row) / sizeof(T) % V); }

template <class T, int V, int LAY>
__device__ __forceinline__ Vec<T, V> load_slot(const T *row, int e0, int D)
{
    Vec<T, V> v;
    if constexpr (LAY == kAligned) {
        v = load_vec<T, V>(row + e0);
    } else if (LAY == kAlike && e0 >= 0 && e0 + V <= D) {
        v = load_vec<T, V>(row + e0);
    } else {
#pragma unroll
        for (int q = 0; q < V; ++q)
            v.v[q] = e0 + q >= 0 && e0 + q < D ? row[e0 + q] : from_float<T>(0.f);
    }
    return v;
}

template <class T, int V, int LAY>
__device__ __forceinline__ void store_slot(T *row, int e0, int D, const Vec<T, V> &v)
{
    if constexpr (LAY == kAligned) {
        store_vec<T, V>(row + e0, v);
    } else if (LAY == kAlike && e0 >= 0 && e0 + V <= D) {
        store_vec<T, V>(row + e0, v);
    } else {
#pragma unroll
        for (int q = 0; q < V; ++q)
            if (e0 + q >= 0 && e0 + q < D)
                row[e0 + q] = v.v[q];
    }
}

// The slot's weights (read again by every row: from the caches).
template <int V, int LAY>
__device__ __forceinline__ Vec<float, V> load_weight(const float *w, int e0, int D)
{
    Vec<float, V> r;
    if constexpr (LAY == kAligned) {
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(w + e0 + q));
            r.v[q] = f.x; r.v[q + 1] = f.y; r.v[q + 2] = f.z; r.v[q + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int q = 0; q < V; ++q)
            r.v[q] = e0 + q >= 0 && e0 + q < D ? __ldg(w + e0 + q) : 0.f;
    }
    return r;
}

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

// The larger one; a NaN if either is one.
__device__ __forceinline__ float max_or_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
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

// threadIdx.x walks a row (slot j of a thread: j * blockDim.x + threadIdx.x),
// threadIdx.y the rows of the block (more than one only with one warp a row).
template <class TX, class TR, int V, int NV, int MODE, int LAY>
__global__ void __launch_bounds__(norm_threads(V, NV)) add_norm_kernel(const NormArgs a)
{
    griddep_entry();
    __shared__ float red[64];
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= a.rows)
        return;
    const TX *x = static_cast<const TX *>(a.x) + row * a.sx;
    const int D = a.D, m = LAY == kAlike ? slot_offset<TX, V>(x) : 0, slots = (D + m + V - 1) / V;
    Vec<TX, V> xv[NV];
    Vec<TR, V> rv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = j * blockDim.x + threadIdx.x;
        if (c < slots)
            xv[j] = load_slot<TX, V, LAY>(x, c * V - m, D);
    }
    const bool add = MODE != kCodesOnly && a.residual != nullptr;
    if (add) {
        const TR *r = static_cast<const TR *>(a.residual) + row * a.sr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < slots)
                rv[j] = load_slot<TR, V, LAY>(r, c * V - m, D);
        }
    }
    TR *hrow = add && a.h ? static_cast<TR *>(a.h) + row * a.sh : nullptr;
    float v[NV][V];                                        // h, or h w for the codes
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = j * blockDim.x + threadIdx.x;
        if (c < slots) {
            Vec<float, V> w;
            if (MODE == kNormCodes)
                w = load_weight<V, LAY>(a.w, c * V - m, D);
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
                    top = max_or_nan(top, fabsf(v[j][q]));
            }
            if (hrow)
                store_slot<TR, V, LAY>(hrow, c * V - m, D, rv[j]);
        }
    }
    if (MODE != kNormOut && top != top)
        top = __int_as_float(0x7f800000);                  // (the row's maximum passes over NaN)
    row_reduce(ss, top, red);
    const float inv = 1.f / sqrtf(ss / (float)D + a.eps);
    if (MODE == kNormOut) {
        TX *y = static_cast<TX *>(a.y) + row * a.sy;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < slots) {
                Vec<TX, V> o;
                const Vec<float, V> w = load_weight<V, LAY>(a.w, c * V - m, D);
#pragma unroll
                for (int q = 0; q < V; ++q)
                    o.v[q] = from_float<TX>(v[j][q] * inv * w.v[q]);
                store_slot<TX, V, LAY>(y, c * V - m, D, o);
            }
        }
        return;
    }
    const float f = fminf(__fdiv_rn(127.f, top), FLT_MAX);
    int8_t *codes = a.codes + row * a.sy;
    // bytes from a slot's codes back to their boundary (the codes' rows need not lie like x's)
    const int shift = LAY == kAlike ? (slot_offset<int8_t, V>(codes) + V - m) % V : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = j * blockDim.x + threadIdx.x;
        uint64_t word = 0;
        const int e0 = c * V - m;
        const bool whole = c < slots && e0 >= 0 && e0 + V <= D;
        if (c < slots) {
#pragma unroll
            for (int q = 0; q < V; ++q)
                word |= (uint64_t)(uint8_t)__float2int_rn(__fmul_rn(v[j][q], f)) << (8 * q);
        }
        bool straddles = false;
        if constexpr (LAY == kAlike && V == 8) {
            straddles = shift != 0;
            if (straddles) {
                // The codes of a slot straddle two aligned words: each lane writes the one that
                // holds its last `shift` codes and the next lane's first.
                const uint64_t next = __shfl_down_sync(kFullMask, word, 1);
                const unsigned ws = __ballot_sync(kFullMask, whole);
                const int lane = threadIdx.x & 31;
                const bool up = lane < 31 && whole && (ws >> (lane + 1) & 1), down = lane > 0 && whole && (ws >> (lane - 1) & 1);
                if (up)
                    *reinterpret_cast<uint64_t *>(codes + e0 + V - shift) = word >> (8 * (V - shift)) | next << (8 * shift);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const bool covered = q < V - shift ? down : up;
                    if (c < slots && !covered && e0 + q >= 0 && e0 + q < D)
                        codes[e0 + q] = (int8_t)(word >> (8 * q));
                }
            }
        }
        if (!straddles && c < slots) {
            Vec<int8_t, V> o;
#pragma unroll
            for (int q = 0; q < V; ++q)
                o.v[q] = (int8_t)(word >> (8 * q));
            if (LAY == kAlike && shift != 0)
                store_slot<int8_t, V, kElements>(codes, e0, D, o);
            else
                store_slot<int8_t, V, LAY>(codes, e0, D, o);
        }
    }
    if (threadIdx.x == 0)
        a.scales[row] = top <= FLT_MAX ? (MODE == kCodesOnly ? 1.f : inv) / f : __int_as_float(0x7fc00000);
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

// A block walks rows blockIdx.x, blockIdx.x + gridDim.x, ... and keeps its columns'
// share of grad_w in registers; its sum goes to row blockIdx.x of part.  (A column
// belongs to one slot for all rows, so there is no kAlike form.)
template <class TY, class TR, int V, int NV, int LAY>
__global__ void __launch_bounds__(kGradThreads) add_norm_backward_kernel(const NormGradArgs a)
{
    griddep_entry();
    __shared__ float red[2][64];
    const int D = a.D, slots = (D + V - 1) / V;
    float gw[NV][V] = {};
    struct Row {
        Vec<TY, V> g[NV];
        Vec<TR, V> h[NV], gh[NV];
    };
    auto load = [&](long long row, Row &r) {
        const TY *gy = static_cast<const TY *>(a.gy) + row * a.sgy;
        const TR *h = static_cast<const TR *>(a.h) + row * a.sh;
        const TR *ghr = a.gh ? static_cast<const TR *>(a.gh) + row * a.sgh : nullptr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < slots) {
                r.g[j] = load_slot<TY, V, LAY>(gy, c * V, D);
                r.h[j] = load_slot<TR, V, LAY>(h, c * V, D);
                if (ghr)
                    r.gh[j] = load_slot<TR, V, LAY>(ghr, c * V, D);
            }
        }
    };
    auto process = [&](long long row, const Row &r, int flip) {
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < slots) {
                const Vec<float, V> w = load_weight<V, LAY>(a.w, c * V, D);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float hf = to_float(r.h[j].v[q]);
                    ss = fmaf(hf, hf, ss);
                    dot = fmaf(to_float(r.g[j].v[q]) * w.v[q], hf, dot);
                }
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
        const float inv = 1.f / sqrtf(ss / (float)D + a.eps);
        const float s = dot * inv / (float)D;              // mean(n w gy)
        TR *gin = static_cast<TR *>(a.gin) + row * a.sgi;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < slots) {
                const Vec<float, V> w = load_weight<V, LAY>(a.w, c * V, D);
                Vec<TR, V> o;
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float n = to_float(r.h[j].v[q]) * inv, gq = to_float(r.g[j].v[q]);
                    float d = inv * fmaf(-n, s, gq * w.v[q]);
                    if (a.gh)
                        d += to_float(r.gh[j].v[q]);
                    o.v[q] = from_float<TR>(d);
                    gw[j][q] = fmaf(gq, n, gw[j][q]);
                }
                store_slot<TR, V, LAY>(gin, c * V, D, o);
            }
        }
    };
    Row r;
    int flip = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        load(row, r);
        process(row, r, flip);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = j * blockDim.x + threadIdx.x;
        if (c < slots)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const int e = c * V + q;
                if (e < D)
                    a.part[(long long)blockIdx.x * D + e] = gw[j][q];
            }
    }
}

// grad_w from the blocks' sums in a fixed order: 32 warps a block of 32 columns, warp k
// adds rows k, k + 32, ...
__global__ void __launch_bounds__(1024)
norm_weight_kernel(const float *part, int nparts, int D, float *gw)
{
    griddep_entry();
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < D)
#pragma unroll 4
        for (int k = warp; k < nparts; k += 32)
            s += part[(long long)k * D + c];
    sum[lane][warp] = s;
    __syncthreads();
    s = sum[warp][lane];                                   // warp: column, lane: row of sums
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        s += __shfl_xor_sync(kFullMask, s, o);
    if (lane == 0 && blockIdx.x * 32 + warp < D)
        gw[blockIdx.x * 32 + warp] = s;
}

// Threads a row and slots a thread: up to `target` threads first.  (256 for the
// forward kernel, 4096 x 4096 bf16 in 8 bits: 22 us, with 128 or 64 threads 30; 512 for the
// gradient: 40 us, with 256 46.)
struct RowShape {
    int threads, nv;
};

RowShape row_shape(int D, int V, int lay, int target)
{
    const int slots = lay == kAlike ? (D + V - 2) / V + 1 : (D + V - 1) / V;   // at any offset
    RowShape s{32, 1};
    while (s.nv < 8 && (slots + s.nv - 1) / s.nv > target)
        s.nv *= 2;
    s.threads = ((slots + s.nv - 1) / s.nv + 31) / 32 * 32;
    return s;
}

template <class TX, class TR, int V, int MODE, int LAY>
cudaError_t launch_norm_v(const NormArgs &a, cudaStream_t st)
{
    const RowShape s = row_shape(a.D, V, LAY, 256);
    const unsigned rows = s.threads == 32 ? 4 : 1;
    const dim3 grid(((unsigned)a.rows + rows - 1) / rows), block(s.threads, rows);
    if (s.threads > norm_threads(V, s.nv))
        return cudaErrorInvalidValue;
    switch (s.nv) {
    case 1: return launch_pdl(add_norm_kernel<TX, TR, V, 1, MODE, LAY>, grid, block, 0, st, a);
    case 2: return launch_pdl(add_norm_kernel<TX, TR, V, 2, MODE, LAY>, grid, block, 0, st, a);
    case 4: return launch_pdl(add_norm_kernel<TX, TR, V, 4, MODE, LAY>, grid, block, 0, st, a);
    default: return launch_pdl(add_norm_kernel<TX, TR, V, 8, MODE, LAY>, grid, block, 0, st, a);
    }
}

template <class TX, class TR, int MODE>
cudaError_t launch_norm_t(const NormArgs &a, cudaStream_t st)
{
    constexpr int V = sizeof(TX) == 2 && sizeof(TR) == 2 ? 8 : 4;
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y);
    const uintptr_t r = reinterpret_cast<uintptr_t>(a.residual) | reinterpret_cast<uintptr_t>(a.h);
    const bool aligned = ((a.D | a.sx | a.sr | a.sh | a.sy) % V) == 0 && p % (V * sizeof(TX)) == 0 &&
                         r % (V * sizeof(TR)) == 0 && reinterpret_cast<uintptr_t>(a.codes) % V == 0 &&
                         reinterpret_cast<uintptr_t>(a.w) % 16 == 0;
    if (aligned)
        return launch_norm_v<TX, TR, V, MODE, kAligned>(a, st);
    if constexpr (MODE == kCodesOnly)                      // x's are the only rows that count
        return launch_norm_v<TX, TR, V, MODE, kAlike>(a, st);
    // rows of x, residual, h and y at the same offset from a boundary, row after row
    const long long mx = reinterpret_cast<uintptr_t>(a.x) / sizeof(TX) % V;
    auto alike = [&](const void *t, size_t size, long long stride) {
        return !t || ((long long)(reinterpret_cast<uintptr_t>(t) / size % V) == mx && (stride - a.sx) % V == 0);
    };
    const bool same = alike(a.residual, sizeof(TR), a.sr) && alike(a.h, sizeof(TR), a.sh) &&
                      (MODE != kNormOut || alike(a.y, sizeof(TX), a.sy));
    return same ? launch_norm_v<TX, TR, V, MODE, kAlike>(a, st) : launch_norm_v<TX, TR, V, MODE, kElements>(a, st);
}

template <class TX, int MODE>
cudaError_t launch_norm_r(const NormArgs &a, int dr, cudaStream_t st)
{
    if constexpr (MODE != kCodesOnly && sizeof(TX) == 2)   // the quantiser has no residual
        if (dr == kF32)
            return launch_norm_t<TX, float, MODE>(a, st);
    return launch_norm_t<TX, TX, MODE>(a, st);
}

template <int MODE>
cudaError_t launch_norm(const NormArgs &a, int dx, int dr, cudaStream_t st)
{
    if (dx == kF32)
        return launch_norm_r<float, MODE>(a, dr, st);
    return dx == kBF16 ? launch_norm_r<__nv_bfloat16, MODE>(a, dr, st) : launch_norm_r<__half, MODE>(a, dr, st);
}

template <class TY, class TR, int V, int LAY>
cudaError_t launch_norm_grad_v(const NormGradArgs &a, int nparts, cudaStream_t st)
{
    const RowShape s = row_shape(a.D, V, LAY, 512);
    const dim3 grid((unsigned)nparts), block(s.threads);
    if (s.threads > kGradThreads)
        return cudaErrorInvalidValue;
    switch (s.nv) {
    case 1: return launch_pdl(add_norm_backward_kernel<TY, TR, V, 1, LAY>, grid, block, 0, st, a);
    case 2: return launch_pdl(add_norm_backward_kernel<TY, TR, V, 2, LAY>, grid, block, 0, st, a);
    case 4: return launch_pdl(add_norm_backward_kernel<TY, TR, V, 4, LAY>, grid, block, 0, st, a);
    default: return launch_pdl(add_norm_backward_kernel<TY, TR, V, 8, LAY>, grid, block, 0, st, a);
    }
}

template <class TY, class TR>
cudaError_t launch_norm_grad_t(const NormGradArgs &a, int nparts, cudaStream_t st)
{
    constexpr int V = sizeof(TY) == 2 && sizeof(TR) == 2 ? 8 : 4;
    const uintptr_t r = reinterpret_cast<uintptr_t>(a.h) | reinterpret_cast<uintptr_t>(a.gh) |
                        reinterpret_cast<uintptr_t>(a.gin);
    const bool aligned = ((a.D | a.sgy | a.sh | a.sgh | a.sgi) % V) == 0 &&
                         reinterpret_cast<uintptr_t>(a.gy) % (V * sizeof(TY)) == 0 && r % (V * sizeof(TR)) == 0 &&
                         reinterpret_cast<uintptr_t>(a.w) % 16 == 0;
    return aligned ? launch_norm_grad_v<TY, TR, V, kAligned>(a, nparts, st)
                   : launch_norm_grad_v<TY, TR, V, kElements>(a, nparts, st);
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

// Blocks of the gradient (rows of partial sums): two an SM for wide rows, whose blocks
// are up to 544 threads, six for narrow ones (304 / 912 blocks, us: 4096 x 4096 bf16
// 40 / 46, 16384 x 512 71 / 31).
int add_norm_parts(int rows, int D)
{
    const int most = (D >= 2048 ? 2 : 6) * kSms;
    return rows < most ? (rows < 1 ? 1 : rows) : most;
}

cudaError_t launch_add_norm_backward(const void *gy, const void *h, const void *gh, const float *w, float eps,
                                     void *gin, float *gw, float *part, int rows, int D, int dy, int dr,
                                     long long sgy, long long sh, long long sgh, long long sgi, cudaStream_t st)
{
    NormGradArgs a{gy, h, gh, w, eps, gin, gw, part, rows, D, sgy, sh, gh ? sgh : 0, sgi};
    const int nparts = add_norm_parts(rows, D);
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
    return launch_pdl(norm_weight_kernel, dim3((unsigned)((D + 31) / 32)), dim3(1024), 0, st, (const float *)part,
                      nparts, D, gw);
}

}  // namespace ssm
