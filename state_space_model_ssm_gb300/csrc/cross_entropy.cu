// Softmax cross entropy of a projection onto a large vocabulary, and its gradients,
// without the logits in memory (sm_103a):
//
//   l[t,v] = sum_d h[t,d] w[v,d],  lse[t] = log sum_v exp l[t,v],  loss[t] = lse[t] - l[t,target[t]]
//   G[t,v] = (exp(l[t,v] - lse[t]) - [v = target[t]]) grad_loss[t],  grad h = G w,  grad w = G^T h
//
// Tokens whose target is ignored are left out before anything is multiplied: a first pass counts
// them, a second one writes the hidden rows of the others back to back (zeros up to a whole
// tile), so ignored tokens cost nothing and whatever stands in their rows reaches no sum.  How
// many remain is known on the device only; the products take it from there.
//
// Forward: a product (pair_gemm.cuh) whose epilogue keeps, for each row and 128 columns, the
// largest logit and the sum of the exponentials above it, and the target's logit; a small kernel
// joins them.  Backward, in pieces of the vocabulary: the product again, with G of the piece as
// its output in the inputs' 16-bit type; then grad h += G w and grad w = G^T h of the
// piece, whose operands the tensor cores read in either orientation.  Operations bound it: 2 T V D
// forward, 2 T V D again and 4 T V D backward.
//
// Roundings: G is rounded to 16 bits for its products (half a step of each term; the sums
// are fp32, and what is written is rounded once).  It is held relative to the largest finite |grad_loss|,
// so that a mean's 1 / T is no rounding, and for fp16 2^15 times that, so that probabilities down to
// 2^-29 keep all their bits; the sums get the factors back in fp32.  The tensor cores truncate as they add: at a width of
// 4096 the lse is off by 9e-6 (rms, logits of order one), 20 times what an fp32 product rounded to nearest is.
#include <algorithm>
#include <atomic>
#include <climits>

#include "packed.cuh"
#include "pair_gemm.cuh"

namespace ssm {

namespace {

constexpr int kCountRows = 1024;              // rows of a block of the counting kernel
constexpr int kPackRows = 8;                  // rows of a block of the packing kernel, a warp each
// Rows that every packing block counts by itself, without that kernel: up to here its launch costs as much (256 x 64,
// forward: 8192 rows counted by the blocks 16.6 us, 8200 by the kernel 16.2; 1024 by the blocks 11.2).
constexpr int kCountAlone = 8192;
constexpr int kJoinLanes = 32;                // threads that join a row's parts
constexpr int kGroupM = 16;                   // row tiles that share the vocabulary's rows in L2

struct LossArgs {
    const void *h, *w, *target, *grad_loss_lse;
    const float *grad_loss, *lse_in;
    float *loss, *lse;
    void *grad_h, *grad_w;
    int T, V, D, wide;                        // wide: 64-bit targets
    long long sh, sw, sgh, sgw, ignore;
    int dp;                                   // packed row length
    // workspace
    int *counts;                              // [blocks] kept rows of each kCountRows
    float *tops;                              // [blocks] largest finite |grad_loss| of them
    int *kept;                                // rows that are kept
    float *top;                               // largest finite |grad_loss| of them, 1 if that is 0
    int *index;                               // [T] row of each kept one
    int *label;                               // [T rounded up to a tile] its target, -1 past the end
    float *scale;                             // its grad_loss relative to the largest, times the type's factor
    float *row_lse;
    float *label_logit;                       // [T]
    float2 *part;                             // [2 vocabulary tiles][T rounded up]
    void *hp, *wp, *G;
    float *acc;                               // [splits][T rounded up][dp] fp32: grad h of the pieces or splits
    int t_pad, blocks;                        // T rounded up to a tile
    float factor;                             // 2^15 for fp16, else 1
    int v0, vp, first_piece, last_piece;      // a piece of the vocabulary
    int splits;                               // most pairs that share a tile of grad h
    int fail_waits;
};

__device__ __forceinline__ long long target_of(const LossArgs &a, int t)
{
    return a.wide ? static_cast<const long long *>(a.target)[t] : (long long)static_cast<const int32_t *>(a.target)[t];
}

// A block's sum and maximum, for all threads.
struct Counted {
    int n;
    float m;
};

__device__ __forceinline__ Counted block_sum(int n, float m)
{
    __shared__ int ns[8];
    __shared__ float ms[8];
#pragma unroll
    for (int off = 16; off >= 1; off /= 2) {
        n += __shfl_xor_sync(kFullMask, n, off);
        m = fmaxf(m, __shfl_xor_sync(kFullMask, m, off));
    }
    __syncthreads();                                        // (of an earlier call)
    if ((threadIdx.x & 31) == 0) {
        ns[threadIdx.x >> 5] = n;
        ms[threadIdx.x >> 5] = m;
    }
    __syncthreads();
    Counted c{0, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c.n += ns[i];
        c.m = fmaxf(c.m, ms[i]);
    }
    return c;
}

// Kept ones of rows [t0, t1), and the largest finite |grad_loss| of them (a NaN's or an infinity's row is no number
// by itself; as what the others are relative to, it would take them along).
__device__ __forceinline__ Counted count_rows(const LossArgs &a, int t0, int t1, bool tops)
{
    int n = 0;
    float m = 0.f;
#pragma unroll 4
    for (int t = t0 + threadIdx.x; t < t1; t += 256) {
        const bool keep = target_of(a, t) != a.ignore;
        n += keep ? 1 : 0;
        if (tops) {
            const float g = keep ? fabsf(a.grad_loss[t]) : 0.f;
            m = fmaxf(m, g < INFINITY ? g : 0.f);
        }
    }
    return block_sum(n, m);
}

__global__ void __launch_bounds__(256)
loss_count_kernel(const LossArgs a)
{
    griddep_entry();
    const int t0 = blockIdx.x * kCountRows;
    const Counted c = count_rows(a, t0, min(a.T, t0 + kCountRows), a.grad_loss != nullptr);
    if (threadIdx.x == 0) {
        a.counts[blockIdx.x] = c.n;
        a.tops[blockIdx.x] = c.m;
    }
}

// Kept rows back to back, zeros after them up to a whole tile; outputs of ignored rows.
template <class T>
__global__ void __launch_bounds__(256)
loss_pack_kernel(const LossArgs a)
{
    griddep_entry();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r0 = blockIdx.x * kPackRows, r = r0 + warp;
    const bool vec = ((reinterpret_cast<uintptr_t>(a.h) | (uintptr_t)(a.sh * 2)) & 15) == 0;
    // kept rows before this block's, and of all of them (for the gradient's scale, and behind the last row)
    int before;
    Counted all;
    if (a.T <= kCountAlone) {
        before = count_rows(a, 0, min(r0, a.T), false).n;
        all = count_rows(a, min(r0, a.T), a.T, false);
        all.n += before;
        if (a.grad_loss)
            all.m = count_rows(a, 0, a.T, true).m;
    } else {
        const int whole = min(r0, a.T) / kCountRows;
        int n = 0, every = 0;
        float m = 0.f;
        for (int i = threadIdx.x; i < a.blocks; i += 256) {
            const int c = a.counts[i];
            every += c;
            n += i < whole ? c : 0;
            m = fmaxf(m, a.tops[i]);
        }
        before = block_sum(n, 0.f).n + count_rows(a, whole * kCountRows, min(r0, a.T), false).n;
        all = block_sum(every, m);
    }
    if (all.m == 0.f)                                       // (rows that are no number stay so)
        all.m = 1.f;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *a.kept = all.n;
        *a.top = all.m;
    }
    const bool real = r < a.T;
    const long long label = real ? target_of(a, r) : 0;
    if (real && label == a.ignore) {
        if (lane == 0 && a.loss)
            a.loss[r] = a.lse[r] = 0.f;
        if (a.grad_h)
            for (int d = lane; d < a.D; d += 32)
                static_cast<T *>(a.grad_h)[r * a.sgh + d] = from_float<T>(0.f);
        return;
    }
    int at = before;
    if (real) {
        const unsigned keep = __ballot_sync(kFullMask, lane < warp && target_of(a, r0 + min(lane, warp)) != a.ignore);
        at += __popc(keep);
    } else {
        at = all.n + r - a.T;
        if (at >= (all.n + pair::kTileM - 1) / pair::kTileM * pair::kTileM)
            return;
    }
    const T *src = static_cast<const T *>(a.h) + (real ? r * a.sh : 0);
    T *dst = static_cast<T *>(a.hp) + (long long)at * a.dp;
    constexpr int kAhead = 4;
    for (int d0 = lane * 8; d0 < a.dp; d0 += 256 * kAhead) {
        Vec<T, 8> v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int d = d0 + 256 * k;
            if (real && vec && d + 8 <= a.D) {
                v[k] = load_vec<T, 8>(src + d);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[k].v[i] = real && d + i < a.D ? src[d + i] : from_float<T>(0.f);
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (d0 + 256 * k < a.dp)
                store_vec<T, 8>(dst + d0 + 256 * k, v[k]);
    }
    if (lane == 0) {
        const bool in = label >= 0 && label < a.V;
        a.label[at] = real && in ? (int)label : -1;
        if (real)
            a.index[at] = r;
        if (a.grad_loss) {
            // a target outside the vocabulary has no loss: NaN
            const float g = real ? a.grad_loss[r] : 0.f;
            a.scale[at] = real && !in ? __int_as_float(0x7fc00000) : g == 0.f ? 0.f : g / all.m * a.factor;
            a.row_lse[at] = real ? a.lse_in[r] : 0.f;
        }
    }
}

// Weight rows that TMA cannot describe, as rows of dp values.
template <class T>
__global__ void __launch_bounds__(256)
loss_pack_weight_kernel(const LossArgs a)
{
    griddep_entry();
    const int per = a.dp / 8;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, r = i / per;
    const int d = (int)(i - r * per) * 8;
    if (r >= a.V)
        return;
    const T *src = static_cast<const T *>(a.w) + r * a.sw + d;
    Vec<T, 8> v;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v.v[e] = d + e < a.D ? src[e] : from_float<T>(0.f);
    store_vec<T, 8>(static_cast<T *>(a.wp) + r * a.dp + d, v);
}

// Largest logit (times log2 e) and the sum of the exponentials above it, of 128 columns of a row.
struct StatsEpilogue {
    const LossArgs &a;
    int rows;
    __device__ __forceinline__ void tile(int row, int col, uint32_t at, bool ok, bool any, int split, float *block)
    {
        const int label = row < rows ? a.label[row] : -1;
        float m = -INFINITY, s = 0.f;
#pragma unroll 1
        for (int j = 0; j < pair::kHalf; j += 32) {
            float v[32];
            pair::columns(v, at, j, ok, any);
            const int c = col + j;
            if (label >= c && label < c + 32) {
                float own = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    own = label == c + i ? v[i] : own;
                a.label_logit[row] = own;
            }
            if (c + 32 > a.V) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[i] = c + i < a.V ? v[i] : -INFINITY;
            }
            float top = v[0];                               // (a maximum drops a NaN; its exponential keeps it)
#pragma unroll
            for (int i = 1; i < 32; ++i)
                top = fmaxf(top, v[i]);
            top = fmaxf(m, top * kLog2e);
            if (fabsf(top) == INFINITY) {                   // an infinite logit: sum 1; or columns past the last, logits of
#pragma unroll                                              // -inf, NaN alone: no terms
                for (int i = 0; i < 32; ++i)
                    s = v[i] != v[i] ? v[i] : s;
                s = top > 0.f && s == s ? 1.f : s;
                m = top;
            } else {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    sum += ex2(fmaf(v[i], kLog2e, -top));
                s = fmaf(s, ex2(m - top), sum);
                m = top;
            }
        }
        if (row < rows)
            a.part[(long long)(col / pair::kHalf) * a.t_pad + row] = make_float2(ok ? m : __int_as_float(0x7fc00000), s);
    }
};

template <bool BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair::kThreads, 1)
loss_stats_kernel(const LossArgs a, const __grid_constant__ CUtensorMap hmap, const __grid_constant__ CUtensorMap wmap)
{
    pair::run<BF16, false, false>(kGroupM, hmap, wmap, a.fail_waits, [&] {
        const int rows = *a.kept;
        return pair::Work<StatsEpilogue>{{rows, a.V, a.D, 1}, {a, rows}};
    });
}

// G of a piece: rows up to a whole tile, zeros past the rows and past the vocabulary.
template <class T>
struct GradEpilogue {
    const LossArgs &a;
    __device__ __forceinline__ void tile(int row, int col, uint32_t at, bool ok, bool any, int split, float *block)
    {
        const int label = a.label[row] - a.v0;
        const float scale = a.scale[row], lse = a.row_lse[row] * kLog2e;
        T *out = static_cast<T *>(a.G) + (long long)row * a.vp + col;
        const int left = a.V - a.v0;                        // of the piece's columns that exist
#pragma unroll 1
        for (int j = 0; j < pair::kHalf; j += 32) {
            float v[32];
            pair::columns(v, at, j, ok, any);
            const int c = col + j;
            Vec<T, 8> o[4];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float p = ex2(fmaf(v[i], kLog2e, -lse)) - (label == c + i ? 1.f : 0.f);
                o[i / 8].v[i % 8] = from_float<T>(c + i < left ? p * scale : 0.f);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                store_vec<T, 8>(out + j + 8 * i, o[i]);
        }
    }
};

template <class T, bool BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair::kThreads, 1)
loss_grad_kernel(const LossArgs a, const __grid_constant__ CUtensorMap hmap, const __grid_constant__ CUtensorMap wmap)
{
    pair::run<BF16, false, false>(kGroupM, hmap, wmap, a.fail_waits,
                                  [&] { return pair::Work<GradEpilogue<T>>{{*a.kept, a.vp, a.D, 1}, {a}}; });
}

// 32 columns of a warp's rows in 16 bits: `out` a lane's row (null: none), `left` how many columns exist.  Rows
// on 16-byte boundaries are written as they lie in the lanes; others go through shared memory, so that
// the lanes write neighbouring columns (grad w of 466 x 32003 x 1001 fp16: element by element along
// rows 263 us, so 53).
template <class T>
__device__ __forceinline__ void write_rows(T *out, const float (&v)[32], int left, float back, bool aligned, float *block)
{
    const int lane = threadIdx.x & 31;
    if (aligned && left >= 32) {
        if (out)
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                Vec<T, 8> o;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    o.v[k] = from_float<T>(v[i + k] * back);
                store_vec<T, 8>(out + i, o);
            }
        return;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i)
        block[lane * 33 + i] = v[i] * back;
    __syncwarp();
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
        T *row = reinterpret_cast<T *>(__shfl_sync(kFullMask, reinterpret_cast<unsigned long long>(out), r));
        if (row && lane < left)
            row[lane] = from_float<T>(block[r * 33 + lane]);
    }
}

// Pairs that share a tile's terms (the vocabulary) where rows and width alone do not give every pair a tile.
__host__ __device__ __forceinline__ int splits_of(int pairs, int rows, int D, int most)
{
    const int tiles = ((rows + pair::kTileM - 1) / pair::kTileM) * ((D + pair::kTileN - 1) / pair::kTileN);
    const int n = tiles > 0 ? pairs / tiles : 1;
    return n < 1 ? 1 : n > most ? most : n;
}

// grad h.  Sums that are whole go where they belong; those of a split, or of a piece that is not the last, to fp32
// rows, in which pieces add up.
template <class T>
struct HiddenEpilogue {
    const LossArgs &a;
    int rows;
    float back;
    bool aligned;
    __device__ __forceinline__ void tile(int row, int col, uint32_t at, bool ok, bool any, int split, float *block)
    {
        const bool in = row < rows, direct = a.splits == 1 && a.last_piece;
        float *acc = a.acc + ((long long)split * a.t_pad + row) * a.dp + col;
        T *out = in && direct ? static_cast<T *>(a.grad_h) + a.index[row] * a.sgh + col : nullptr;
#pragma unroll 1
        for (int j = 0; j < pair::kHalf; j += 32) {
            float v[32];
            pair::columns(v, at, j, ok, any);
            if (col + j >= a.D)
                continue;
            if (in && (a.splits > 1 || !direct || !a.first_piece)) {    // rows of acc are dp long: whole groups of 4
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    if (col + j + i >= a.dp)
                        break;
                    float4 *p = reinterpret_cast<float4 *>(acc + j + i);
                    if (!a.first_piece) {
                        const float4 q = *p;
                        v[i] += q.x; v[i + 1] += q.y; v[i + 2] += q.z; v[i + 3] += q.w;
                    }
                    if (!direct)
                        *p = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
            if (direct)
                write_rows<T>(out ? out + j : nullptr, v, a.D - col - j, back, aligned, block);
        }
    }
};

template <class T, bool BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair::kThreads, 1)
loss_hidden_kernel(const LossArgs a, const __grid_constant__ CUtensorMap gmap, const __grid_constant__ CUtensorMap wmap)
{
    const bool aligned = ((reinterpret_cast<uintptr_t>(a.grad_h) | (uintptr_t)(a.sgh * 2)) & 15) == 0;
    pair::run<BF16, false, true>(kGroupM, gmap, wmap, a.fail_waits, [&] {
        const int rows = *a.kept, splits = splits_of(gridDim.x / 2, rows, a.D, a.splits);
        return pair::Work<HiddenEpilogue<T>>{{rows, a.D, min(a.vp, a.V - a.v0), splits}, {a, rows, *a.top / a.factor, aligned}};
    });
}

// Rows of grad h from their splits' sums, where they belong: a block a row.
template <class T>
__global__ void __launch_bounds__(128)
loss_hidden_join_kernel(const LossArgs a, int pairs)
{
    griddep_entry();
    const int row = blockIdx.x, rows = *a.kept;
    if (row >= rows)
        return;
    const int splits = splits_of(pairs, rows, a.D, a.splits);
    const float back = *a.top / a.factor;
    const long long next = (long long)a.t_pad * a.dp;
    T *out = static_cast<T *>(a.grad_h) + a.index[row] * a.sgh;
    for (int d = threadIdx.x; d < a.D; d += 128) {
        const float *p = a.acc + (long long)row * a.dp + d;
        float v = 0.f;
        for (int s0 = 0; s0 < splits; s0 += 8) {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q[i] = p[min(s0 + i, splits - 1) * next];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v += s0 + i < splits ? q[i] : 0.f;
        }
        out[d] = from_float<T>(v * back);
    }
}

template <class T>
struct WeightEpilogue {
    const LossArgs &a;
    float back;
    bool aligned;
    __device__ __forceinline__ void tile(int row, int col, uint32_t at, bool ok, bool any, int split, float *block)
    {
        const int v = a.v0 + row;
        const bool in = v < a.V && row < a.vp;
        T *out = in ? static_cast<T *>(a.grad_w) + v * a.sgw + col : nullptr;
#pragma unroll 1
        for (int j = 0; j < pair::kHalf; j += 32) {
            float x[32];
            pair::columns(x, at, j, ok, any);
            if (col + j < a.D)
                write_rows<T>(in ? out + j : nullptr, x, a.D - col - j, back, aligned, block);
        }
    }
};

template <class T, bool BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair::kThreads, 1)
loss_weight_kernel(const LossArgs a, const __grid_constant__ CUtensorMap gmap, const __grid_constant__ CUtensorMap hmap)
{
    const bool aligned = ((reinterpret_cast<uintptr_t>(a.grad_w) | (uintptr_t)(a.sgw * 2)) & 15) == 0;
    pair::run<BF16, true, true>(kGroupM, gmap, hmap, a.fail_waits, [&] {
        return pair::Work<WeightEpilogue<T>>{{min(a.vp, a.V - a.v0), a.D, *a.kept, 1}, {a, *a.top / a.factor, aligned}};
    });
}

// (largest logit, sum) of two disjoint sets of columns.  Under an infinite maximum a finite part has no share, but for
// its NaN.
__device__ __forceinline__ float2 join(float2 p, float2 q)
{
    const float top = fmaxf(p.x, q.x);
    if (p.x != p.x || q.x != q.x)                           // a wait gave up
        return make_float2(__int_as_float(0x7fc00000), 0.f);
    if (fabsf(top) == INFINITY)
        return make_float2(top, (p.x == top ? p.y : 0.f * p.y) + (q.x == top ? q.y : 0.f * q.y));
    return make_float2(top, p.y * ex2(p.x - top) + q.y * ex2(q.x - top));
}

// lse and loss of every kept row from its parts: 32 rows a block, the parts over 32 warps.
__global__ void __launch_bounds__(32 * kJoinLanes)
loss_join_kernel(const LossArgs a, int parts)
{
    griddep_entry();
    __shared__ float2 sh[kJoinLanes][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x * 32 + lane;
    const int rows = *a.kept;
    if (blockIdx.x * 32 >= rows)
        return;
    constexpr int kRun = 8;                                 // parts whose loads are issued together
    float2 s = make_float2(-INFINITY, 0.f);
    for (int p0 = warp; p0 < parts; p0 += kJoinLanes * kRun) {
        float2 q[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            q[i] = a.part[(long long)min(p0 + i * kJoinLanes, parts - 1) * a.t_pad + min(row, rows - 1)];
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            if (p0 + i * kJoinLanes < parts)
                s = join(s, q[i]);
    }
    sh[warp][lane] = s;
    __syncthreads();
    // a warp's lanes join the 32 parts of one row
    s = sh[lane][warp];
#pragma unroll
    for (int off = 16; off >= 1; off /= 2)
        s = join(s, make_float2(__shfl_xor_sync(kFullMask, s.x, off), __shfl_xor_sync(kFullMask, s.y, off)));
    const int r = blockIdx.x * 32 + warp;
    if (lane != 0 || r >= rows)
        return;
    const float lse = fmaf(s.x, kLn2, logf(s.y));
    const int t = a.index[r], label = a.label[r];
    a.lse[t] = lse;
    a.loss[t] = label < 0 ? __int_as_float(0x7fc00000) : lse - a.label_logit[r];
}

// ---- host ----

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

bool encode(CUtensorMap *map, const void *p, bool bf16, long long width, long long rows, long long stride, int box_rows)
{
    const auto fn = tensor_map_encoder();
    if (!fn)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void *>(p), dims,
              strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

long long tiles_of(long long m, long long n)
{
    return ((m + pair::kTileM - 1) / pair::kTileM) * ((n + pair::kTileN - 1) / pair::kTileN);
}

// What lies where in the workspace.
struct Plan {
    int t_pad, blocks, dp, pieces, vp, splits;
    bool pack_w;
    size_t counts, tops, kept, index, label, scale, row_lse, logit, part, hp, wp, G, acc, total;
};

Plan plan(const void *w, int T, int V, int D, long long sw, bool backward)
{
    Plan p;
    p.t_pad = (T + pair::kTileM - 1) / pair::kTileM * pair::kTileM;
    p.blocks = (T + kCountRows - 1) / kCountRows;
    p.dp = (D + 7) / 8 * 8;
    p.pack_w = ((reinterpret_cast<uintptr_t>(w) | (uintptr_t)(sw * 2)) & 15) != 0;
    // G of a piece: up to 256 MB, or four times the hidden rows' fp32 sums (which every piece reads and writes)
    const size_t room = (size_t)16 * p.t_pad * p.dp > ((size_t)256 << 20) ? (size_t)16 * p.t_pad * p.dp : (size_t)256 << 20;
    const long long fits = (long long)(room / ((size_t)p.t_pad * 2) / pair::kTileN * pair::kTileN);
    const long long all = ((long long)V + pair::kTileN - 1) / pair::kTileN * pair::kTileN;
    const long long most = fits < pair::kTileN ? pair::kTileN : fits;
    p.pieces = (int)((all + most - 1) / most);
    p.vp = (int)((all / pair::kTileN + p.pieces - 1) / p.pieces * pair::kTileN);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t v = at;
        at += up256(bytes);
        return v;
    };
    p.counts = take((size_t)p.blocks * 4);
    p.tops = take((size_t)p.blocks * 4);
    p.kept = take(8);
    p.index = take((size_t)T * 4);
    p.label = take((size_t)p.t_pad * 4);
    p.hp = take((size_t)p.t_pad * p.dp * 2);
    p.wp = p.pack_w ? take((size_t)V * p.dp * 2) : at;
    if (backward) {
        p.scale = take((size_t)p.t_pad * 4);
        p.row_lse = take((size_t)p.t_pad * 4);
        p.G = take((size_t)p.t_pad * p.vp * 2);
        // with one piece and few tiles, splits: up to 16, at least 16 stages each, and 64 MB of sums
        p.splits = 1;
        if (p.pieces == 1) {
            const size_t sums = (size_t)p.t_pad * p.dp * 4;
            const long long most = std::min<long long>({16, p.vp / (16 * pair::kTerms), (long long)(((size_t)64 << 20) / sums)});
            if (most > 1 && tiles_of(T, D) * 2 <= kSms / 2)
                p.splits = (int)most;
        }
        p.acc = p.pieces > 1 || p.splits > 1 ? take((size_t)p.splits * p.t_pad * p.dp * 4) : at;
        p.logit = p.part = 0;
    } else {
        p.logit = take((size_t)T * 4);
        p.part = take((size_t)(all / pair::kHalf) * p.t_pad * sizeof(float2));
        p.scale = p.row_lse = p.G = p.acc = 0;
        p.splits = 1;
    }
    p.total = at;
    return p;
}

// Pairs of SMs that run at once (the pairs' tiles are dealt out among them).
template <class K>
int resident_pairs(K kernel)
{
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return kSms / 2;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kSms);
        cfg.blockDim = dim3(pair::kThreads);
        cfg.dynamicSmemBytes = pair::Smem::kTotal;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1)
            n = kSms / 2;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <class K>
cudaError_t launch_pairs(K kernel, long long tiles, cudaStream_t st, const LossArgs &a, const CUtensorMap &x, const CUtensorMap &y)
{
    const cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kernel), pair::Smem::kTotal);
    if (e != cudaSuccess)
        return e;
    const long long pairs = resident_pairs(kernel);
    return launch_pdl(kernel, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(pair::kThreads),
                      pair::Smem::kTotal, st, a, x, y);
}

template <class T, bool BF16>
cudaError_t launch_loss(LossArgs a, const Plan &p, bool backward, cudaStream_t st)
{
    cudaError_t e = cudaSuccess;
    if (a.T > kCountAlone)
        e = launch_pdl(loss_count_kernel, dim3(p.blocks), dim3(256), 0, st, a);
    if (e == cudaSuccess)
        e = launch_pdl(loss_pack_kernel<T>, dim3((a.T + pair::kTileM + kPackRows - 1) / kPackRows), dim3(256), 0, st, a);
    if (e == cudaSuccess && p.pack_w)
        e = launch_pdl(loss_pack_weight_kernel<T>, dim3((unsigned)(((long long)a.V * (a.dp / 8) + 255) / 256)), dim3(256), 0, st, a);
    if (e != cudaSuccess)
        return e;
    const void *w = p.pack_w ? a.wp : a.w;
    const long long sw = p.pack_w ? a.dp : a.sw;
    CUtensorMap hmap, wmap;
    if (!encode(&hmap, a.hp, BF16, a.dp, p.t_pad, a.dp, 128) || !encode(&wmap, w, BF16, a.D, a.V, sw, 128))
        return cudaErrorInvalidValue;
    if (!backward) {
        e = launch_pairs(loss_stats_kernel<BF16>, tiles_of(a.T, a.V), st, a, hmap, wmap);
        if (e != cudaSuccess)
            return e;
        const int parts = (a.V + pair::kHalf - 1) / pair::kHalf;
        return launch_pdl(loss_join_kernel, dim3((a.T + 31) / 32), dim3(32 * kJoinLanes), 0, st, a, parts);
    }
    CUtensorMap hmap_n, gmap, gmap_m;
    if (!encode(&hmap_n, a.hp, BF16, a.dp, p.t_pad, a.dp, 64) || !encode(&gmap, a.G, BF16, p.vp, p.t_pad, p.vp, 128) ||
        !encode(&gmap_m, a.G, BF16, p.vp, p.t_pad, p.vp, 64))
        return cudaErrorInvalidValue;
    for (int i = 0; i < p.pieces; ++i) {
        a.v0 = i * p.vp;
        a.vp = p.vp;
        a.first_piece = i == 0;
        a.last_piece = i == p.pieces - 1;
        const long long rows = (long long)a.V - a.v0 < a.vp ? a.V - a.v0 : a.vp;       // of the piece
        const unsigned char *wv = static_cast<const unsigned char *>(w) + (size_t)a.v0 * sw * 2;
        CUtensorMap wpiece, wpiece_n;
        if (!encode(&wpiece, wv, BF16, a.D, rows, sw, 128) || !encode(&wpiece_n, wv, BF16, a.D, rows, sw, 64))
            return cudaErrorInvalidValue;
        e = launch_pairs(loss_grad_kernel<T, BF16>, tiles_of(a.T, a.vp), st, a, hmap, wpiece);
        const long long tiles = a.splits > 1 ? INT_MAX : tiles_of(a.T, a.D);     // (every pair: the device knows the splits)
        if (e == cudaSuccess)
            e = launch_pairs(loss_hidden_kernel<T, BF16>, tiles, st, a, gmap, wpiece_n);
        if (e == cudaSuccess && a.splits > 1)
            e = launch_pdl(loss_hidden_join_kernel<T>, dim3(a.T), dim3(128), 0, st, a,
                           resident_pairs(loss_hidden_kernel<T, BF16>));
        if (e == cudaSuccess && a.grad_w)
            e = launch_pairs(loss_weight_kernel<T, BF16>, tiles_of(rows, a.D), st, a, gmap_m, hmap_n);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t cross_entropy_workspace_bytes(const void *w, int T, int V, int D, long long sw, bool backward)
{
    return plan(w, T, V, D, sw, backward).total;
}

cudaError_t launch_cross_entropy(const CrossEntropy &c, void *workspace, bool backward, cudaStream_t st)
{
    const Plan p = plan(c.w, c.T, c.V, c.D, c.sw, backward);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    LossArgs a{};
    a.h = c.h; a.w = c.w; a.target = c.target; a.grad_loss = c.grad_loss; a.lse_in = c.lse_in;
    a.loss = c.loss; a.lse = c.lse; a.grad_h = c.grad_h; a.grad_w = c.grad_w;
    a.T = c.T; a.V = c.V; a.D = c.D; a.wide = c.wide; a.ignore = c.ignore;
    a.sh = c.sh; a.sw = c.sw; a.sgh = c.sgh; a.sgw = c.sgw;
    a.dp = p.dp; a.t_pad = p.t_pad; a.blocks = p.blocks; a.splits = backward ? p.splits : 1;
    a.counts = reinterpret_cast<int *>(ws + p.counts);
    a.tops = reinterpret_cast<float *>(ws + p.tops);
    a.kept = reinterpret_cast<int *>(ws + p.kept);
    a.top = reinterpret_cast<float *>(ws + p.kept) + 1;
    a.index = reinterpret_cast<int *>(ws + p.index);
    a.label = reinterpret_cast<int *>(ws + p.label);
    a.scale = reinterpret_cast<float *>(ws + p.scale);
    a.row_lse = reinterpret_cast<float *>(ws + p.row_lse);
    a.label_logit = reinterpret_cast<float *>(ws + p.logit);
    a.part = reinterpret_cast<float2 *>(ws + p.part);
    a.hp = ws + p.hp; a.wp = ws + p.wp; a.G = ws + p.G;
    a.acc = reinterpret_cast<float *>(ws + p.acc);
    a.factor = c.dtype == kF16 ? 32768.f : 1.f;
    a.fail_waits = debug_fail_waits() ? 1 : 0;
    return c.dtype == kBF16 ? launch_loss<__nv_bfloat16, true>(a, p, backward, st) : launch_loss<__half, false>(a, p, backward, st);
}

}  // namespace ssm
