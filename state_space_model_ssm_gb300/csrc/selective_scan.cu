// Selective scan with a decay for each channel and state, forward (sm_103a).
// Formulas and the layout of a warp: selective_common.cuh.
//
// The walk itself: selective_walk.cuh.
#include <algorithm>

#include "selective_walk.cuh"

namespace ssm {

namespace {

// Units of every sequence: one, or as many segments as its tokens take.
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
        const int len = seq < a.n_seqs ? sel_seq_len(a, seq, t0) : 0;
        const int mine = seq >= a.n_seqs ? 0 : len <= a.whole ? 1 : (len + a.seg - 1) / a.seg;
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

// The state entering each unit, in place of the unit's state from zero.  grid: (channels and states, shares of the
// sequences); a whole sequence reads its slot itself.
__global__ void __launch_bounds__(256)
sel_combine_kernel(const SelArgs a)
{
    griddep_entry();
    const long long width = (long long)a.channels * a.N, e = (long long)blockIdx.x * 256 + threadIdx.x;
    if (e >= width)
        return;
    const int c = (int)(e / a.N);
    const float A = a.A[e] * kLog2e;
    for (int seq = blockIdx.y; seq < a.n_seqs; seq += gridDim.y) {
        const int u0 = a.first[seq], u1 = a.first[seq + 1];
        if (u1 - u0 <= 1)
            continue;
        float h = a.resume[seq] != 0 ? a.state[seq * width + e] : 0.f;
        // loads of a run of units together (one by one, each waited for the store before it)
        for (int u = u0; u < u1; u += kCombineRun) {
            float own[kCombineRun], step[kCombineRun];
#pragma unroll
            for (int k = 0; k < kCombineRun; ++k) {
                const long long v = min(u + k, u1 - 1);
                own[k] = a.unit_state[v * width + e];
                step[k] = a.unit_step[v * a.channels + c];
            }
#pragma unroll
            for (int k = 0; k < kCombineRun; ++k) {
                if (u + k >= u1)
                    break;
                a.unit_state[(u + k) * width + e] = h;
                h = sel_passed(h, step[k] * A, own[k]);     // (the last unit's values are not there, and not used)
            }
        }
    }
}

template <class T>
cudaError_t launch_type(const SelArgs &a, int units, cudaStream_t st)
{
    if (a.seg) {
        cudaError_t e = launch_walk_states<T, kState>(a, units, st);
        if (e != cudaSuccess)
            return e;
        e = launch_pdl(sel_combine_kernel, sel_combine_grid(a), dim3(256), 0, st, a);
        if (e != cudaSuccess)
            return e;
    }
    return launch_walk_states<T, kFull>(a, units, st);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

long long sel_chunk_rows(long long n_seqs, long long n_tokens) { return n_seqs + n_tokens / kSelChunk + 1; }

SelShape sel_shape(int channels, int N, int groups, bool backward)
{
    // lanes of a channel: eight states each in the walks, four in the backward kernel
    const int lanes = (N <= 16 ? 2 : N <= 32 ? 4 : N <= 64 ? 8 : 16) * (backward ? 2 : 1);
    SelShape s;
    s.wc = 32 / lanes * kSelCh;
    s.cblocks = groups * sel_group_blocks(channels, groups, s.wc);
    s.tiles = groups * ((channels / groups + s.wc - 1) / s.wc);
    return s;
}

// The walks' blocks of channels with narrow tiles.
int sel_narrow_blocks(int channels, int N, int groups)
{
    const int lanes = N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32;
    return groups * sel_group_blocks(channels, groups, 32 / lanes * 2);
}

// Tokens of a segment, for `resident` blocks at once and `cblocks` of them a unit.
// Up to 8 sequences: the one for which rounds of blocks take the least time, r rounds of segments that are just short
// enough for r, if the sequences were alike.  More of them are rarely alike and the longest, cut too coarsely, ends last:
// `rounds` of all tokens.  That also bounds how many units there are beside the sequences.  Both, in us, bf16, 16 states:
//   4 x 777 tokens x 1001 channels x 13, fp32, forward and backward     alike 210   rounds 234
//   6508 and four short sequences x 320 channels, the same              alike 220   rounds 251
//   20 x 300 and one of 3000 tokens x 4096 channels                     alike 335, forward and backward 1647   rounds 326, 1520
//   60 x 200 and one of 1000                                            alike 505, 2767                        rounds 459, 2686
//   16 x 512 and one of 4096                                            alike 466, 2518                        rounds 470, 2072
// One round of all tokens takes 932 forward where 100 sequences of 128 and one of 4096 take 562 with four.
long long sel_segment(int n_seqs, int n_tokens, long long cblocks, long long resident, int rounds)
{
    const long long each = (n_tokens + n_seqs - 1) / n_seqs;
    if (n_seqs > 8) {
        const long long even = (n_tokens * cblocks + rounds * resident - 1) / (rounds * resident);
        return std::max(64LL, (even + kSelChunk - 1) / kSelChunk * kSelChunk);
    }
    long long best = 0, least = 0;
    for (int r = 1; r <= 4; ++r) {
        const long long units = std::max(1LL, r * resident / cblocks / n_seqs);     // of a sequence
        const long long seg = std::max(64LL, ((each + units - 1) / units + kSelChunk - 1) / kSelChunk * kSelChunk);
        const long long blocks = n_seqs * ((each + seg - 1) / seg) * cblocks;
        const long long time = (blocks + resident - 1) / resident * seg;
        if (r == 1 || time < least) {
            best = seg;
            least = time;
        }
    }
    return best;
}

SelCut sel_cut(int n_seqs, int n_tokens, int channels, int N, int groups, bool backward)
{
    // Warps that are resident at once (three blocks an SM; two backward), and the tokens that each would walk if
    // all had the same to do.  A sequence of at most one and a half times that is not worth the second walk.
    const SelShape s = sel_shape(channels, N, groups, backward);
    const long long blocks = kSms * (backward ? 2 : 3), warps = kSelWarps * blocks;
    const long long even = ((long long)n_tokens * s.tiles + warps - 1) / warps, whole = even + even / 2 < 128 ? 128 : even + even / 2;
    if (n_tokens <= whole || n_tokens == n_seqs)            // (as many tokens as sequences: a decode step)
        return SelCut{0, 0};
    long long seg = sel_segment(n_seqs, n_tokens, s.cblocks, blocks, backward ? 8 : 4);
    if (!backward && sel_narrow(n_seqs, n_tokens, sel_max_units(n_seqs, n_tokens, (int)seg), s.tiles))
        seg = sel_segment(n_seqs, n_tokens, sel_narrow_blocks(channels, N, groups), 5 * kSms, 4);
    return SelCut{(int)seg, (int)std::max(whole, seg)};
}

// Whether the walks take narrow tiles.  Wide ones have four channels and eight states (four, up to 8 states) a
// lane.  Where that leaves the device without work, or has little to do but loads, four states and two channels a lane,
// a quarter of the work and four times the warps, take less time: a warp alone on its scheduler waits for its own
// instructions.  4096 channels x 16 states, bf16, one token a sequence, wide / narrow: 16 sequences 9.3 / 6.9 us,
// 32 14.9 / 10.3, 64 23.8 / 21.6, 256 75.8 / 76.8; 1 x 4096 tokens 209 / 259.
bool sel_narrow(int n_seqs, int n_tokens, int units, int tiles)
{
    return (long long)units * tiles < (n_tokens <= 8LL * n_seqs ? 48 : 6) * (long long)kSms;
}

// Whether two channels of each of these rows are one aligned word.
bool sel_pairs(const SelArgs &a, int dtype)
{
    const int e = dtype_size(dtype);
    auto even = [&](const void *p, long long stride) {
        return !p || (reinterpret_cast<uintptr_t>(p) % (2 * e) == 0 && stride % 2 == 0);
    };
    return a.channels / a.groups % 2 == 0 && even(a.x, a.sx) && even(a.dt, a.sdt) && even(a.z, a.sz) && even(a.y, a.sy) &&
           even(a.grad_y, a.sgy) && even(a.grad_x, a.sgx) && even(a.grad_dt, a.sgdt) && even(a.grad_z, a.sgz);
}

// Of the combining kernels: at most as many shares of the sequences as can have been cut.
dim3 sel_combine_grid(const SelArgs &a)
{
    const long long width = (long long)a.channels * a.N, cut = a.n_tokens / (a.whole + 1LL) + 1;
    return dim3((unsigned)((width + 255) / 256), (unsigned)std::min<long long>({cut, a.n_seqs, 65535}));
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
    const int seg = sel_cut(n_seqs, n_tokens, channels, N, groups, false).seg;
    return seg ? layout(n_seqs, channels, N, sel_max_units(n_seqs, n_tokens, seg)).total : 0;
}

cudaError_t launch_selective_scan(SelArgs a, int dtype, void *workspace, cudaStream_t st)
{
    const SelShape s = sel_shape(a.channels, a.N, a.groups, false);
    a.cblocks = s.cblocks;
    a.pairs = sel_pairs(a, dtype);
    const SelCut cut = sel_cut(a.n_seqs, a.n_tokens, a.channels, a.N, a.groups, false);
    a.seg = cut.seg;
    a.whole = cut.whole;
    const int units = sel_max_units(a.n_seqs, a.n_tokens, a.seg);
    a.narrow = sel_narrow(a.n_seqs, a.n_tokens, units, s.tiles);
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
