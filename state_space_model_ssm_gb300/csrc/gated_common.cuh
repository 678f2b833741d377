// The gated linear recurrence: arguments, gates and the passing of state
// between time chunks, shared by the forward and the backward kernel.
//
// For token t of a sequence and channel c:
//
//   r = sigmoid(gate_a), i = sigmoid(gate_x)
//   log a = -decay_scale softplus(lam[c]) r,  a = exp(log a),  m = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + b_t,  b_t = m_t i_t x_t,  y_t = h_t
//
// Time chunks.  The map of a run of tokens on the state is h -> P h + H, P the
// product of its a_t and H the state it leaves from zero, and two such maps
// compose: (P2, H2) after (P1, H1) is (P1 P2, P2 H1 + H2).  So a sequence is cut
// into chunks of kGatedChunk tokens, a block scans one chunk of some channels
// from zero, publishes (P, H), and obtains the state that enters its chunk from
// the chunks before it: from the nearest one whose outgoing state is already
// known and the (P, H) of those between.  Every input is read once.  Blocks
// take their chunk from a counter in time order (tickets), so a chunk that a
// block waits for is always in the hands of a block that runs already.
#pragma once

#include "layer_common.cuh"

namespace ssm {

constexpr int kGatedLen = 8;                               // tokens a thread holds in registers
constexpr int kGatedWarps = 8;                             // runs of kGatedLen tokens per block
constexpr int kGatedChunk = kGatedLen * kGatedWarps;       // tokens of a time chunk

struct GatedArgs {
    float *state;                       // [n][C], in/out (forward)
    const void *x, *gate_a, *gate_x;    // [T][C], token strides below
    const float *lam;                   // [C]
    float decay_scale;
    void *y;                            // forward: [T][C]
    const int32_t *seq_starts, *seq_lens, *resume;
    int n_seqs, n_tokens, C;
    long long sx, sga, sgx, sy;         // token strides (elements)
    float *chunk_states;                // [units][C]: the state entering each chunk (forward: out, may be null)
    // backward
    const void *grad_y;                 // [T][C], token stride sy
    const float *grad_state;            // [n][C] gradient of the slots after the call, or null
    void *grad_x, *grad_ga, *grad_gx;   // [T][C], token strides gsx, gsga, gsgx
    long long gsx, gsga, gsgx;
    float *grad_lam;                    // [C]
    float *grad_state0;                 // [n][C] gradient of the slots before the call, or null
    // workspace
    int max_units;
    int cblocks;                        // channel blocks of the launch (the stride of flags)
    int2 *units;                        // (sequence, chunk) of each unit, sequences in order
    int *unit_base;                     // [n + 1] first unit of each sequence
    int *control;                       // [0] units, [1] ticket, [2] status
    int *flags;                         // [units][cblocks]: 0 nothing, 1 (P, H), 2 the outgoing state
    float *agg_p, *agg_h;               // [units][C]
    float *out_state;                   // [units][C]
    float *lam_part;                    // [units][C] (backward)
};

// A sequence's token range; one that is not inside the packed rows counts as empty.
__device__ __forceinline__ int gated_seq_len(const GatedArgs &a, int seq, long long &t0)
{
    t0 = a.seq_starts[seq];
    const long long len = a.seq_lens[seq];
    return t0 >= 0 && len > 0 && t0 + len <= a.n_tokens ? (int)len : 0;
}

__device__ __forceinline__ float softplus_f(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// 1 / (1 + e^-v) from the hardware exponential and an approximate division
// (a few 1e-7 relative; 0 and 1 at the infinities, NaN stays).
__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// One token's decay.  d = 1 - a with v = -log a >= 0: for v < 1/4 the Taylor
// series of 1 - e^-v to v^7 (the next term is below 2e-9 relative), else 1 - e^-v.
// A long memory multiplies hundreds of decays close to 1, where the hardware
// exponential's error (2^-22) would add up; 1 - d is rounded once (2^-25).  And
// m^2 = 1 - a^2 = d (1 + a) keeps its digits where a is close to 1.
struct Decay {
    float a, m, im;                     // a, sqrt(1 - a^2) and its inverse
};

__device__ __forceinline__ Decay decay_of(float v)
{
    float s = fmaf(v, -1.f / 7.f, 1.f);
    s = fmaf(v * (-1.f / 6.f), s, 1.f);
    s = fmaf(v * (-1.f / 5.f), s, 1.f);
    s = fmaf(v * (-1.f / 4.f), s, 1.f);
    s = fmaf(v * (-1.f / 3.f), s, 1.f);
    s = fmaf(v * (-1.f / 2.f), s, 1.f);
    s *= v;
    const float e = __expf(-v);
    Decay r;
    r.a = v < 0.25f ? 1.f - s : e;
    const float m2 = (v < 0.25f ? s : 1.f - e) * (1.f + r.a);
    // m2 = 0 (a closed gate) gives m ~ 1e-19, whose products with the gate's
    // vanishing derivative are zero, and not 0 / 0
    r.im = rsqrtf(fmaxf(m2, 1e-38f));
    r.m = m2 * r.im;
    return r;
}

// State (or its gradient) arriving at unit u from the units on its side `dir`
// (-1: earlier chunks, +1: later ones) down to `last`, the sequence's end on
// that side.  Called by one warp; lane's channels c0 .. c0 + V - 1 (V values in
// s).  It waits until one of the nearest 32 units has its outgoing state and
// every unit between has its (P, H), and applies those from the far one to the
// near one: s -> P s + H, the very operation each of those units does for its own
// outgoing state, so the bits do not depend on which unit was found.  Returns
// false when the bounded wait gave up.
template <int V>
__device__ __forceinline__ bool gated_gather(const GatedArgs &a, int u, int dir, int last, int cb, int c0, int lane,
                                             float (&s)[V])
{
    const int idx = u + dir * (lane + 1);
    const bool valid = dir < 0 ? idx >= last : idx <= last;
    const int *flag = a.flags + (long long)idx * a.cblocks + cb;
    for (int spin = 0; spin < (1 << 22); ++spin) {
        const int f = valid ? ld_acquire(flag) : 0;
        const unsigned known = __ballot_sync(kFullMask, f == 2), none = __ballot_sync(kFullMask, f == 0);
        if (known && (none == 0 || __ffs(known) < __ffs(none))) {
            __syncwarp();                                  // the lanes' acquires order every lane's reads below
            if (c0 < a.C) {
                int k = __ffs(known);
                const long long step = (long long)dir * a.C;
                const float *p = a.agg_p + (long long)u * a.C + c0, *h = a.agg_h + (long long)u * a.C + c0;
                const float *o = a.out_state + (long long)u * a.C + c0 + k * step;
#pragma unroll
                for (int q = 0; q < V; ++q)
                    s[q] = __ldcg(o + q);
#pragma unroll 4
                for (--k; k > 0; --k)
#pragma unroll
                    for (int q = 0; q < V; ++q)
                        s[q] = fmaf(__ldcg(p + k * step + q), s[q], __ldcg(h + k * step + q));
            }
            return true;
        }
        if (spin > 8)
            __nanosleep(32);
    }
    return false;
}

// Host side.  Chunks of a batch: at most one begun chunk a sequence beside the full ones.
long long gated_max_units(long long n_seqs, long long n_tokens);
size_t gated_workspace_bytes(int n_seqs, int n_tokens, int C);
cudaError_t launch_gated_scan(GatedArgs a, int dtype, void *workspace, cudaStream_t stream);
cudaError_t launch_gated_scan_backward(GatedArgs a, int dtype, void *workspace, cudaStream_t stream);
// Two channels a thread where every row starts on a pair.
bool gated_pairs(const GatedArgs &a, int dtype, bool backward);
void gated_carve(GatedArgs &a, void *workspace);
cudaError_t launch_gated_plan(const GatedArgs &a, cudaStream_t stream);

}  // namespace ssm
