// The gated linear recurrence: arguments, gates and the passing of state
// between time chunks, shared by the forward and the backward kernel.
//
// For token t of a sequence and channel c:
//
//   r = sigmoid(gate_a), i = sigmoid(gate_x)
//   log a = -decay_scale softplus(lam[c]) r,  a = exp(log a),  m = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + b_t,  b_t = m_t i_t x_t,  y_t = h_t
//
// Time.  The map of a run of tokens on the state is h -> P h + H, P the product of
// its a_t and H the state it leaves from zero, and two such maps compose: (P2, H2)
// after (P1, H1) is (P1 P2, P2 H1 + H2).  A block owns 64 channels of one sequence and
// walks its time chunks of 64 tokens with the state carried in registers; inside a
// chunk its warps take a run of tokens each from zero and put their maps together
// through shared memory.  Where that leaves too few blocks, a cluster of R blocks
// shares the sequence: in a round its blocks take R consecutive chunks, send each
// other their chunk's map (16 bytes a channel pair, by asynchronous stores into the
// peers' shared memory), and each composes the maps before its own.  Every input
// is read once, there is no workspace and no word in global memory
// that anybody waits for; the order of every operation is fixed, so the bits are too.
//
// A first version cut time into chunks for independent blocks that passed their
// states on through global memory (look-back with flags): its fences and polls
// cost 13 us a chunk, 7 times the arithmetic.
#pragma once

#include "layer_common.cuh"
#include "tc_common.cuh"

namespace ssm {

constexpr int kGatedChunk = 64;                            // tokens of a time chunk
// A block's warps and the tokens of a warp's run, in registers: the forward kernel 8 x 8
// (its barriers cost more than the longer runs), the backward kernel 16 x 4 (it needs
// twice the registers a token).
constexpr int kForwardWarps = 8, kForwardRun = kGatedChunk / kForwardWarps;
constexpr int kBackwardWarps = 16, kBackwardRun = kGatedChunk / kBackwardWarps;
constexpr int kGatedCh = 64;                               // channels of a block: two a lane
constexpr int kGatedTile = kGatedChunk * kGatedCh;
constexpr int kGatedMaxCluster = 8;

struct GatedArgs {
    float *state;                       // [n][C], in/out (forward)
    const void *x, *gate_a, *gate_x;    // [T][C], token strides below
    const float *lam;                   // [C]
    float decay_scale;
    void *y;                            // forward: [T][C]
    const int32_t *seq_starts, *seq_lens, *resume;
    int n_seqs, n_tokens, C;
    long long sx, sga, sgx, sy;         // token strides (elements)
    float *chunk_states;                // the state entering each chunk (gated_chunk_row; forward: out, may be null)
    // backward
    const void *grad_y;                 // [T][C], token stride sy
    const float *grad_state;            // [n][C] gradient of the slots after the call, or null
    void *grad_x, *grad_ga, *grad_gx;   // [T][C], token strides gsx, gsga, gsgx
    long long gsx, gsga, gsgx;
    float *grad_lam;                    // [C]
    float *grad_state0;                 // [n][C] gradient of the slots before the call, or null
    float *lam_part;                    // [n * cluster][C] workspace
    int cblocks;                        // blocks of kGatedCh channels
    int cluster;                        // blocks that share a sequence's time
    int fail_waits;                     // test hook: bounded waits give up at once
    int step_most;                      // stepping kernels: longest sequence they take
};

// Row of chunk_states for chunk j of a sequence that starts at token t0: the first
// chunk's by the sequence, the others' by their position (two chunks that begin in
// the same 64 rows would overlap before them).  n_seqs + n_tokens / 64 + 1 rows.
__host__ __device__ __forceinline__ long long gated_chunk_row(int n_seqs, int seq, long long t0, int j)
{
    return j == 0 ? seq : n_seqs + t0 / kGatedChunk + j;
}

// Which sequence the n-th job takes: with up to 32 sequences the longest first, so that
// the longest walk does not begin when the others end (each lane holds one length;
// the n-th has n lengths before it).
__device__ __forceinline__ int gated_job_seq(const GatedArgs &a, int n, int lane)
{
    if (a.n_seqs > 32 || a.n_seqs == 1)
        return n;
    const int mine = lane < a.n_seqs ? a.seq_lens[lane] : 0;
    int before = 0;
    for (int k = 0; k < a.n_seqs; ++k) {
        const int other = __shfl_sync(kFullMask, mine, k);
        before += other > mine || (other == mine && k < lane) ? 1 : 0;
    }
    return __ffs(__ballot_sync(kFullMask, lane < a.n_seqs && before == n)) - 1;
}

// A sequence's token range; one that is not inside the packed rows counts as empty.
__device__ __forceinline__ int gated_seq_len(const GatedArgs &a, int seq, long long &t0)
{
    t0 = a.seq_starts[seq];
    const long long len = a.seq_lens[seq];
    if (t0 >= 0 && len > 0 && t0 + len <= a.n_tokens)
        return (int)len;
    t0 = 0;
    return 0;
}

// Sequences that a call of short ones leaves to the walk: those of more than step_most
// tokens, in order.  A block asks for the n-th of them with n growing (all threads; the
// same answer in each), so it reads the table once; -1 past the last one.
template <int WARPS>
struct GatedLongs {
    static constexpr int kEach = 4;                         // lengths a thread reads at a time
    uint32_t (*masks)[WARPS];                               // [kEach][WARPS], in shared memory
    int base = 0, before = 0;                               // lengths passed, long ones among them
    __device__ __forceinline__ int find(const GatedArgs &a, long long n)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        for (; base < a.n_seqs; base += kEach * 32 * WARPS) {
            __syncthreads();                                // the masks have been read
            unsigned any = 0;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int s = base + (e * WARPS + warp) * 32 + lane;
                long long t0;
                const unsigned m = __ballot_sync(kFullMask, s < a.n_seqs && gated_seq_len(a, s, t0) > a.step_most);
                if (lane == 0)
                    masks[e][warp] = m;
                any |= m;
            }
            if (!__syncthreads_or(any != 0))                // the usual case: no long one here
                continue;
            int seen = before;
            for (int e = 0; e < kEach * WARPS; ++e) {
                unsigned m = masks[e / WARPS][e % WARPS];
                if (n < seen + __popc(m)) {
                    for (; seen < n; ++seen)
                        m &= m - 1;
                    return base + e * 32 + __ffs(m) - 1;
                }
                seen += __popc(m);
            }
            before = seen;
        }
        return -1;
    }
};

// Blocks of the cluster that a sequence of this length has work for; the others leave at once.
__device__ __forceinline__ int gated_ranks(int len, int cluster)
{
    const int chunks = (len + kGatedChunk - 1) / kGatedChunk;
    int r = 1;
    while (r < cluster && r < chunks)
        r *= 2;
    return r;
}

__device__ __forceinline__ float softplus_f(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// Two channels at a time: sm_103a's packed fp32 operations.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float ex2(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rsq(float v)
{
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-v) from the hardware exponential and reciprocal (a few 1e-7
// relative; 0 and 1 at the infinities, NaN stays).
__device__ __forceinline__ float2 sigmoid2(float2 v)
{
    const float2 t = mul2(v, both(-kLog2e));
    const float2 d = add2(make_float2(ex2(t.x), ex2(t.y)), both(1.f));
    return make_float2(rcp(d.x), rcp(d.y));
}

// Both gates of a token's two channels, r = sigmoid(ga) and i = sigmoid(gx), with one
// reciprocal for the four: a special-function result costs eight times an fma's issue
// (16 a cycle and SM; with this the unit is 19 % busy in the forward walk, whose
// bound is the latency of its own arithmetic), and four denominators below 2^31
// have a product below 2^124.  So only for gates above kGateLow; `low` ones take a reciprocal each.  So do
// runs with a NaN: through the shared reciprocal it would reach the other channel.
constexpr float kGateLow = -21.f;         // e^21 < 2^31

template <bool LOW>
__device__ __forceinline__ void gates2(float2 ga, float2 gx, float2 &r, float2 &i)
{
    if (LOW) {
        r = sigmoid2(ga);
        i = sigmoid2(gx);
        return;
    }
    const float2 ta = mul2(ga, both(-kLog2e)), tx = mul2(gx, both(-kLog2e));
    const float2 da = add2(make_float2(ex2(ta.x), ex2(ta.y)), both(1.f));
    const float2 dx = add2(make_float2(ex2(tx.x), ex2(tx.y)), both(1.f));
    const float2 q = mul2(da, dx);
    const float inv = rcp(q.x * q.y);
    const float2 iq = mul2(make_float2(q.y, q.x), both(inv));       // 1 / q
    r = mul2(iq, dx);
    i = mul2(iq, da);
}

__device__ __forceinline__ float sigmoid_f(float v) { return rcp(1.f + ex2(v * -kLog2e)); }

// One token's decay of two channels.  d = 1 - a with v = -log a >= 0: for v < 1/4
// the Taylor series of 1 - e^-v to v^7 (the next term is below 2e-9 relative),
// else 1 - e^-v.  A long memory multiplies hundreds of decays close to 1, where
// the hardware exponential's error (2^-22) would add up; 1 - d is rounded once
// (2^-25).  And m^2 = 1 - a^2 = d (1 + a) keeps its digits where a is close to 1.
struct Decay {
    float2 a, m, im;                    // a, sqrt(1 - a^2) and its inverse
};

__device__ __forceinline__ Decay decay_of(float2 v)
{
    float2 s = fma2(v, both(1.f / 5040.f), both(-1.f / 720.f));
    s = fma2(s, v, both(1.f / 120.f));
    s = fma2(s, v, both(-1.f / 24.f));
    s = fma2(s, v, both(1.f / 6.f));
    s = fma2(s, v, both(-0.5f));
    s = fma2(s, v, both(1.f));
    s = mul2(s, v);
    const float2 t = mul2(v, both(-kLog2e));
    const float2 e = make_float2(ex2(t.x), ex2(t.y));
    const bool nx = v.x < 0.25f, ny = v.y < 0.25f;
    const float2 d = make_float2(nx ? s.x : 1.f - e.x, ny ? s.y : 1.f - e.y);
    Decay r;
    r.a = make_float2(nx ? 1.f - s.x : e.x, ny ? 1.f - s.y : e.y);
    const float2 m2 = fma2(d, r.a, d);
    // m2 = 0 (a closed gate) gives 1/m ~ 1e19, whose products with the gate's
    // vanishing derivative are zero, and not 0 / 0
    r.im = make_float2(rsq(fmaxf(m2.x, 2e-38f)), rsq(fmaxf(m2.y, 2e-38f)));
    r.m = mul2(m2, r.im);
    return r;
}

__device__ __forceinline__ float2 pair(float2 v) { return v; }
__device__ __forceinline__ float2 pair(__nv_bfloat162 v) { return __bfloat1622float2(v); }
__device__ __forceinline__ float2 pair(__half2 v) { return __half22float2(v); }

// Two neighbouring elements in shared memory as floats.
__device__ __forceinline__ float2 load_pair(const float *p) { return *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ float2 load_pair(const __nv_bfloat16 *p) { return pair(*reinterpret_cast<const __nv_bfloat162 *>(p)); }
__device__ __forceinline__ float2 load_pair(const __half *p) { return pair(*reinterpret_cast<const __half2 *>(p)); }

// Whether all of a warp's run of gates are above kGateLow; a NaN is not.  Minima that
// keep a NaN, on the stored type: one instruction for two 16-bit values.
__device__ __forceinline__ float min_or_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 min_pairs(float2 a, float2 b) { return make_float2(min_or_nan(a.x, b.x), min_or_nan(a.y, b.y)); }
__device__ __forceinline__ __nv_bfloat162 min_pairs(__nv_bfloat162 a, __nv_bfloat162 b) { return __hmin2_nan(a, b); }
__device__ __forceinline__ __half2 min_pairs(__half2 a, __half2 b) { return __hmin2_nan(a, b); }
template <class T>
struct PairOf;
template <>
struct PairOf<float> { using type = float2; };
template <>
struct PairOf<__nv_bfloat16> { using type = __nv_bfloat162; };
template <>
struct PairOf<__half> { using type = __half2; };

template <class T, int L>
__device__ __forceinline__ bool gates_above(const T *ga, const T *gx)
{
    using P = typename PairOf<T>::type;
    P least = *reinterpret_cast<const P *>(ga);
#pragma unroll
    for (int i = 0; i < L; ++i) {
        least = min_pairs(least, *reinterpret_cast<const P *>(ga + i * kGatedCh));
        least = min_pairs(least, *reinterpret_cast<const P *>(gx + i * kGatedCh));
    }
    const float2 v = pair(least);
    return __all_sync(kFullMask, v.x > kGateLow && v.y > kGateLow);
}

// v to p and p + 1: one store where the rows allow it (`pairs`: every row starts
// on a pair), the second element only inside the row (`two`).
template <class T>
__device__ __forceinline__ void store_pair(T *p, float2 v, bool pairs, bool two)
{
    Vec<T, 2> o;
    o.v[0] = from_float<T>(v.x);
    o.v[1] = from_float<T>(v.y);
    if (pairs && two) {
        store_vec<T, 2>(p, o);
    } else {
        p[0] = o.v[0];
        if (two)
            p[1] = o.v[1];
    }
}

template <bool B>
struct Flag {
    static constexpr bool value = B;
};

// Tokens t .. of one tensor (the chunk's, `n` of them) x the block's channels into
// shared memory [kGatedChunk][kGatedCh] for rows that TMA cannot describe: 4 bytes a
// copy where pairs of 16-bit elements (or fp32) lie on 4 bytes, else plain loads.
// Channels and tokens outside are zero.
template <class T>
__device__ __forceinline__ void gated_copy(T *dst, const void *src, long long stride, long long t, int n, int c, int C,
                                           bool words)
{
    const T *p = static_cast<const T *>(src) + t * stride + c;
    constexpr int E = 4 / sizeof(T);
    if (words) {
        for (int i = threadIdx.x; i < kGatedTile / E; i += blockDim.x) {
            const int row = i / (kGatedCh / E), col = i % (kGatedCh / E) * E;
            if (row < n && c + col < C)                     // (pairs: C is even)
                cp_async4(dst + i * E, p + row * stride + col);
            else
                *reinterpret_cast<uint32_t *>(dst + i * E) = 0;
        }
        return;
    }
    for (int i = threadIdx.x; i < kGatedTile; i += blockDim.x) {
        const int row = i / kGatedCh, col = i % kGatedCh;
        dst[i] = row < n && c + col < C ? p[row * stride + col] : from_float<T>(0.f);
    }
}

// One chunk's map of two channels, as the blocks of a cluster exchange it.
struct alignas(16) GatedMsg {
    float2 p, h;
};

// 16 bytes into block `rank` of the cluster, counted on its mbarrier (both given as
// addresses of this block).
__device__ __forceinline__ void send_map(uint32_t dst, uint32_t bar, uint32_t rank, const GatedMsg &m)
{
    asm volatile("{\n\t.reg .b32 d, b;\n\t"
                 "mapa.shared::cluster.u32 d, %0, %2;\n\tmapa.shared::cluster.u32 b, %1, %2;\n\t"
                 "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [d], {%3, %4, %5, %6}, [b];\n\t}\n"
                 ::"r"(dst), "r"(bar), "r"(rank), "f"(m.p.x), "f"(m.p.y), "f"(m.h.x), "f"(m.h.y) : "memory");
}

// Shared memory of the exchange: maps by round and sender.  A block sends round k + 1's
// map before it reads round k's, so a peer can be three rounds ahead of one
// that has not read round k yet: four buffers.
constexpr int kGatedBufs = 4;
struct GatedExchange {
    GatedMsg *msg;                      // [kGatedBufs][cluster][32], in dynamic shared memory
    uint64_t *bar;                      // [kGatedBufs]
    int cluster;
    __device__ __forceinline__ GatedMsg &at(int k, int rank, int lane) const
    {
        return msg[(k % kGatedBufs * cluster + rank) * 32 + lane];
    }
};
constexpr size_t gated_exchange_bytes(int cluster) { return cluster > 1 ? kGatedBufs * cluster * 32 * sizeof(GatedMsg) : 0; }

// Wait for an mbarrier phase; false after `cap` polls.
__device__ __forceinline__ bool gated_wait(uint64_t *bar, uint32_t parity, int cap)
{
    return tc::mbar_poll(tc::smem_u32(bar), parity, cap);
}

// Once at the kernel's start (thread 0), before gated_cluster_start.
__device__ __forceinline__ void exchange_init(const GatedExchange &x)
{
    for (int i = 0; i < kGatedBufs; ++i)
        tc::mbar_init(&x.bar[i], 1);
}

// Every block of the cluster runs and has its barriers (all threads).
__device__ __forceinline__ void gated_cluster_start(int cluster)
{
    if (cluster > 1) {
        asm volatile("barrier.cluster.arrive.release;\n" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory");
    } else {
        __syncthreads();
    }
}

// After a wait that gave up: NaN into this block's rows of tokens from chunk j0 on (every
// step-th chunk, down to 0 or up to the end), channels c .. c + 63.
template <class T>
__device__ __forceinline__ void gated_poison(T *out, long long stride, long long t0, int len, int j0, int step, int c, int C)
{
    const int width = min(kGatedCh, C - c);
    for (int j = j0; j >= 0 && (step < 0 || j * kGatedChunk < len); j += step)
        for (int i = threadIdx.x; i < kGatedChunk * width; i += blockDim.x) {
            const int t = j * kGatedChunk + i / width;
            if (t < len)
                out[(t0 + t) * stride + c + i % width] = from_float<T>(__int_as_float(0x7fc00000));
        }
}

// An mbarrier's place given back before it is initialised again (one thread; nobody waits for it).
__device__ __forceinline__ void mbar_inval(uint64_t *mbar)
{
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];\n" ::"r"(tc::smem_u32(mbar)) : "memory");
}

// No block leaves while a peer may still send to it (all threads).  A block whose waits all
// came through has met every map sent to it.  After a wait that gave up (ok false) maps may be
// on their way still: past the barrier no more are sent, and these get 20 us to land.
__device__ __forceinline__ void gated_cluster_end(int cluster, bool ok)
{
    __syncwarp();
    if (cluster > 1) {
        asm volatile("barrier.cluster.arrive.release;\n" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory");
        if (!ok)
            for (int i = 0; i < 20; ++i)
                __nanosleep(1000);
    }
}

// Round k's map of this block (rank) to the others (one whole warp).
__device__ __forceinline__ void exchange_send(const GatedExchange &x, int k, int rank, int cluster, int lane,
                                              const GatedMsg &m)
{
    const int b = k % kGatedBufs;
    x.at(k, rank, lane) = m;
    __syncwarp();                                           // before the arrival that publishes it
    if (lane == 0)
        tc::mbar_expect_tx(&x.bar[b], (cluster - 1) * 32 * sizeof(GatedMsg));
    __syncwarp();
    for (int r = 0; r < cluster; ++r)
        if (r != rank)
            send_map(tc::smem_u32(&x.at(k, rank, lane)), tc::smem_u32(&x.bar[b]), r, m);
}

// A tensor map of [T][C] rows in boxes of kGatedChunk x kGatedCh.
struct alignas(64) GatedMap {
    unsigned char image[128];
};

// The first 128-byte boundary of the dynamic shared memory (TMA's destination).
__device__ __forceinline__ unsigned char *align128(unsigned char *p) { return p + (-tc::smem_u32(p) & 127u); }

// TMA: the box at channel c, token t into shared memory (zeros outside the tensor).
__device__ __forceinline__ void tma_rows(void *dst, const GatedMap *map, int c, int t, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];\n"
                 ::"r"(tc::smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(t), "r"(tc::smem_u32(bar))
                 : "memory");
}

// Round k's maps of the other blocks are here.
__device__ __forceinline__ bool exchange_wait(const GatedExchange &x, int k, int cap)
{
    return gated_wait(&x.bar[k % kGatedBufs], (k / kGatedBufs) & 1, cap);
}

// Short sequences (16 tokens or fewer on average): a thread steps through the tokens of
// one sequence for two channels, both ways; no chunk is shared.  A block of the walk
// spends 4 us before its first result: 256 sequences of 8 tokens, 2048 channels, us:
// forward 73 with the walk, 11 stepping; backward 132, 39.
inline bool gated_short(const GatedArgs &a) { return (long long)a.n_tokens <= 16LL * a.n_seqs; }

// Among many short sequences a long one would be stepped by one thread a channel pair, so a
// call of short ones steps those of up to kGatedStep tokens and walks the others, one block
// each for 64 channels, in a launch of its own before it, whose blocks leave if there are
// none.  us with 4096 channels, bf16, forward / backward, everything stepped against this:
//   255 x 1 and 3800 tokens       2640 / 5390     96 / 296
//   100 x 1 and 64                  26 / 65        9.4 / 20
//   250 x 1 and 50 x 64             64 / 263      61 / 136
//   250 x 1 and 50 x 40             35 / 166      55 / 124   (512 channels: 16 / 36, 16 / 32)
//   256 x 8                         20.5 / 116    21.5 / 126
//   64 x 4                           5.2 / 13.5    6.4 / 14.7
// (limits of 64 and 16 tokens instead of 32: 26 / 60 for the second line, 52 / 108 against
// 19 / 84 for 250 x 1 and 50 x 20.)  Not with 128 tokens or fewer, the longest of which
// costs 48 / 115 us stepped, where the launch would cost every call its share (10 x 10:
// 5.4 / 10.8 against 6.7 / 12.9); nor with as many tokens as sequences, a decode step as in
// ssm_scan (other lengths are right there too, stepped).
constexpr int kGatedStep = 32;
inline bool gated_mixed(const GatedArgs &a) { return a.n_tokens > 4 * kGatedStep && a.n_tokens != a.n_seqs; }
// Blocks of that launch: two an SM where there can be work for four, else one (256 x 8 tokens
// of 512 channels, no long one: 6.4 us against 9.5; 600 x 1 and 100 x 100 of 4096: 310 against 169).
inline unsigned gated_mixed_blocks(const GatedArgs &a)
{
    const long long most = (long long)(a.n_tokens / (kGatedStep + 1)) * a.cblocks;
    return (unsigned)(most < kSms ? most : most < 4 * kSms ? kSms : 2 * kSms);
}

// Two neighbouring elements of a row in global memory (`pairs`: one access).
template <class T>
__device__ __forceinline__ float2 global_pair(const void *base, long long at, bool pairs, bool two)
{
    const T *p = static_cast<const T *>(base) + at;
    if (pairs) {
        const Vec<T, 2> v = load_vec<T, 2>(p);
        return make_float2(to_float(v.v[0]), to_float(v.v[1]));
    }
    return make_float2(to_float(p[0]), two ? to_float(p[1]) : 0.f);
}

// Host side.
long long gated_chunk_rows(long long n_seqs, long long n_tokens);
// Blocks of a cluster for these sizes (gated_scan.cu); wide: the forward kernel on fp32.
int gated_cluster(int n_seqs, int n_tokens, int C, bool wide);
// False where TMA cannot describe the rows (address or stride no multiple of 16 bytes).
bool gated_map(GatedMap *map, const void *p, int dtype, int n_tokens, int C, long long stride);
// Whether 4-byte copies of a tensor's rows are aligned (its pairs, for 16-bit types).
bool gated_words(const void *p, int dtype, int C, long long stride);
cudaError_t launch_gated_scan(GatedArgs a, int dtype, cudaStream_t stream);
cudaError_t launch_gated_scan_backward(GatedArgs a, int dtype, cudaStream_t stream);

// Blocks of a walk over every sequence.
inline unsigned gated_walk_blocks(const GatedArgs &a) { return (unsigned)((long long)a.n_seqs * a.cblocks * a.cluster); }

// `kernel` over `blocks` blocks in clusters of a.cluster.
template <class... KArgs, class... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), const GatedArgs &a, unsigned blocks, int warps, size_t smem,
                            cudaStream_t stream, Args &&...args)
{
    cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace ssm
