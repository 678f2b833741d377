/*
 * ssmscan.h -- C ABI of libssmscan, the Mamba2 selective-state scan on sm_103a.
 *
 * The operation (for every sequence i, head h, head-dim row p and token t of
 * the sequence, in token order; g(h) = h / (n_heads / n_groups)):
 *
 *     dA          = exp(dt[t,h] * A[h])
 *     S[h,p,:]    = dA * S[h,p,:] + dt[t,h] * x[t,h,p] * B[t,g(h),:]
 *     y[t,h,p]    = S[h,p,:] . C[t,g(h),:] + D[h] * x[t,h,p]
 *
 * S is the fp32 recurrent state of sequence i.  It lives in slot i of
 * state_slots and persists between calls.  Defined by:
 *   - "The llama journey", Day 14: the ssm_scan_f32_group kernel body (decay
 *     exp(dt*A) with a scalar A per head, input term B*x*dt, y = state . C
 *     from the state that already includes token t, one B/C per group of
 *     contiguous heads);
 *   - "The llama journey", Day 12: the SSM_SCAN tensor table (state
 *     [seq][head][dim][d_state]; x [token][head][dim]; dt [token][head];
 *     B, C [token][group][d_state]);
 *   - "keep the Mamba2 scan state in registers, stage tokens by chunk"
 *     (gllm PR 90), "What changes" and "Testing": batches mix fresh and
 *     resuming sequences; state is fp32 and moves between slot and registers.
 * The skip term D[h] * x[t,h,p] is part of the operation.  dt is used as given
 * (no softplus or bias is applied here).
 *
 * Memory and ownership (all calls):
 *   - Every pointer is CUDA device memory owned by the caller.  The library
 *     allocates nothing and never synchronises the stream; work is enqueued on
 *     `stream` (a cudaStream_t passed as void*; NULL = the legacy default
 *     stream) and its execution errors surface at the caller's next sync.
 *   - Tokens of all sequences are packed: sequence i owns tokens
 *     [seq_starts[i], seq_starts[i] + seq_lens[i]) of the n_tokens rows of
 *     x, dt, B, C and y.  Tokens owned by no sequence are neither read nor
 *     written.
 *   - resume_flags[i] != 0: start from slot i.  == 0: start from zero; the
 *     slot's old contents are never read (they may be NaN).  After the call
 *     slot i holds the state after the sequence's last token.  A zero-length
 *     sequence writes no y; a fresh one still leaves a zero slot.
 *   - Layouts (row-major, contiguous, fp32 unless stated):
 *       state_slots [n_seqs][n_heads][head_dim][d_state]   in/out
 *       x           [n_tokens][n_heads][head_dim]
 *       dt          [n_tokens][n_heads]
 *       A, D        [n_heads]
 *       B, C        [n_tokens][n_groups][d_state]
 *       y           [n_tokens][n_heads][head_dim]               out
 *       seq_starts, seq_lens, resume_flags   int32 [n_seqs], device memory
 *   - y must not overlap any input; inputs are read only.
 *   - Alignment: state_slots, B and C 16-byte aligned (the state moves as
 *     128-bit vectors); the others 4-byte aligned.
 *
 * Preconditions checked only on the device metadata's request: sequence
 * ranges must lie in [0, n_tokens) and not overlap.  With the environment
 * variable SSM_SCAN_CHECK=1 the library copies the metadata to the host,
 * synchronises and rejects bad ranges with SSM_ERR_INVALID_ARG (debug only).
 *
 * Errors: host-checkable faults return before any launch:
 *   SSM_ERR_INVALID_ARG  null pointer, negative size, n_heads % n_groups != 0,
 *                        misaligned pointer, bad tuning value;
 *   SSM_ERR_UNSUPPORTED  d_state not a multiple of 4, d_state > 1024;
 *   SSM_ERR_CUDA         a CUDA call or launch failed (cudaGetLastError);
 *   SSM_ERR_TIMEOUT      a bounded device wait gave up (the pipelined
 *                        tensor-core kernels: the segments' state pass and the
 *                        SSD chunk-state and output kernels).  Each such wait
 *                        polls an mbarrier a bounded number of times (seconds);
 *                        on giving up the kernel sets a status word in the
 *                        workspace, waits for its copies and products in
 *                        flight, frees its tensor memory and returns, so the
 *                        context stays usable.  The word is read back (and this
 *                        code returned) only under SSM_SCAN_CHECK=1; the library
 *                        never synchronises otherwise.  Without that check the
 *                        failure shows in the outputs instead:
 *                          - a segmented ssm_scan_* call: y is NaN for every
 *                            owned token and every slot keeps the contents it
 *                            had before the call;
 *                          - ssm_scan_ssd: when the chunk states gave up, y is
 *                            NaN for every owned token and the slots keep their
 *                            contents; when an output block gave up, y is NaN
 *                            over that block's chunk and heads (the slots hold
 *                            the final states).
 *                        SSM_SCAN_TEST_FAIL_WAITS=1 makes those waits give up
 *                        at once (tests of this path).
 * n_seqs == 0 is a successful no-op.
 */
#ifndef SSMSCAN_H
#define SSMSCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SSM_OK = 0,
    SSM_ERR_INVALID_ARG = -1,
    SSM_ERR_UNSUPPORTED = -2,
    SSM_ERR_CUDA = -3,
    SSM_ERR_TIMEOUT = -4
} ssm_status;

/* Kernel path selection for ssm_scan_tuned. */
enum {
    SSM_PATH_AUTO = 0,           /* decode when n_tokens == n_seqs, else prefill */
    SSM_PATH_DECODE = 1,         /* warp-per-row kernel; correct for any lengths */
    SSM_PATH_PREFILL = 2,        /* chunk-staged kernel, decay-rescaled state with packed
                                    fp32x2 FMAs; correct for any lengths */
    SSM_PATH_PREFILL_DIRECT = 3  /* chunk-staged kernel stepping S itself (one multiply
                                    more per state element); correct for any lengths */
};

/*
 * Launch-shape overrides for ssm_scan_tuned.  Zero in any field means "pick
 * automatically".  Every combination that is accepted computes the same
 * result (up to float association); unsupported values give
 * SSM_ERR_INVALID_ARG.
 *   path             SSM_PATH_*
 *   lanes_per_row    lanes of a warp that share one state row: 1,2,4,8,16,32
 *   rows_per_thread  state rows each lane holds (a power of two, <= lanes_per_row:
 *                    up to 8 on SSM_PATH_PREFILL, up to 4 on the other paths;
 *                    automatic on SSM_PATH_PREFILL: about 16 state elements of a
 *                    row per lane and 4 rows)
 *   rows_per_cta     prefill: state rows per thread block (a multiple of the
 *                    rows one warp holds, at most 256 threads, 224 on
 *                    SSM_PATH_PREFILL, whose blocks add a producer warp except
 *                    where they are exactly four warps of 8 lanes x 4 rows: those
 *                    stage their own chunks, three blocks per SM); decode: ignored
 *   chunk_tokens     prefill: tokens staged in shared memory per chunk (1..256;
 *                    at most 32 on SSM_PATH_PREFILL, automatic 16 there, 32 on
 *                    SSM_PATH_PREFILL_DIRECT)
 *   ctas_per_sm      decode: if > 0, the grid is capped at this many blocks
 *                    per SM and warps loop over the remaining rows
 *   segment_tokens   SSM_PATH_PREFILL with a workspace (ssm_scan_ws): length of
 *                    the time segments long sequences are cut into (a multiple
 *                    of the chunk; an automatic chunk is the largest of 16, 8,
 *                    ... that divides it); 0 = automatic, < 0 = never segment
 *   segment_state    how the state pass of the time segments runs
 *                    (SSM_SEGMENT_STATE_*); ignored without segments
 */
enum {
    SSM_SEGMENT_STATE_AUTO = 0,   /* the tensor cores where d_state <= 128, head_dim <= 256 and
                                     a multiple of 4, and x 16-byte aligned; else the sequential
                                     kernel */
    SSM_SEGMENT_STATE_FP32 = 1,   /* the sequential kernel's state-only mode (fp32 FMAs) */
    SSM_SEGMENT_STATE_TENSOR = 2  /* the segment's state as a matrix product over its tokens on
                                     the tensor cores, operands split into two TF32 parts
                                     (hi*hi + hi*lo + lo*hi, fp32 accumulation: fp32-level
                                     accuracy); SSM_ERR_UNSUPPORTED where the shapes do not fit */
};
typedef struct {
    int path;
    int lanes_per_row;
    int rows_per_thread;
    int rows_per_cta;
    int chunk_tokens;
    int ctas_per_sm;
    int segment_tokens;
    int segment_state;
} ssm_scan_tuning;

/*
 * The scan.  Advances every sequence of the batch through its tokens, writes
 * y for each of them and leaves each sequence's final state in its slot.
 * n_tokens is the number of packed token rows of x, dt, B, C and y.
 */
int ssm_scan(float *state_slots, const float *x, const float *dt,
             const float *A, const float *B, const float *C, const float *D,
             float *y, const int32_t *seq_starts, const int32_t *seq_lens,
             const int32_t *resume_flags, int n_seqs, int n_tokens,
             int n_heads, int head_dim, int d_state, int n_groups,
             void *stream);

/* The same operation with explicit launch-shape choices (tests, tuning). */
int ssm_scan_tuned(float *state_slots, const float *x, const float *dt,
                   const float *A, const float *B, const float *C,
                   const float *D, float *y, const int32_t *seq_starts,
                   const int32_t *seq_lens, const int32_t *resume_flags,
                   int n_seqs, int n_tokens, int n_heads, int head_dim,
                   int d_state, int n_groups, const ssm_scan_tuning *tuning,
                   void *stream);

/*
 * Optional steps around the scan (all NULL / 0 = the plain scan).
 *   dt_bias, dt_softplus  Mamba2's discretisation of dt ("The llama journey",
 *       Day 14 kernel body; the decay-gate kernel of "ssm_gated_delta.cu"):
 *       v = dt[t,h] + dt_bias[h] (dt_bias NULL: no bias), then with dt_softplus
 *       nonzero the step is v for v > 20 and log1p(exp(v)) otherwise; that step
 *       replaces dt[t,h] everywhere in the recurrence above.  It is computed by
 *       a pass of its own into the first n_tokens*n_heads floats (rounded up to
 *       256 bytes) of the workspace, so these options need a workspace (see
 *       ssm_scan_ex_workspace_bytes); the scan kernels then read it as their
 *       step.  dt_bias: device, [n_heads] fp32, 4-byte aligned.
 *   state_snapshots  device, [n_tokens][n_heads][head_dim][d_state] fp32, out:
 *       row t receives the state right after token t for every token owned by a
 *       sequence, so accepting the first M tokens of a speculative run restores
 *       one contiguous [n_heads][head_dim][d_state] image (the rows of tokens
 *       owned by no sequence are not written).  16-byte aligned.
 *   gated_y, gate_z, norm_weight, norm_eps  Mamba2's gated RMSNorm after the
 *       scan, per (token, head) row of head_dim values:
 *       gated_y[t,h,p] = y[t,h,p] / sqrt(mean_p(y[t,h,:]^2) + norm_eps)
 *                        * norm_weight[p] * silu(gate_z[t,h,p]),
 *       silu(z) = z / (1 + exp(-z)), the weight shared by all heads (kernel 3
 *       of "ssm_gated_delta.cu").  gated_y, gate_z: device [n_tokens][n_heads]
 *       [head_dim] fp32; norm_weight: device [head_dim]; norm_eps > 0.  y is
 *       still written.  gated_y NULL: off (the other three are then ignored).
 *   launch_events, n_launch_events  timing of the call's kernels: an array of
 *       n_launch_events CUDA events (cudaEvent_t handles the caller created on
 *       the stream's device).  The call records launch_events[2k] on its stream
 *       right before its k-th kernel launch and launch_events[2k+1] right
 *       after it, while 2k+1 < n_launch_events, so cudaEventElapsedTime of a
 *       pair is that kernel's device time.  Launch order: the dt pass (with
 *       the dt options); then for ssm_scan_* the decode kernel, or the prefill
 *       kernel, or with time segments the plan, state-pass, combine and
 *       full-pass kernels; for ssm_scan_ssd the plan, chunk-state, state-pass
 *       and output kernels; then the gated RMSNorm (with gated_y), except
 *       where the rescaled prefill's last kernel writes it itself (its blocks
 *       then hold exactly one head each, as the automatic shape does at
 *       head_dim 64 and d_state 64 or 128, and z is 16-byte aligned).  NULL / 0:
 *       none; n_launch_events < 0, or > 0 with NULL events: SSM_ERR_INVALID_ARG;
 *       a failed record: SSM_ERR_CUDA.
 */
typedef struct {
    const float *dt_bias;
    int dt_softplus;
    float *state_snapshots;
    const float *gate_z;
    const float *norm_weight;
    float norm_eps;
    float *gated_y;
    void *const *launch_events;
    int n_launch_events;
} ssm_scan_options;

/*
 * The scan with tuning, options and workspace (each may be NULL / 0):
 * ssm_scan_ws plus the optional steps of ssm_scan_options.  With state
 * snapshots the call runs the decode kernel whatever the lengths (it steps
 * each sequence token by token with the state in registers and writes every
 * intermediate state; meant for the few tokens of a speculative verify step);
 * a tuning that asks for a prefill path then returns SSM_ERR_UNSUPPORTED.
 * Errors as for ssm_scan_ws, and SSM_ERR_INVALID_ARG for a misaligned option
 * pointer, norm_eps <= 0 with gated_y set, or dt options without a workspace
 * of at least the discretised step's bytes.  The workspace is used as by
 * ssm_scan_ws after that step's bytes.
 */
int ssm_scan_ex(float *state_slots, const float *x, const float *dt,
                const float *A, const float *B, const float *C, const float *D,
                float *y, const int32_t *seq_starts, const int32_t *seq_lens,
                const int32_t *resume_flags, int n_seqs, int n_tokens,
                int n_heads, int head_dim, int d_state, int n_groups,
                const ssm_scan_tuning *tuning, const ssm_scan_options *options,
                void *workspace, size_t workspace_bytes, void *stream);

/*
 * The scan with a caller-owned device workspace.  With a workspace the
 * prefill path may cut long sequences into time segments and run them in
 * parallel: a state-only pass per segment, a combine of the segment states
 * (S_in[k+1] = d_k S_in[k] + L_k, d_k the segment's decay prod exp(dt*A)),
 * then the full pass from each segment's incoming state.  This is the same
 * recurrence applied to whole segments; only float association changes.  The
 * state pass runs on the tensor cores where the shapes fit (see
 * tuning->segment_state): L_k unrolled into a sum over the segment's tokens,
 * sum_s dt_s exp(A sum_{r>s} dt_r) x_s B_s^T, with split TF32 operands.
 *   tuning          may be NULL
 *   workspace       device memory, 256-byte aligned, at least
 *                   ssm_scan_workspace_bytes(...) bytes for the same arguments
 *                   and tuning; NULL or too small: runs without segments
 *                   (SSM_ERR_INVALID_ARG if tuning->segment_tokens > 0)
 * The workspace is scratch: its contents are undefined afterwards and two
 * calls that overlap on the GPU must not share it.
 */
int ssm_scan_ws(float *state_slots, const float *x, const float *dt,
                const float *A, const float *B, const float *C, const float *D,
                float *y, const int32_t *seq_starts, const int32_t *seq_lens,
                const int32_t *resume_flags, int n_seqs, int n_tokens,
                int n_heads, int head_dim, int d_state, int n_groups,
                const ssm_scan_tuning *tuning, void *workspace,
                size_t workspace_bytes, void *stream);

/*
 * Bytes of workspace ssm_scan_ws uses for these sizes and tuning (NULL =
 * automatic) on the current device; 0 when it would not cut any sequence into
 * segments (for example decode batches) or the arguments are invalid.
 */
size_t ssm_scan_workspace_bytes(int n_seqs, int n_tokens, int n_heads,
                                int head_dim, int d_state, int n_groups,
                                const ssm_scan_tuning *tuning);

/*
 * The scan in chunked matrix form ("SSD") on the TF32 tensor cores.  The
 * gllm PR 90 page ("keep the Mamba2 scan state in registers, stage tokens by
 * chunk", "What changes" and "Not in this PR") names Mamba2's SSD
 * chunked-matmul algorithm as the way to parallelise prefill over time and
 * gives no algorithm; this form is the recurrence above unrolled over chunks
 * of `chunk` tokens of each sequence.  With a_t = sum_{s<=t in the chunk}
 * dt[s,h] A[h]:
 *     y_t   = exp(a_t) S_in.C_t + sum_{s<=t} exp(a_t - a_s) dt_s (C_t.B_s) x_s + D x_t
 *     S_out = exp(a_last) S_in + sum_s exp(a_last - a_s) dt_s x_s (x) B_s
 * and S_in of chunk k+1 is S_out of chunk k.  In exact arithmetic it equals
 * ssm_scan.  The contractions C B^T, (masked decay-weighted C B^T) x, S_in C^T
 * and x^T B round their operands to TF32 (10-bit mantissa, round to nearest)
 * and accumulate in fp32; the pass over chunks is fp32.  Expect
 * |y - y_exact| <= 5e-3 (1 + |y_exact|), not the 1e-4 of ssm_scan.
 *   chunk         tokens per chunk: 64 or 128 (0 = 128)
 *   workspace     device memory, 256-byte aligned, at least
 *                 ssm_scan_ssd_workspace_bytes(...) bytes for the same sizes
 *                 and chunk (chunk states [units][n_heads][head_dim][d_state]
 *                 fp32, units <= n_seqs + ceil(n_tokens / chunk), and room for
 *                 the discretised step of the dt options); scratch:
 *                 undefined afterwards, not shared by calls that overlap on
 *                 the GPU
 * Same arguments, layouts and metadata rules as ssm_scan, and also:
 *   - x and y 16-byte aligned;
 *   - head_dim a multiple of 16 and at most 128 (else SSM_ERR_UNSUPPORTED);
 *   - the chunk's shared-memory tiles must fit one block: SSM_ERR_UNSUPPORTED
 *     otherwise (for example d_state 1024; d_state up to 256 fits with
 *     chunk 64, up to 128 with chunk 128).
 * options: as for ssm_scan_ex (NULL = none); state snapshots are not
 * available in this form (SSM_ERR_UNSUPPORTED).
 * SSM_ERR_INVALID_ARG for a missing, misaligned or too small workspace or a
 * chunk other than 0, 64 or 128.
 */
int ssm_scan_ssd(float *state_slots, const float *x, const float *dt,
                 const float *A, const float *B, const float *C, const float *D,
                 float *y, const int32_t *seq_starts, const int32_t *seq_lens,
                 const int32_t *resume_flags, int n_seqs, int n_tokens,
                 int n_heads, int head_dim, int d_state, int n_groups,
                 int chunk, const ssm_scan_options *options, void *workspace,
                 size_t workspace_bytes, void *stream);

/*
 * Bytes of workspace ssm_scan_ex uses for these sizes, tuning and options
 * (NULL = none): the discretised step when dt options are set, plus what
 * ssm_scan_workspace_bytes reports (nothing with state snapshots); 0 for
 * invalid arguments or when none is needed.
 */
size_t ssm_scan_ex_workspace_bytes(int n_seqs, int n_tokens, int n_heads,
                                   int head_dim, int d_state, int n_groups,
                                   const ssm_scan_tuning *tuning,
                                   const ssm_scan_options *options);

/*
 * Bytes of workspace ssm_scan_ssd needs for these sizes and chunk (the same on
 * every device); 0 for invalid or unsupported arguments.
 */
size_t ssm_scan_ssd_workspace_bytes(int n_seqs, int n_tokens, int n_heads,
                                    int head_dim, int d_state, int n_groups,
                                    int chunk);

/*
 * Size of the scratch that ssm_scan_static keeps in device memory (32 MiB per
 * device, held from the library's load on that device until process exit).
 */
#define SSM_SCAN_STATIC_SCRATCH_BYTES (32u << 20)

/*
 * The scan for callers that cannot allocate device memory (the pages have no
 * counterpart: it is a packaging choice of this library).  Some callers never
 * get to hand the library a workspace: a runtime without a device allocator,
 * a plugin whose host owns every allocation, a path that must not enter
 * cudaMalloc.  ssm_scan_static takes the same arguments as ssm_scan and runs
 * what ssm_scan_ws runs with an automatic plan, using instead a fixed scratch
 * array of SSM_SCAN_STATIC_SCRATCH_BYTES in device global memory that the
 * library owns.  It allocates nothing.
 *   - The first call on a device looks up the scratch's device address (a
 *     cudaGetSymbolAddress with that device current) and caches it; make that
 *     first call before any stream capture.  The cached address belongs to
 *     the device's context as it was then: a cudaDeviceReset while the
 *     library is loaded is not supported.
 *   - The stream must belong to the current device (SSM_ERR_INVALID_ARG
 *     otherwise), since the scratch address is looked up for that device.
 *   - When the automatic plan's segment states would not fit the scratch
 *     (very long or many long sequences, large states), the call runs with
 *     longer time segments (1024 tokens, doubled until they fit) or without
 *     segments (also when no such segment would be shorter than the longest
 *     sequence can be): the same results, less parallelism than ssm_scan_ws
 *     with a workspace of the size ssm_scan_workspace_bytes asks for.
 *   - Every call in the process shares the scratch, which keeps the last
 *     call's contents (nothing in it needs to start at zero).  Calls whose GPU
 *     work overlaps, on two streams or from two threads, race on it: the
 *     caller must serialise them.
 * Errors otherwise as for ssm_scan.
 */
int ssm_scan_static(float *state_slots, const float *x, const float *dt,
                    const float *A, const float *B, const float *C,
                    const float *D, float *y, const int32_t *seq_starts,
                    const int32_t *seq_lens, const int32_t *resume_flags,
                    int n_seqs, int n_tokens, int n_heads, int head_dim,
                    int d_state, int n_groups, void *stream);

/*
 * Causal depthwise conv1d + SiLU with a rolling conv-state slot, Mamba2's op in
 * front of the scan ("ssm_gated_delta.cu", kernel 2 and its batched variant;
 * the pages' kernel has no bias, the optional bias here is added before SiLU).
 * For sequence i (tokens packed as for ssm_scan) and channel c, the stream of
 * inputs is the slot's kernel_size-1 remembered inputs (oldest first; zeros
 * when resume_flags[i] == 0) followed by the sequence's tokens, and
 *     out[t, c] = silu(bias[c] + sum_{u < K} weight[c, u] * stream[t + u]),
 * silu(v) = v / (1 + exp(-v)), with stream[K-1+t] = x[t, c] (so weight[c, K-1]
 * multiplies the current token).  Afterwards slot i holds the stream's last
 * K-1 entries, and snapshot row t (optional) the slot image right after
 * token t.
 *   x, out      [n_tokens][channels] fp32, device (out written for owned tokens)
 *   weight      [channels][kernel_size] fp32, device
 *   bias        [channels] fp32, device, or NULL
 *   conv_state  [n_seqs][channels][kernel_size-1] fp32, device, in/out
 *   snapshots   [n_tokens][channels][kernel_size-1] fp32, device, or NULL
 *   kernel_size 1 .. 8
 * Ownership, metadata, stream and 4-byte alignment rules as for ssm_scan.
 * Errors: SSM_ERR_INVALID_ARG (sizes, NULL or misaligned pointers),
 * SSM_ERR_UNSUPPORTED (n_tokens * channels above 2^31), SSM_ERR_CUDA.
 */
int ssm_conv1d(const float *x, const float *weight, const float *bias,
               float *conv_state, float *out, const int32_t *seq_starts,
               const int32_t *seq_lens, const int32_t *resume_flags,
               int n_seqs, int n_tokens, int channels, int kernel_size,
               float *snapshots, void *stream);

/* Element types of the layer operators below. */
typedef enum {
    SSM_F32 = 0,
    SSM_BF16 = 1,
    SSM_F16 = 2
} ssm_dtype;

/*
 * The layer operators around the scan: a gated linear recurrence per channel
 * (forward, backward), the RMS norm with the residual's addition (forward,
 * 8-bit output, backward), a row quantiser and the 8-bit integer matrix product
 * that reads the codes.  Ownership, stream and error rules are those of
 * ssm_scan: caller-owned device memory, nothing allocated, nothing
 * synchronised, host-checkable faults return before any launch.  Rows are
 * contiguous and `..._stride` is the distance of two rows in elements (at least
 * the row's length), so x and the gates may be slices of one projection.
 * Sums, states, norms and statistics are held in fp32 or exact integers; a
 * result is rounded to its type once.
 */

/*
 * Gated linear recurrence.  For token t of a sequence and channel c:
 *     r = sigmoid(gate_a[t,c]),  i = sigmoid(gate_x[t,c])
 *     log a = -decay_scale * softplus(lam[c]) * r,  a = exp(log a)
 *     h_t = a h_{t-1} + sqrt(1 - a^2) i x[t,c],  y[t,c] = h_t
 * at every token.  (Some models take i x[t,c] without the root at the first token of
 * a fresh sequence; there is no flag for that.)  h is the fp32 state of the
 * sequence's slot; packed tokens, seq_starts, seq_lens and resume_flags as for
 * ssm_scan (a fresh sequence never reads its slot; a zero-length one leaves zeros
 * if fresh and its slot if resuming).  A
 * sequence whose range is not inside [0, n_tokens) counts as empty; ranges that
 * overlap are not supported (SSM_SCAN_CHECK=1 reports both).
 *   state_slots  [n_seqs][channels] fp32, in/out
 *   x, gate_a, gate_x, y   [n_tokens][channels] of `dtype` (ssm_dtype)
 *   lam          [channels] fp32;  decay_scale > 0 and finite
 *   chunk_states NULL, or (training) fp32 [ssm_gated_scan_chunks(...)][channels],
 *                out: the state entering each time chunk, which the backward
 *                pass reads
 * With 16 tokens a sequence or fewer on average (decode: one each) the call steps
 * the sequences token by token, but for those of more than 32 tokens in a call of
 * more than 128 tokens whose number is not that of the sequences; otherwise, and
 * for those, blocks walk a sequence's time chunks, with the time of a sequence
 * shared by a cluster of blocks where there are few sequences and channels.  One
 * launch (two for a call that may have both), no workspace, the same bits every
 * time.  The cluster's waits are bounded: on giving up y and the slots
 * behind it become NaN (and a block's y up to two rounds of chunks before it).
 * y must not overlap an input.
 * Errors: SSM_ERR_INVALID_ARG (sizes, NULL or misaligned pointers, strides
 * below channels), SSM_ERR_UNSUPPORTED (more than 2^28 (sequence, 64 channels)
 * pairs or 2^31 - 513 tokens), SSM_ERR_CUDA.
 */
int ssm_gated_scan(float *state_slots, const void *x, const void *gate_a, const void *gate_x, const float *lam,
                   float decay_scale, void *y, const int32_t *seq_starts, const int32_t *seq_lens,
                   const int32_t *resume_flags, int n_seqs, int n_tokens, int channels, int dtype,
                   long long x_stride, long long gate_a_stride, long long gate_x_stride, long long y_stride,
                   float *chunk_states, void *stream);

/* Rows of chunk_states for these sizes; 0 for invalid or unsupported ones. */
long long ssm_gated_scan_chunks(int n_seqs, int n_tokens, int channels);

/*
 * Gradients of ssm_gated_scan.  Takes the forward call's inputs, metadata and
 * chunk_states, the gradient of y (grad_y) and optionally of the slots after
 * the call (grad_state [n_seqs][channels] fp32 or NULL), and writes
 *   grad_x, grad_gate_a, grad_gate_x   [n_tokens][channels] of dtype (tokens
 *                owned by no sequence are not written)
 *   grad_lam     [channels] fp32, summed in a fixed order (the same bits every
 *                time; zeros when n_seqs is 0)
 *   grad_initial_state  [n_seqs][channels] fp32 or NULL: gradient of the slots
 *                before the call (zeros for fresh sequences)
 * h is recomputed in fp32 from chunk_states.  workspace: 256-byte aligned, at
 * least ssm_gated_scan_backward_workspace_bytes(...); scratch, not shared by
 * calls that overlap on the GPU.
 */
int ssm_gated_scan_backward(const void *grad_y, const float *grad_state, const void *x, const void *gate_a,
                            const void *gate_x, const float *lam, float decay_scale, const float *chunk_states,
                            const int32_t *seq_starts, const int32_t *seq_lens, const int32_t *resume_flags,
                            int n_seqs, int n_tokens, int channels, int dtype, long long x_stride,
                            long long gate_a_stride, long long gate_x_stride, long long grad_y_stride,
                            void *grad_x, void *grad_gate_a, void *grad_gate_x, long long grad_x_stride,
                            long long grad_gate_a_stride, long long grad_gate_x_stride, float *grad_lam,
                            float *grad_initial_state, void *workspace, size_t workspace_bytes, void *stream);

size_t ssm_gated_scan_backward_workspace_bytes(int n_seqs, int n_tokens, int channels);

/*
 * RMS norm with the residual's addition, per row of `width` elements:
 *     h = x + residual, rounded to residual_dtype (written to residual_out)
 *     inv = 1 / sqrt(mean(h^2) + eps),  y = h * inv * weight
 * or, with codes and scales instead of y, in 8 bits:
 *     v = h * weight,  f = min(127 / max|v|, FLT_MAX),  both in fp32
 *     codes = rint(v * f) (half to even),  scales = inv / f
 * so codes * scales is y to half a step of its row's largest value / 127.  The
 * codes do not depend on inv, nor on any order of summation.  A row of zeros
 * has codes 0; a row with a NaN or an infinity (in h or in v) has scale NaN.
 *   x, y          [rows][width] of dtype;  weight [width] fp32
 *   residual      [rows][width] of residual_dtype (dtype or SSM_F32), or NULL:
 *                 h = x
 *   residual_out  as residual, or NULL: not written; may be residual itself
 *                 (same stride), else it must not overlap an input
 *   y or codes (int8) with scales [rows] fp32: exactly one of the two outputs;
 *                 out_stride is y's or codes'
 * eps >= 0; width at most 16384 (SSM_ERR_UNSUPPORTED above).
 */
int ssm_add_norm(const void *x, const void *residual, const float *weight, float eps, void *residual_out, void *y,
                 int8_t *codes, float *scales, int rows, int width, int dtype, int residual_dtype,
                 long long x_stride, long long residual_stride, long long residual_out_stride, long long out_stride,
                 void *stream);

/*
 * Gradient of ssm_add_norm's y and residual_out.  With n = h * inv:
 *     grad_in = grad_h + inv * (weight * grad_y - n * mean(n * weight * grad_y))
 *     grad_weight = sum over rows of grad_y * n
 * grad_in (residual_dtype) is the gradient of x and of residual alike.
 *   grad_y [rows][width] of dtype; h as written by the forward call; grad_h as
 *   h: the gradient that reaches residual_out from elsewhere, or NULL
 *   grad_weight [width] fp32, summed in a fixed order
 *   grad_in may be grad_h itself (same stride)
 * workspace: 256-byte aligned, ssm_add_norm_backward_workspace_bytes(...).
 */
int ssm_add_norm_backward(const void *grad_y, const void *h, const float *weight, float eps, const void *grad_h,
                          void *grad_in, float *grad_weight, int rows, int width, int dtype, int residual_dtype,
                          long long grad_y_stride, long long h_stride, long long grad_h_stride,
                          long long grad_in_stride, void *workspace, size_t workspace_bytes, void *stream);

size_t ssm_add_norm_backward_workspace_bytes(int rows, int width);

/*
 * Rows in 8 bits with a scale each (activations in front of a projection,
 * weights once when they are loaded): f = min(127 / max|x|, FLT_MAX),
 * codes = rint(x * f), scales = 1 / f; zeros, NaN and infinities as above.
 */
int ssm_quantize_rows(const void *x, int8_t *codes, float *scales, int rows, int width, int dtype,
                      long long x_stride, long long codes_stride, void *stream);

/*
 * 8-bit integer matrix product with a scale for each token and each output
 * channel:
 *     out[t][n] = (sum_k x[t][k] * w[n][k]) * x_scales[t] * w_scales[n] + bias[n]
 *   x  [rows][inner] int8, w [out_features][inner] int8 (any value, -128 too)
 *   x_scales [rows], w_scales [out_features], bias [out_features] or NULL: fp32
 *   out [rows][out_features] of out_dtype
 * The sum is the exact integer, rounded once to fp32 (inner at most 131071;
 * SSM_ERR_UNSUPPORTED above, as for more than 2^31 - 257 rows or channels); the
 * scales and the bias are applied in fp32.
 * workspace: 256-byte aligned, at least ssm_int8_matmul_workspace_bytes(...)
 * of the same operands, sizes and strides (0: none is needed); scratch, not
 * shared by calls that overlap on the GPU.  It holds the weights if their
 * rows are not 16-byte aligned, and with many tokens (more than 64, or 32 and 8192
 * channels) the tokens as fp16; with few, either operand whose rows are not 16-byte
 * aligned, and both if inner is no multiple of 16.
 * So keep weights in whole, aligned multiples of 16 bytes.
 * The waits of the many-token kernel are bounded; a block that gives up writes NaN.
 */
int ssm_int8_matmul(const int8_t *x, const float *x_scales, const int8_t *w, const float *w_scales, const float *bias,
                    void *out, int rows, int out_features, int inner, int out_dtype, long long x_stride,
                    long long w_stride, long long out_stride, void *workspace, size_t workspace_bytes, void *stream);

size_t ssm_int8_matmul_workspace_bytes(const int8_t *x, const int8_t *w, int rows, int out_features, int inner,
                                       long long x_stride, long long w_stride);

/*
 * Operators that a selective-scan model is trained and served with: the
 * selective scan with a decay for each channel and state, the short causal
 * convolution in front of it, and the cross entropy of a projection onto a large
 * vocabulary.  Rules as for the layer operators above.
 */

/*
 * Selective scan with a decay for each channel and state (ssm_scan has one for
 * each head).  For token t of a sequence, channel c of group g = c / (channels /
 * n_groups) and state n:
 *     v = dt[t,c] + dt_bias[c];  step = v, or with dt_softplus v > 20 ? v : log1p(exp(v))
 *     h[c,n] = exp(step A[c,n]) h[c,n] + step x[t,c] B[t,g,n]
 *     p = sum_n h[c,n] C[t,g,n] + D[c] x[t,c];  y[t,c] = p z[t,c] sigmoid(z[t,c])
 * Packed tokens, seq_starts, seq_lens, resume_flags and slots as for ssm_scan (a
 * fresh sequence never reads its slot; a zero-length one leaves zeros if fresh and
 * its slot if resuming).  A sequence whose range is not inside [0, n_tokens)
 * counts as empty; ranges that overlap are not supported (SSM_SCAN_CHECK=1
 * reports both).
 *   state_slots  [n_seqs][channels][d_state] fp32, in/out
 *   x, dt, y     [n_tokens][channels] of dtype;  z the same, or NULL: y = p
 *   B, C         [n_tokens][n_groups][d_state] of dtype (contiguous within a token)
 *   A            [channels][d_state] fp32, finite;  D, dt_bias [channels] fp32 or NULL (zeros)
 *                (either sign: a decay may grow; one token's exp(step A) is fp32, infinite above step A = 88)
 *   chunk_states NULL, or (training) fp32 [ssm_selective_scan_chunks(...)][channels][d_state],
 *                out: the state entering every 16 tokens, which the backward pass reads
 * d_state 1 .. 128 (SSM_ERR_UNSUPPORTED above).  Where sequences and channels alone
 * do not fill the device, long sequences run as parallel segments, whose states pass
 * through the workspace; the sums depend on the sizes only (the same bits every time).
 * y must not overlap an input.
 * workspace: 256-byte aligned, ssm_selective_scan_workspace_bytes(...) (0: none is
 * needed); scratch, not shared by calls that overlap on the GPU.
 */
int ssm_selective_scan(float *state_slots, const void *x, const void *dt, const float *A, const void *B, const void *C,
                       const float *D, const void *z, const float *dt_bias, int dt_softplus, void *y,
                       const int32_t *seq_starts, const int32_t *seq_lens, const int32_t *resume_flags, int n_seqs,
                       int n_tokens, int channels, int d_state, int n_groups, int dtype, long long x_stride,
                       long long dt_stride, long long B_stride, long long C_stride, long long z_stride,
                       long long y_stride, float *chunk_states, void *workspace, size_t workspace_bytes, void *stream);

size_t ssm_selective_scan_workspace_bytes(int n_seqs, int n_tokens, int channels, int d_state, int n_groups);

/* Rows of chunk_states for these sizes; 0 for invalid ones. */
long long ssm_selective_scan_chunks(int n_seqs, int n_tokens);

/*
 * Gradients of ssm_selective_scan.  Takes the forward call's inputs, metadata and
 * chunk_states, the gradient of y (grad_y) and optionally of the slots after the
 * call (grad_state, or NULL), and writes
 *   grad_x, grad_dt, grad_z   [n_tokens][channels] of dtype, grad_B, grad_C
 *                [n_tokens][n_groups][d_state] of dtype (tokens owned by no
 *                sequence are not written; grad_z with z, else NULL)
 *   grad_A       [channels][d_state], grad_D, grad_dt_bias [channels] fp32 (the last two with
 *                their inputs, else NULL), zeros when n_seqs is 0
 *   grad_initial_state  [n_seqs][channels][d_state] fp32 or NULL: gradient of the slots
 *                before the call (zeros for fresh sequences)
 * Sums over tokens and channels are fp32 in a fixed order.  The states are
 * recomputed from chunk_states.  workspace: as above,
 * ssm_selective_scan_backward_workspace_bytes(...).  Outputs must not overlap inputs.
 */
int ssm_selective_scan_backward(const void *grad_y, const float *grad_state, const void *x, const void *dt,
                                const float *A, const void *B, const void *C, const float *D, const void *z,
                                const float *dt_bias, int dt_softplus, const float *chunk_states,
                                const int32_t *seq_starts, const int32_t *seq_lens, const int32_t *resume_flags,
                                int n_seqs, int n_tokens, int channels, int d_state, int n_groups, int dtype,
                                long long grad_y_stride, long long x_stride, long long dt_stride, long long B_stride,
                                long long C_stride, long long z_stride, void *grad_x, void *grad_dt, float *grad_A,
                                void *grad_B, void *grad_C, float *grad_D, void *grad_z, float *grad_dt_bias,
                                float *grad_initial_state, long long grad_x_stride, long long grad_dt_stride,
                                long long grad_B_stride, long long grad_C_stride, long long grad_z_stride,
                                void *workspace, size_t workspace_bytes, void *stream);

size_t ssm_selective_scan_backward_workspace_bytes(int n_seqs, int n_tokens, int channels, int d_state, int n_groups);

/*
 * Short causal convolution: ssm_conv1d's operation on rows of any of the three
 * types with strides (slices of a projection), with or without SiLU:
 *     v[t,c] = bias[c] + sum_u weight[c,u] stream[t+u,c];  out = silu ? v sigmoid(v) : v
 * where a sequence's stream is its slot's kernel_size - 1 inputs (zeros when fresh)
 * followed by its tokens, and the slot afterwards holds the stream's last
 * kernel_size - 1 entries.
 *   x, out      [n_tokens][channels] of dtype;  weight [channels][kernel_size] fp32
 *   bias        [channels] fp32 or NULL
 *   conv_state  [n_seqs][channels][kernel_size-1] fp32, in/out (NULL allowed for kernel_size 1)
 *   kernel_size 1 .. 8 (SSM_ERR_UNSUPPORTED above)
 * out must not overlap an input.  Fastest with an even number of channels and rows on whole words of two
 * channels (4 bytes for 16-bit types, 8 for fp32).
 */
int ssm_causal_conv(const void *x, const float *weight, const float *bias, float *conv_state, void *out,
                    const int32_t *seq_starts, const int32_t *seq_lens, const int32_t *resume_flags, int n_seqs,
                    int n_tokens, int channels, int kernel_size, int silu, int dtype, long long x_stride,
                    long long out_stride, void *stream);

/*
 * Gradients of ssm_causal_conv.  initial_state: what the slots held before the
 * forward call, with resume_flags; both NULL where every sequence was fresh (one
 * without the other is SSM_ERR_INVALID_ARG, but for kernel_size 1, which has no slots).
 * grad_state: the gradient of the slots after the call, or NULL.
 *   grad_x       [n_tokens][channels] of dtype (tokens owned by no sequence are not written)
 *   grad_weight  [channels][kernel_size], grad_bias [channels] fp32 (with bias, else NULL), summed in a
 *                fixed order; zeros when n_seqs is 0
 *   grad_initial_state  as the slots, or NULL (zeros for fresh sequences)
 * workspace: 256-byte aligned, ssm_causal_conv_backward_workspace_bytes(...).
 */
int ssm_causal_conv_backward(const void *grad_out, const float *grad_state, const void *x, const float *weight,
                             const float *bias, const float *initial_state, const int32_t *seq_starts,
                             const int32_t *seq_lens, const int32_t *resume_flags, int n_seqs, int n_tokens,
                             int channels, int kernel_size, int silu, int dtype, long long grad_out_stride,
                             long long x_stride, void *grad_x, float *grad_weight, float *grad_bias,
                             float *grad_initial_state, long long grad_x_stride, void *workspace,
                             size_t workspace_bytes, void *stream);

size_t ssm_causal_conv_backward_workspace_bytes(int n_seqs, int n_tokens, int channels, int kernel_size);

/*
 * Softmax cross entropy of a projection onto a large vocabulary, without the
 * logits in memory:
 *     l[t,v] = sum_d hidden[t,d] weight[v,d];  lse[t] = log sum_v exp(l[t,v])
 *     loss[t] = lse[t] - l[t,targets[t]]
 * A row whose target is ignore_index has loss and lse 0, takes no work, and nothing that
 * stands in it reaches a result.  A target outside [0, vocab) otherwise makes its row's loss
 * NaN (and in the backward pass grad_hidden of the row and grad_weight).
 *   hidden [rows][width], weight [vocab][width] of dtype: SSM_BF16 or SSM_F16
 *          (SSM_ERR_UNSUPPORTED for SSM_F32, and for width above 65536)
 *   targets [rows] int32, or int64 with targets_64;  loss, lse [rows] fp32
 * Sums are fp32; the tensor cores' truncate (lse of 4096 products of order one a logit: 9e-6 rms, where fp32
 * products rounded to nearest have 4e-7).  workspace: 256-byte aligned,
 * ssm_linear_cross_entropy_workspace_bytes(weight, ..., 0): the rows that count, back to
 * back, the parts of the sums, and the weights if their rows are not 16-byte
 * aligned; scratch, not shared by calls that overlap on the GPU.
 * The waits are bounded; where one gives up, results are NaN.
 */
int ssm_linear_cross_entropy(const void *hidden, const void *weight, const void *targets, int targets_64,
                             long long ignore_index, float *loss, float *lse, int rows, int vocab, int width, int dtype,
                             long long hidden_stride, long long weight_stride, void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * Gradients of ssm_linear_cross_entropy's loss: with G[t,v] = (exp(l[t,v] - lse[t]) -
 * [v = targets[t]]) grad_loss[t],
 *     grad_hidden = G weight (zeros for ignored rows),   grad_weight = G^T hidden
 * both in dtype.  lse as the forward call wrote it; its own gradient is not
 * taken.  The logits are recomputed in pieces of the vocabulary; G of a piece is held
 * in dtype relative to the largest finite |grad_loss| (fp16: times 2^15), so each of its terms is rounded
 * to half a step before the products (fp16: terms below 2^-29 of the largest |grad_loss| to 2^-40 of it, which is all of a
 * row whose grad_loss is that much smaller); the sums are fp32 and rounded once.  A grad_loss that is infinite or
 * NaN reaches its own row of grad_hidden, and grad_weight.
 * grad_weight may be NULL (a frozen projection): it is not computed.  Outputs must not overlap
 * inputs.  Where there are few rows, several pairs of SMs share the terms of grad_hidden; the
 * order of its sum depends on the sizes and on how many rows count, not on the run.
 * workspace: as above with backward = 1: also one piece of G (256 MB, or for large calls 16 bytes an
 * element of hidden) and, where there are several, grad_hidden in fp32.
 */
int ssm_linear_cross_entropy_backward(const float *grad_loss, const void *hidden, const void *weight,
                                      const void *targets, int targets_64, long long ignore_index, const float *lse,
                                      void *grad_hidden, void *grad_weight, int rows, int vocab, int width, int dtype,
                                      long long hidden_stride, long long weight_stride, long long grad_hidden_stride,
                                      long long grad_weight_stride, void *workspace, size_t workspace_bytes,
                                      void *stream);

size_t ssm_linear_cross_entropy_workspace_bytes(const void *weight, int rows, int vocab, int width,
                                                long long weight_stride, int backward);

/* Text for a status code (static storage; never NULL). */
const char *ssm_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* SSMSCAN_H */
