// libssmscan C ABI of the operators a selective-scan model is trained and served with (the
// selective scan, the short causal convolution, the cross entropy of a projection): argument
// checks.  Everything here runs on the host and returns before any launch when an argument is
// wrong; nothing is allocated and the stream is not synchronised (except in the opt-in
// SSM_SCAN_CHECK=1 debug mode).
#include <climits>
#include <cstdint>

#include "../../include/ssmscan.h"
#include "selective_common.cuh"

namespace {

constexpr int kMaxTaps = 8;
constexpr int kMaxWidth = 65536;              // of a hidden row
constexpr int kMaxTokens = INT_MAX - 1024;    // 32-bit counts, with a tile past the last

bool is_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool known_dtype(int d) { return d == SSM_F32 || d == SSM_BF16 || d == SSM_F16; }

int status_of(cudaError_t e) { return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

int debug_check(const int32_t *starts, const int32_t *lens, int n_seqs, int n_tokens, cudaStream_t stream)
{
    return ssm::debug_checks() ? ssm::debug_check_sequences(starts, lens, n_seqs, n_tokens, stream) : SSM_OK;
}

// Sizes of a selective scan: 0 ok, else a status.
int sel_sizes(int n_seqs, int n_tokens, int channels, int d_state, int n_groups)
{
    if (n_seqs < 0 || n_tokens < 0 || channels <= 0 || d_state <= 0 || n_groups <= 0 || channels % n_groups != 0)
        return SSM_ERR_INVALID_ARG;
    if (d_state > ssm::kSelMaxState || n_tokens > kMaxTokens)
        return SSM_ERR_UNSUPPORTED;
    // blocks of either pass at the shortest segments, and of the kernels over states
    const long long units = n_seqs + n_tokens / 64LL;
    for (int backward = 0; backward < 2; ++backward)
        if (units * ssm::sel_shape(channels, d_state, n_groups, backward != 0).cblocks > INT_MAX)
            return SSM_ERR_UNSUPPORTED;
    if ((long long)channels * (d_state + 2) > INT_MAX || (long long)n_groups * d_state > INT_MAX ||
        (long long)n_seqs * channels > (long long)INT_MAX * 256 / d_state || n_seqs > INT_MAX / 1024)
        return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

int conv_sizes(int n_seqs, int n_tokens, int channels, int K)
{
    if (n_seqs < 0 || n_tokens < 0 || channels <= 0 || K <= 0)
        return SSM_ERR_INVALID_ARG;
    if (K > kMaxTaps || n_tokens > kMaxTokens || channels > INT_MAX - 1024)
        return SSM_ERR_UNSUPPORTED;
    return ssm::causal_conv_blocks(n_seqs, n_tokens, channels) > INT_MAX ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

int loss_sizes(int rows, int vocab, int width)
{
    if (rows < 0 || vocab <= 0 || width <= 0)
        return SSM_ERR_INVALID_ARG;
    if (width > kMaxWidth || rows > kMaxTokens || vocab > kMaxTokens)
        return SSM_ERR_UNSUPPORTED;
    const long long tiles = (rows / 256 + 1LL) * (vocab / 256 + 1LL);
    return tiles > INT_MAX || (long long)vocab * (width / 8 + 1) / 256 > INT_MAX - 1 ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

ssm::SelArgs sel_args(const void *x, const void *dt, const float *A, const void *B, const void *C, const float *D,
                      const void *z, const float *dt_bias, const int32_t *starts, const int32_t *lens,
                      const int32_t *resume, int n_seqs, int n_tokens, int channels, int d_state, int n_groups,
                      int softplus, long long sx, long long sdt, long long sB, long long sC, long long sz)
{
    ssm::SelArgs a{};
    a.x = x; a.dt = dt; a.A = A; a.B = B; a.C = C; a.D = D; a.z = z; a.bias = dt_bias;
    a.starts = starts; a.lens = lens; a.resume = resume;
    a.n_seqs = n_seqs; a.n_tokens = n_tokens; a.channels = channels; a.N = d_state; a.groups = n_groups; a.softplus = softplus;
    a.sx = sx; a.sdt = sdt; a.sB = sB; a.sC = sC; a.sz = sz;
    return a;
}

// What both directions of the scan check of their inputs.
bool sel_inputs_ok(const void *x, const void *dt, const float *A, const void *B, const void *C, const float *D,
                   const void *z, const float *dt_bias, const int32_t *starts, const int32_t *lens,
                   const int32_t *resume, int n_tokens, int channels, int bc, int dtype, long long sx, long long sdt,
                   long long sB, long long sC, long long sz)
{
    if (sx < channels || sdt < channels || sB < bc || sC < bc || (z && sz < channels))
        return false;
    if (!A || !starts || !lens || !resume || (n_tokens > 0 && (!x || !dt || !B || !C)))
        return false;
    const uintptr_t e = ssm::dtype_size(dtype);
    return is_aligned(A, 4) && is_aligned(D, 4) && is_aligned(dt_bias, 4) && is_aligned(starts, 4) && is_aligned(lens, 4) &&
           is_aligned(resume, 4) && is_aligned(x, e) && is_aligned(dt, e) && is_aligned(B, e) && is_aligned(C, e) &&
           is_aligned(z, e);
}

}  // namespace

extern "C" {

long long ssm_selective_scan_chunks(int n_seqs, int n_tokens)
{
    return n_seqs < 0 || n_tokens < 0 || n_tokens > kMaxTokens ? 0 : ssm::sel_chunk_rows(n_seqs, n_tokens);
}

size_t ssm_selective_scan_workspace_bytes(int n_seqs, int n_tokens, int channels, int d_state, int n_groups)
{
    if (n_seqs <= 0 || sel_sizes(n_seqs, n_tokens, channels, d_state, n_groups) != SSM_OK)
        return 0;
    return ssm::sel_scan_workspace_bytes(n_seqs, n_tokens, channels, d_state, n_groups);
}

size_t ssm_selective_scan_backward_workspace_bytes(int n_seqs, int n_tokens, int channels, int d_state, int n_groups)
{
    if (n_seqs <= 0 || sel_sizes(n_seqs, n_tokens, channels, d_state, n_groups) != SSM_OK)
        return 0;
    return ssm::sel_backward_workspace_bytes(n_seqs, n_tokens, channels, d_state, n_groups);
}

int ssm_selective_scan(float *state_slots, const void *x, const void *dt, const float *A, const void *B, const void *C,
                       const float *D, const void *z, const float *dt_bias, int dt_softplus, void *y,
                       const int32_t *seq_starts, const int32_t *seq_lens, const int32_t *resume_flags, int n_seqs,
                       int n_tokens, int channels, int d_state, int n_groups, int dtype, long long x_stride,
                       long long dt_stride, long long B_stride, long long C_stride, long long z_stride,
                       long long y_stride, float *chunk_states, void *workspace, size_t workspace_bytes, void *stream_v)
{
    int rc = sel_sizes(n_seqs, n_tokens, channels, d_state, n_groups);
    if (rc != SSM_OK)
        return rc;
    if (!known_dtype(dtype))
        return SSM_ERR_INVALID_ARG;
    if (n_seqs == 0)
        return SSM_OK;
    if (!sel_inputs_ok(x, dt, A, B, C, D, z, dt_bias, seq_starts, seq_lens, resume_flags, n_tokens, channels,
                       n_groups * d_state, dtype, x_stride, dt_stride, B_stride, C_stride, z_stride))
        return SSM_ERR_INVALID_ARG;
    if (!state_slots || !is_aligned(state_slots, 4) || !is_aligned(chunk_states, 4) || y_stride < channels ||
        (n_tokens > 0 && !y) || !is_aligned(y, ssm::dtype_size(dtype)))
        return SSM_ERR_INVALID_ARG;
    const size_t need = ssm_selective_scan_workspace_bytes(n_seqs, n_tokens, channels, d_state, n_groups);
    if (need > 0 && (!workspace || !is_aligned(workspace, 256) || workspace_bytes < need))
        return SSM_ERR_INVALID_ARG;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_v);
    rc = debug_check(seq_starts, seq_lens, n_seqs, n_tokens, stream);
    if (rc != SSM_OK)
        return rc;
    ssm::SelArgs a = sel_args(x, dt, A, B, C, D, z, dt_bias, seq_starts, seq_lens, resume_flags, n_seqs, n_tokens, channels,
                              d_state, n_groups, dt_softplus != 0, x_stride, dt_stride, B_stride, C_stride, z_stride);
    a.state = state_slots;
    a.y = y;
    a.sy = y_stride;
    a.chunk_states = chunk_states;
    return status_of(ssm::launch_selective_scan(a, dtype, workspace, stream));
}

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
                                void *workspace, size_t workspace_bytes, void *stream_v)
{
    int rc = sel_sizes(n_seqs, n_tokens, channels, d_state, n_groups);
    if (rc != SSM_OK)
        return rc;
    const int bc = n_groups * d_state;
    if (!known_dtype(dtype) || grad_y_stride < channels || grad_x_stride < channels || grad_dt_stride < channels ||
        grad_B_stride < bc || grad_C_stride < bc || (z && grad_z_stride < channels))
        return SSM_ERR_INVALID_ARG;
    // a gradient for each input that is there, none for one that is not
    if (!grad_A || (D != nullptr) != (grad_D != nullptr) || (dt_bias != nullptr) != (grad_dt_bias != nullptr) ||
        !is_aligned(grad_A, 4) || !is_aligned(grad_D, 4) || !is_aligned(grad_dt_bias, 4))
        return SSM_ERR_INVALID_ARG;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_v);
    if (n_seqs == 0) {                                      // no token: the parameters' gradients are zero
        cudaError_t e = cudaMemsetAsync(grad_A, 0, (size_t)channels * d_state * 4, stream);
        if (e == cudaSuccess && grad_D)
            e = cudaMemsetAsync(grad_D, 0, (size_t)channels * 4, stream);
        if (e == cudaSuccess && grad_dt_bias)
            e = cudaMemsetAsync(grad_dt_bias, 0, (size_t)channels * 4, stream);
        return status_of(e);
    }
    if (!sel_inputs_ok(x, dt, A, B, C, D, z, dt_bias, seq_starts, seq_lens, resume_flags, n_tokens, channels, bc, dtype,
                       x_stride, dt_stride, B_stride, C_stride, z_stride))
        return SSM_ERR_INVALID_ARG;
    const uintptr_t e = ssm::dtype_size(dtype);
    if (!chunk_states || !is_aligned(chunk_states, 4) || !is_aligned(grad_state, 4) || !is_aligned(grad_initial_state, 4) ||
        !is_aligned(grad_y, e) || !is_aligned(grad_x, e) || !is_aligned(grad_dt, e) || !is_aligned(grad_B, e) ||
        !is_aligned(grad_C, e) || !is_aligned(grad_z, e))
        return SSM_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!grad_y || !grad_x || !grad_dt || !grad_B || !grad_C || (z != nullptr) != (grad_z != nullptr)))
        return SSM_ERR_INVALID_ARG;
    if (!workspace || !is_aligned(workspace, 256) ||
        workspace_bytes < ssm_selective_scan_backward_workspace_bytes(n_seqs, n_tokens, channels, d_state, n_groups))
        return SSM_ERR_INVALID_ARG;
    rc = debug_check(seq_starts, seq_lens, n_seqs, n_tokens, stream);
    if (rc != SSM_OK)
        return rc;
    ssm::SelArgs a = sel_args(x, dt, A, B, C, D, z, dt_bias, seq_starts, seq_lens, resume_flags, n_seqs, n_tokens, channels,
                              d_state, n_groups, dt_softplus != 0, x_stride, dt_stride, B_stride, C_stride, z_stride);
    a.chunk_states = const_cast<float *>(chunk_states);
    a.grad_y = grad_y; a.grad_state = grad_state; a.sgy = grad_y_stride;
    a.grad_x = grad_x; a.grad_dt = grad_dt; a.grad_A = grad_A; a.grad_B = grad_B; a.grad_C = grad_C; a.grad_D = grad_D;
    a.grad_z = grad_z; a.grad_bias = grad_dt_bias; a.grad_state0 = grad_initial_state;
    a.sgx = grad_x_stride; a.sgdt = grad_dt_stride; a.sgB = grad_B_stride; a.sgC = grad_C_stride; a.sgz = grad_z_stride;
    return status_of(ssm::launch_selective_scan_backward(a, dtype, workspace, stream));
}

int ssm_causal_conv(const void *x, const float *weight, const float *bias, float *conv_state, void *out,
                    const int32_t *seq_starts, const int32_t *seq_lens, const int32_t *resume_flags, int n_seqs,
                    int n_tokens, int channels, int kernel_size, int silu, int dtype, long long x_stride,
                    long long out_stride, void *stream_v)
{
    int rc = conv_sizes(n_seqs, n_tokens, channels, kernel_size);
    if (rc != SSM_OK)
        return rc;
    if (!known_dtype(dtype) || x_stride < channels || out_stride < channels)
        return SSM_ERR_INVALID_ARG;
    if (n_seqs == 0)
        return SSM_OK;
    if (!weight || !seq_starts || !seq_lens || !resume_flags || (kernel_size > 1 && !conv_state) ||
        (n_tokens > 0 && (!x || !out)))
        return SSM_ERR_INVALID_ARG;
    const uintptr_t e = ssm::dtype_size(dtype);
    if (!is_aligned(weight, 4) || !is_aligned(bias, 4) || !is_aligned(conv_state, 4) || !is_aligned(seq_starts, 4) ||
        !is_aligned(seq_lens, 4) || !is_aligned(resume_flags, 4) || !is_aligned(x, e) || !is_aligned(out, e))
        return SSM_ERR_INVALID_ARG;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_v);
    rc = debug_check(seq_starts, seq_lens, n_seqs, n_tokens, stream);
    if (rc != SSM_OK)
        return rc;
    ssm::CausalConv c{};
    c.x = x; c.w = weight; c.bias = bias; c.state = conv_state; c.out = out;
    c.starts = seq_starts; c.lens = seq_lens; c.resume = resume_flags;
    c.n_seqs = n_seqs; c.n_tokens = n_tokens; c.channels = channels; c.K = kernel_size; c.silu = silu != 0; c.dtype = dtype;
    c.sx = x_stride; c.so = out_stride;
    return status_of(ssm::launch_causal_conv(c, false, stream));
}

size_t ssm_causal_conv_backward_workspace_bytes(int n_seqs, int n_tokens, int channels, int kernel_size)
{
    if (n_seqs <= 0 || conv_sizes(n_seqs, n_tokens, channels, kernel_size) != SSM_OK)
        return 0;
    return ssm::causal_conv_backward_workspace_bytes(n_seqs, n_tokens, channels, kernel_size);
}

int ssm_causal_conv_backward(const void *grad_out, const float *grad_state, const void *x, const float *weight,
                             const float *bias, const float *initial_state, const int32_t *seq_starts,
                             const int32_t *seq_lens, const int32_t *resume_flags, int n_seqs, int n_tokens,
                             int channels, int kernel_size, int silu, int dtype, long long grad_out_stride,
                             long long x_stride, void *grad_x, float *grad_weight, float *grad_bias,
                             float *grad_initial_state, long long grad_x_stride, void *workspace,
                             size_t workspace_bytes, void *stream_v)
{
    int rc = conv_sizes(n_seqs, n_tokens, channels, kernel_size);
    if (rc != SSM_OK)
        return rc;
    if (!known_dtype(dtype) || x_stride < channels || grad_out_stride < channels || grad_x_stride < channels)
        return SSM_ERR_INVALID_ARG;
    if (!weight || !grad_weight || (bias != nullptr) != (grad_bias != nullptr) || !is_aligned(weight, 4) ||
        !is_aligned(bias, 4) || !is_aligned(grad_weight, 4) || !is_aligned(grad_bias, 4))
        return SSM_ERR_INVALID_ARG;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_v);
    if (n_seqs == 0) {                                      // no token: the parameters' gradients are zero
        cudaError_t e = cudaMemsetAsync(grad_weight, 0, (size_t)channels * kernel_size * 4, stream);
        if (e == cudaSuccess && grad_bias)
            e = cudaMemsetAsync(grad_bias, 0, (size_t)channels * 4, stream);
        return status_of(e);
    }
    // without the slots' contents every sequence is taken to be fresh, so there must be no flags that say otherwise
    if (!seq_starts || !seq_lens || (kernel_size > 1 && (initial_state != nullptr) != (resume_flags != nullptr)) ||
        (grad_initial_state && !initial_state) || (n_tokens > 0 && (!grad_out || !x || !grad_x)))
        return SSM_ERR_INVALID_ARG;
    const uintptr_t e = ssm::dtype_size(dtype);
    if (!is_aligned(grad_state, 4) || !is_aligned(initial_state, 4) || !is_aligned(grad_initial_state, 4) ||
        !is_aligned(seq_starts, 4) || !is_aligned(seq_lens, 4) || !is_aligned(resume_flags, 4) || !is_aligned(x, e) ||
        !is_aligned(grad_out, e) || !is_aligned(grad_x, e))
        return SSM_ERR_INVALID_ARG;
    if (!workspace || !is_aligned(workspace, 256) ||
        workspace_bytes < ssm_causal_conv_backward_workspace_bytes(n_seqs, n_tokens, channels, kernel_size))
        return SSM_ERR_INVALID_ARG;
    rc = debug_check(seq_starts, seq_lens, n_seqs, n_tokens, stream);
    if (rc != SSM_OK)
        return rc;
    ssm::CausalConv c{};
    c.x = x; c.w = weight; c.bias = bias; c.starts = seq_starts; c.lens = seq_lens; c.resume = resume_flags;
    c.n_seqs = n_seqs; c.n_tokens = n_tokens; c.channels = channels; c.K = kernel_size; c.silu = silu != 0; c.dtype = dtype;
    c.sx = x_stride; c.sgo = grad_out_stride; c.sgx = grad_x_stride;
    c.grad_out = grad_out; c.grad_x = grad_x; c.grad_w = grad_weight; c.grad_bias = grad_bias;
    if (kernel_size > 1) {                                  // one tap has no slots, whatever pointers stand for them (and no flags)
        c.state0 = initial_state; c.grad_state = grad_state; c.grad_state0 = grad_initial_state;
    }
    c.part = static_cast<float *>(workspace);
    return status_of(ssm::launch_causal_conv(c, true, stream));
}

size_t ssm_linear_cross_entropy_workspace_bytes(const void *weight, int rows, int vocab, int width,
                                                long long weight_stride, int backward)
{
    if (rows <= 0 || loss_sizes(rows, vocab, width) != SSM_OK || weight_stride < width)
        return 0;
    return ssm::cross_entropy_workspace_bytes(weight, rows, vocab, width, weight_stride, backward != 0);
}

int ssm_linear_cross_entropy(const void *hidden, const void *weight, const void *targets, int targets_64,
                             long long ignore_index, float *loss, float *lse, int rows, int vocab, int width, int dtype,
                             long long hidden_stride, long long weight_stride, void *workspace, size_t workspace_bytes,
                             void *stream)
{
    const int rc = loss_sizes(rows, vocab, width);
    if (rc != SSM_OK)
        return rc;
    if (!known_dtype(dtype) || hidden_stride < width || weight_stride < width)
        return SSM_ERR_INVALID_ARG;
    if (dtype == SSM_F32)
        return SSM_ERR_UNSUPPORTED;
    if (rows == 0)
        return SSM_OK;
    if (!hidden || !weight || !targets || !loss || !lse || !is_aligned(hidden, 2) || !is_aligned(weight, 2) ||
        !is_aligned(targets, targets_64 ? 8 : 4) || !is_aligned(loss, 4) || !is_aligned(lse, 4))
        return SSM_ERR_INVALID_ARG;
    if (!workspace || !is_aligned(workspace, 256) ||
        workspace_bytes < ssm::cross_entropy_workspace_bytes(weight, rows, vocab, width, weight_stride, false))
        return SSM_ERR_INVALID_ARG;
    ssm::CrossEntropy c{};
    c.h = hidden; c.w = weight; c.target = targets; c.loss = loss; c.lse = lse;
    c.T = rows; c.V = vocab; c.D = width; c.wide = targets_64 != 0; c.dtype = dtype;
    c.sh = hidden_stride; c.sw = weight_stride; c.ignore = ignore_index;
    return status_of(ssm::launch_cross_entropy(c, workspace, false, reinterpret_cast<cudaStream_t>(stream)));
}

int ssm_linear_cross_entropy_backward(const float *grad_loss, const void *hidden, const void *weight,
                                      const void *targets, int targets_64, long long ignore_index, const float *lse,
                                      void *grad_hidden, void *grad_weight, int rows, int vocab, int width, int dtype,
                                      long long hidden_stride, long long weight_stride, long long grad_hidden_stride,
                                      long long grad_weight_stride, void *workspace, size_t workspace_bytes,
                                      void *stream_v)
{
    const int rc = loss_sizes(rows, vocab, width);
    if (rc != SSM_OK)
        return rc;
    if (!known_dtype(dtype) || hidden_stride < width || weight_stride < width || grad_hidden_stride < width ||
        (grad_weight && grad_weight_stride < width))
        return SSM_ERR_INVALID_ARG;
    if (dtype == SSM_F32)
        return SSM_ERR_UNSUPPORTED;
    if (!is_aligned(grad_weight, 2))
        return SSM_ERR_INVALID_ARG;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_v);
    if (rows == 0)
        return grad_weight ? status_of(cudaMemset2DAsync(grad_weight, (size_t)grad_weight_stride * 2, 0, (size_t)width * 2,
                                                         (size_t)vocab, stream))
                           : SSM_OK;
    if (!grad_loss || !hidden || !weight || !targets || !lse || !grad_hidden || !is_aligned(grad_loss, 4) ||
        !is_aligned(hidden, 2) || !is_aligned(weight, 2) || !is_aligned(targets, targets_64 ? 8 : 4) ||
        !is_aligned(lse, 4) || !is_aligned(grad_hidden, 2))
        return SSM_ERR_INVALID_ARG;
    if (!workspace || !is_aligned(workspace, 256) ||
        workspace_bytes < ssm::cross_entropy_workspace_bytes(weight, rows, vocab, width, weight_stride, true))
        return SSM_ERR_INVALID_ARG;
    ssm::CrossEntropy c{};
    c.h = hidden; c.w = weight; c.target = targets; c.grad_loss = grad_loss; c.lse_in = lse;
    c.grad_h = grad_hidden; c.grad_w = grad_weight;
    c.T = rows; c.V = vocab; c.D = width; c.wide = targets_64 != 0; c.dtype = dtype;
    c.sh = hidden_stride; c.sw = weight_stride; c.sgh = grad_hidden_stride; c.sgw = grad_weight_stride;
    c.ignore = ignore_index;
    return status_of(ssm::launch_cross_entropy(c, workspace, true, stream));
}

}  // extern "C"
