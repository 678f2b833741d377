// libssmscan C ABI of the layer operators around the scan: argument checks.
// Everything here runs on the host and returns before any launch when an
// argument is wrong; nothing is allocated and the stream is not synchronised
// (except in the opt-in SSM_SCAN_CHECK=1 debug mode).
#include <climits>
#include <cstdint>
#include <cmath>

#include "../../include/ssmscan.h"
#include "gated_common.cuh"

namespace {

constexpr int kMaxRowWidth = 16384;       // one row lives in a block's registers
constexpr int kMaxInner = 131071;         // 131071 * 128 * 128 < 2^31
// The kernels count tokens (rows, channels) in 32 bits, up to one round of a cluster (one tile) past the last.
constexpr int kMaxTokens = INT_MAX - ssm::kGatedChunk * ssm::kGatedMaxCluster;
constexpr int kMaxTiled = INT_MAX - 256;

bool is_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool known_dtype(int d) { return d == SSM_F32 || d == SSM_BF16 || d == SSM_F16; }

int status_of(cudaError_t e) { return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

// Sizes of a gated scan: 0 ok, else a status.
int gated_sizes(int n_seqs, int n_tokens, int channels)
{
    if (n_seqs < 0 || n_tokens < 0 || channels <= 0)
        return SSM_ERR_INVALID_ARG;
    const long long blocks = (long long)n_seqs * ((channels + ssm::kGatedCh - 1LL) / ssm::kGatedCh) * ssm::kGatedMaxCluster;
    return blocks > INT_MAX || n_tokens > kMaxTokens ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

int int8_sizes(int rows, int out_features, int inner)
{
    if (rows < 0 || out_features <= 0 || inner <= 0)
        return SSM_ERR_INVALID_ARG;
    // blocks of the smallest tiles, and of the repacking kernel
    const long long tiles = (rows / 128 + 1LL) * (out_features / 128 + 1LL);
    const long long cells = ((long long)rows + out_features) * (inner / 16 + 1LL) / 256 + 2;
    return inner > kMaxInner || rows > kMaxTiled || out_features > kMaxTiled || tiles > INT_MAX || cells > INT_MAX ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

int gated_debug_check(const int32_t *starts, const int32_t *lens, int n_seqs, int n_tokens, cudaStream_t stream)
{
    return ssm::debug_checks() ? ssm::debug_check_sequences(starts, lens, n_seqs, n_tokens, stream) : SSM_OK;
}

}  // namespace

extern "C" {

long long ssm_gated_scan_chunks(int n_seqs, int n_tokens, int channels)
{
    return gated_sizes(n_seqs, n_tokens, channels) == SSM_OK ? ssm::gated_chunk_rows(n_seqs, n_tokens) : 0;
}

size_t ssm_gated_scan_backward_workspace_bytes(int n_seqs, int n_tokens, int channels)
{
    if (n_seqs <= 0 || gated_sizes(n_seqs, n_tokens, channels) != SSM_OK)
        return 0;
    return (size_t)n_seqs * ssm::gated_cluster(n_seqs, n_tokens, channels, false) * channels * sizeof(float);
}

int ssm_gated_scan(float *state_slots, const void *x, const void *gate_a, const void *gate_x, const float *lam,
                   float decay_scale, void *y, const int32_t *seq_starts, const int32_t *seq_lens,
                   const int32_t *resume_flags, int n_seqs, int n_tokens, int channels, int dtype,
                   long long x_stride, long long gate_a_stride, long long gate_x_stride, long long y_stride,
                   float *chunk_states, void *stream_v)
{
    int rc = gated_sizes(n_seqs, n_tokens, channels);
    if (rc != SSM_OK)
        return rc;
    if (!known_dtype(dtype) || !(decay_scale > 0.f) || !std::isfinite(decay_scale))
        return SSM_ERR_INVALID_ARG;
    if (x_stride < channels || gate_a_stride < channels || gate_x_stride < channels || y_stride < channels)
        return SSM_ERR_INVALID_ARG;
    if (n_seqs == 0)
        return SSM_OK;
    if (!state_slots || !lam || !seq_starts || !seq_lens || !resume_flags)
        return SSM_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!x || !gate_a || !gate_x || !y))
        return SSM_ERR_INVALID_ARG;
    const uintptr_t e = ssm::dtype_size(dtype);
    if (!is_aligned(state_slots, 4) || !is_aligned(lam, 4) || !is_aligned(seq_starts, 4) || !is_aligned(seq_lens, 4) ||
        !is_aligned(resume_flags, 4) || !is_aligned(chunk_states, 4) || !is_aligned(x, e) || !is_aligned(gate_a, e) ||
        !is_aligned(gate_x, e) || !is_aligned(y, e))
        return SSM_ERR_INVALID_ARG;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_v);
    rc = gated_debug_check(seq_starts, seq_lens, n_seqs, n_tokens, stream);
    if (rc != SSM_OK)
        return rc;
    ssm::GatedArgs a{};
    a.state = state_slots; a.x = x; a.gate_a = gate_a; a.gate_x = gate_x; a.lam = lam; a.decay_scale = decay_scale;
    a.y = y; a.seq_starts = seq_starts; a.seq_lens = seq_lens; a.resume = resume_flags;
    a.n_seqs = n_seqs; a.n_tokens = n_tokens; a.C = channels;
    a.sx = x_stride; a.sga = gate_a_stride; a.sgx = gate_x_stride; a.sy = y_stride;
    a.chunk_states = chunk_states;
    return status_of(ssm::launch_gated_scan(a, dtype, stream));
}

int ssm_gated_scan_backward(const void *grad_y, const float *grad_state, const void *x, const void *gate_a,
                            const void *gate_x, const float *lam, float decay_scale, const float *chunk_states,
                            const int32_t *seq_starts, const int32_t *seq_lens, const int32_t *resume_flags,
                            int n_seqs, int n_tokens, int channels, int dtype, long long x_stride,
                            long long gate_a_stride, long long gate_x_stride, long long grad_y_stride,
                            void *grad_x, void *grad_gate_a, void *grad_gate_x, long long grad_x_stride,
                            long long grad_gate_a_stride, long long grad_gate_x_stride, float *grad_lam,
                            float *grad_initial_state, void *workspace, size_t workspace_bytes, void *stream_v)
{
    int rc = gated_sizes(n_seqs, n_tokens, channels);
    if (rc != SSM_OK)
        return rc;
    if (!known_dtype(dtype) || !(decay_scale > 0.f) || !std::isfinite(decay_scale))
        return SSM_ERR_INVALID_ARG;
    if (x_stride < channels || gate_a_stride < channels || gate_x_stride < channels || grad_y_stride < channels ||
        grad_x_stride < channels || grad_gate_a_stride < channels || grad_gate_x_stride < channels)
        return SSM_ERR_INVALID_ARG;
    if (!lam || !grad_lam || !is_aligned(lam, 4) || !is_aligned(grad_lam, 4))
        return SSM_ERR_INVALID_ARG;
    if (n_seqs > 0 && (!chunk_states || !seq_starts || !seq_lens || !resume_flags))
        return SSM_ERR_INVALID_ARG;
    if (n_seqs > 0 && n_tokens > 0 && (!grad_y || !x || !gate_a || !gate_x || !grad_x || !grad_gate_a || !grad_gate_x))
        return SSM_ERR_INVALID_ARG;
    const uintptr_t e = ssm::dtype_size(dtype);
    if (!is_aligned(grad_state, 4) || !is_aligned(chunk_states, 4) || !is_aligned(seq_starts, 4) ||
        !is_aligned(seq_lens, 4) || !is_aligned(resume_flags, 4) || !is_aligned(grad_initial_state, 4) ||
        !is_aligned(grad_y, e) || !is_aligned(x, e) || !is_aligned(gate_a, e) || !is_aligned(gate_x, e) ||
        !is_aligned(grad_x, e) || !is_aligned(grad_gate_a, e) || !is_aligned(grad_gate_x, e))
        return SSM_ERR_INVALID_ARG;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_v);
    if (n_seqs == 0)                                       // no token: the parameter's gradient is zero
        return status_of(cudaMemsetAsync(grad_lam, 0, (size_t)channels * sizeof(float), stream));
    if (!workspace || !is_aligned(workspace, 256) ||
        workspace_bytes < ssm_gated_scan_backward_workspace_bytes(n_seqs, n_tokens, channels))
        return SSM_ERR_INVALID_ARG;
    rc = gated_debug_check(seq_starts, seq_lens, n_seqs, n_tokens, stream);
    if (rc != SSM_OK)
        return rc;
    ssm::GatedArgs a{};
    a.x = x; a.gate_a = gate_a; a.gate_x = gate_x; a.lam = lam; a.decay_scale = decay_scale;
    a.seq_starts = seq_starts; a.seq_lens = seq_lens; a.resume = resume_flags;
    a.n_seqs = n_seqs; a.n_tokens = n_tokens; a.C = channels;
    a.sx = x_stride; a.sga = gate_a_stride; a.sgx = gate_x_stride; a.sy = grad_y_stride;
    a.chunk_states = const_cast<float *>(chunk_states);
    a.grad_y = grad_y; a.grad_state = grad_state;
    a.grad_x = grad_x; a.grad_ga = grad_gate_a; a.grad_gx = grad_gate_x;
    a.gsx = grad_x_stride; a.gsga = grad_gate_a_stride; a.gsgx = grad_gate_x_stride;
    a.grad_lam = grad_lam; a.grad_state0 = grad_initial_state;
    a.lam_part = static_cast<float *>(workspace);
    return status_of(ssm::launch_gated_scan_backward(a, dtype, stream));
}

int ssm_add_norm(const void *x, const void *residual, const float *weight, float eps, void *residual_out, void *y,
                 int8_t *codes, float *scales, int rows, int width, int dtype, int residual_dtype,
                 long long x_stride, long long residual_stride, long long residual_out_stride, long long out_stride,
                 void *stream)
{
    if (rows < 0 || width <= 0 || !known_dtype(dtype) || !known_dtype(residual_dtype) || !(eps >= 0.f) ||
        !std::isfinite(eps))
        return SSM_ERR_INVALID_ARG;
    if (residual_dtype != dtype && residual_dtype != SSM_F32)
        return SSM_ERR_INVALID_ARG;
    if (x_stride < width || out_stride < width || (residual && residual_stride < width) ||
        (residual_out && residual_out_stride < width))
        return SSM_ERR_INVALID_ARG;
    if (width > kMaxRowWidth)
        return SSM_ERR_UNSUPPORTED;
    if (rows == 0)
        return SSM_OK;
    if (!weight || (y != nullptr) == (codes != nullptr) || (codes != nullptr) != (scales != nullptr) ||
        (residual_out && !residual))
        return SSM_ERR_INVALID_ARG;
    const uintptr_t e = ssm::dtype_size(dtype), er = ssm::dtype_size(residual_dtype);
    if (!x || !is_aligned(x, e) || !is_aligned(y, e) || !is_aligned(residual, er) || !is_aligned(residual_out, er) ||
        !is_aligned(weight, 4) || !is_aligned(scales, 4))
        return SSM_ERR_INVALID_ARG;
    return status_of(ssm::launch_add_norm(x, residual, weight, eps, residual_out, y, codes, scales, rows, width, dtype,
                                          residual_dtype, x_stride, residual_stride, residual_out_stride, out_stride,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

int ssm_quantize_rows(const void *x, int8_t *codes, float *scales, int rows, int width, int dtype,
                      long long x_stride, long long codes_stride, void *stream)
{
    if (rows < 0 || width <= 0 || !known_dtype(dtype) || x_stride < width || codes_stride < width)
        return SSM_ERR_INVALID_ARG;
    if (width > kMaxRowWidth)
        return SSM_ERR_UNSUPPORTED;
    if (rows == 0)
        return SSM_OK;
    if (!x || !codes || !scales || !is_aligned(x, ssm::dtype_size(dtype)) || !is_aligned(scales, 4))
        return SSM_ERR_INVALID_ARG;
    return status_of(ssm::launch_add_norm(x, nullptr, nullptr, 0.f, nullptr, nullptr, codes, scales, rows, width,
                                          dtype, dtype, x_stride, 0, 0, codes_stride,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

size_t ssm_add_norm_backward_workspace_bytes(int rows, int width)
{
    if (rows < 0 || width <= 0 || width > kMaxRowWidth)
        return 0;
    return (size_t)ssm::add_norm_parts(rows, width) * width * sizeof(float);
}

int ssm_add_norm_backward(const void *grad_y, const void *h, const float *weight, float eps, const void *grad_h,
                          void *grad_in, float *grad_weight, int rows, int width, int dtype, int residual_dtype,
                          long long grad_y_stride, long long h_stride, long long grad_h_stride,
                          long long grad_in_stride, void *workspace, size_t workspace_bytes, void *stream_v)
{
    if (rows < 0 || width <= 0 || !known_dtype(dtype) || !known_dtype(residual_dtype) || !(eps >= 0.f) ||
        !std::isfinite(eps))
        return SSM_ERR_INVALID_ARG;
    if (residual_dtype != dtype && residual_dtype != SSM_F32)
        return SSM_ERR_INVALID_ARG;
    if (grad_y_stride < width || h_stride < width || grad_in_stride < width || (grad_h && grad_h_stride < width))
        return SSM_ERR_INVALID_ARG;
    if (width > kMaxRowWidth)
        return SSM_ERR_UNSUPPORTED;
    if (!weight || !grad_weight || !is_aligned(weight, 4) || !is_aligned(grad_weight, 4))
        return SSM_ERR_INVALID_ARG;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_v);
    if (rows == 0)
        return status_of(cudaMemsetAsync(grad_weight, 0, (size_t)width * sizeof(float), stream));
    const uintptr_t e = ssm::dtype_size(dtype), er = ssm::dtype_size(residual_dtype);
    if (!grad_y || !h || !grad_in || !is_aligned(grad_y, e) || !is_aligned(h, er) || !is_aligned(grad_h, er) ||
        !is_aligned(grad_in, er))
        return SSM_ERR_INVALID_ARG;
    if (!workspace || !is_aligned(workspace, 256) ||
        workspace_bytes < ssm_add_norm_backward_workspace_bytes(rows, width))
        return SSM_ERR_INVALID_ARG;
    return status_of(ssm::launch_add_norm_backward(grad_y, h, grad_h, weight, eps, grad_in, grad_weight,
                                                   static_cast<float *>(workspace), rows, width, dtype,
                                                   residual_dtype, grad_y_stride, h_stride, grad_h_stride,
                                                   grad_in_stride, stream));
}

size_t ssm_int8_matmul_workspace_bytes(const int8_t *x, const int8_t *w, int rows, int out_features, int inner,
                                       long long x_stride, long long w_stride)
{
    if (rows <= 0 || int8_sizes(rows, out_features, inner) != SSM_OK || x_stride < inner || w_stride < inner)
        return 0;
    return ssm::int8_matmul_workspace_bytes(x, w, rows, out_features, inner, x_stride, w_stride);
}

int ssm_int8_matmul(const int8_t *x, const float *x_scales, const int8_t *w, const float *w_scales, const float *bias,
                    void *out, int rows, int out_features, int inner, int out_dtype, long long x_stride,
                    long long w_stride, long long out_stride, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!known_dtype(out_dtype) || (inner > 0 && (x_stride < inner || w_stride < inner)) || out_stride < out_features)
        return SSM_ERR_INVALID_ARG;
    const int rc = int8_sizes(rows, out_features, inner);
    if (rc != SSM_OK)
        return rc;
    if (rows == 0)
        return SSM_OK;
    if (!x || !x_scales || !w || !w_scales || !out || !is_aligned(x_scales, 4) || !is_aligned(w_scales, 4) ||
        !is_aligned(bias, 4) || !is_aligned(out, ssm::dtype_size(out_dtype)))
        return SSM_ERR_INVALID_ARG;
    const size_t need = ssm::int8_matmul_workspace_bytes(x, w, rows, out_features, inner, x_stride, w_stride);
    if (need > 0 && (!workspace || !is_aligned(workspace, 256) || workspace_bytes < need))
        return SSM_ERR_INVALID_ARG;
    return status_of(ssm::launch_int8_matmul(x, x_scales, w, w_scales, bias, out, rows, out_features, inner, out_dtype,
                                             x_stride, w_stride, out_stride, workspace,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
