"""libssmscan: the Mamba2 selective-state scan as sm_103a CUDA kernels.

    from state_space_model_ssm_gb300 import ssm_scan
    y = ssm_scan(state_slots, x, dt, A, B, C, D, seq_starts, seq_lens, resume_flags)

Around the scan: the gated linear recurrence with its gradient
(``ssm_gated_scan``, ``ssm_gated_scan_backward``), the RMS norm with the
residual's addition, its 8-bit output and its gradient (``ssm_add_norm``,
``ssm_add_norm_backward``), the row quantiser (``ssm_quantize_rows``) and the
8-bit integer matrix product (``ssm_int8_matmul``); see ``layers``.  They are not
recorded by torch's autograd: a training step calls the backward functions.

The C ABI is declared in ``include/ssmscan.h``; ``binding`` wraps it with
ctypes.  ``workloads`` draws the seeded synthetic inputs.
"""
from .layers import (add_norm_backward_workspace_bytes, gated_scan_backward_workspace_bytes,  # noqa: F401
                     gated_scan_chunk_states, int8_matmul_workspace_bytes, ssm_add_norm, ssm_add_norm_backward,
                     ssm_gated_scan, ssm_gated_scan_backward, ssm_int8_matmul, ssm_quantize_rows)
from .binding import (PATH_AUTO, PATH_DECODE, PATH_PREFILL, PATH_PREFILL_DIRECT,  # noqa: F401
                      SEGMENT_STATE_AUTO, SEGMENT_STATE_FP32, SEGMENT_STATE_TENSOR,
                      Options, SsmScanError, Tuning,
                      load, ssd_workspace_bytes, ssm_conv1d, ssm_scan, ssm_scan_ssd,
                      status_string)

__all__ = ["add_norm_backward_workspace_bytes", "gated_scan_backward_workspace_bytes", "int8_matmul_workspace_bytes",
           "gated_scan_chunk_states", "ssm_add_norm", "ssm_add_norm_backward", "ssm_gated_scan", "ssm_gated_scan_backward",
           "ssm_int8_matmul", "ssm_quantize_rows", "Options", "ssm_conv1d", "ssm_scan", "ssm_scan_ssd", "ssd_workspace_bytes", "Tuning", "SsmScanError", "PATH_AUTO", "PATH_DECODE",
           "PATH_PREFILL", "PATH_PREFILL_DIRECT", "SEGMENT_STATE_AUTO", "SEGMENT_STATE_FP32",
           "SEGMENT_STATE_TENSOR", "load", "status_string"]
