"""ctypes binding of the operators a selective-scan model is trained and served with (argument
marshalling only): the selective scan with a decay for each channel and state, the short causal
convolution, and the cross entropy of a projection onto a large vocabulary, with their gradients.

Streams, allocation, strides and workspaces as in ``layers``: every function runs on the current
CUDA stream of its tensors' device, or on its keyword argument ``stream``; rows may be further
apart than their width; no function is recorded by torch's autograd, so outputs never
require a gradient and a training step calls the backward functions itself (as
``examples/selective_lm.py`` does).  Formulas and rules are those of ``include/ssmscan.h``.
"""
from __future__ import annotations

import torch

from .binding import SSM_OK, SsmScanError, load
from .layers import _dtype, _flat, _flat_out, _placed, _raw_stream, _rows, _rows_out, _workspace

F32, I32 = torch.float32, torch.int32


def _table(seq_starts, seq_lens, resume_flags, dev):
    one = (seq_lens.shape[0],)
    return (_flat(seq_starts, "seq_starts", I32, dev, one), _flat(seq_lens, "seq_lens", I32, dev, one),
            _flat(resume_flags, "resume_flags", I32, dev, one))


def _optional(t, name, dev, shape):
    return None if t is None else _flat(t, name, F32, dev, shape)


# ---- selective scan ----


def selective_scan_workspace_bytes(n_seqs, n_tokens, channels, d_state, n_groups=1) -> int:
    """Bytes of workspace of ``ssm_selective_scan`` (0: none)."""
    return int(load().ssm_selective_scan_workspace_bytes(int(n_seqs), int(n_tokens), int(channels), int(d_state), int(n_groups)))


def selective_scan_backward_workspace_bytes(n_seqs, n_tokens, channels, d_state, n_groups=1) -> int:
    """Bytes of workspace of ``ssm_selective_scan_backward``."""
    return int(load().ssm_selective_scan_backward_workspace_bytes(int(n_seqs), int(n_tokens), int(channels), int(d_state),
                                                                  int(n_groups)))


def selective_scan_chunk_states(n_seqs, n_tokens, channels, d_state, device="cuda"):
    """An empty chunk_states tensor [chunks, channels, d_state] fp32 for these sizes."""
    chunks = int(load().ssm_selective_scan_chunks(int(n_seqs), int(n_tokens)))
    return torch.empty((chunks, int(channels), int(d_state)), dtype=F32, device=device)


def _scan_inputs(x, dt, A, B, C, D, z, dt_bias, n_groups):
    """(dtype code, device, T, channels, states, pointers and strides) of both directions' inputs."""
    code = _dtype(x, "x")
    dev, dtype = x.device, x.dtype
    T, channels = x.shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise TypeError("A must be a 2-dimensional torch.Tensor [channels, d_state]")
    N = A.shape[1]
    bc = (T, n_groups * N)
    px, sx = _rows(x, "x", dtype, dev, x.shape)
    pdt, sdt = _rows(dt, "dt", dtype, dev, x.shape)
    pA = _flat(A, "A", F32, dev, (channels, N))
    pB, sB = _rows(B, "B", dtype, dev, bc)
    pC, sC = _rows(C, "C", dtype, dev, bc)
    pz, sz = (None, 0) if z is None else _rows(z, "z", dtype, dev, x.shape)
    pD, pb = _optional(D, "D", dev, (channels,)), _optional(dt_bias, "dt_bias", dev, (channels,))
    return code, dev, T, channels, N, (px, pdt, pA, pB, pC, pD, pz, pb), (sx, sdt, sB, sC, sz)


@_placed
def ssm_selective_scan(state_slots, x, dt, A, B, C, D, seq_starts, seq_lens, resume_flags, y=None, *, z=None, dt_bias=None,
                       dt_softplus=False, n_groups=1, chunk_states=None, workspace=None):
    """Selective scan with a decay for each channel and state (``ssm_selective_scan``): with v = dt + dt_bias and
    step = v, or softplus(v) with dt_softplus,

        h = exp(step A) h + step x B,   p = h . C + D x,   y = p z sigmoid(z)

    state_slots [n, C, N] fp32 (updated in place); x, dt and z (or None: y = p) [T, C] fp32, bf16 or fp16;
    A [C, N] fp32; B, C [T, n_groups * N] of x's type (slices of one projection are fine);
    D, dt_bias [C] fp32 or None; seq_starts, seq_lens, resume_flags [n] int32.  N at most 128.
    chunk_states: a tensor of ``selective_scan_chunk_states`` to fill for the backward pass.
    Returns y [T, C] (allocated if not given)."""
    code, dev, T, channels, N, p, s = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, n_groups)
    n = seq_lens.shape[0]
    slots = _flat(state_slots, "state_slots", F32, dev, (n, channels, N))
    table = _table(seq_starts, seq_lens, resume_flags, dev)
    lib = load()
    pc = None
    if chunk_states is not None:
        pc = _flat(chunk_states, "chunk_states", F32, dev, (lib.ssm_selective_scan_chunks(n, T), channels, N))
    handle = _raw_stream(dev.index)
    y, py, sy = _rows_out(y, "y", x.dtype, dev, x.shape)
    ws, nb, workspace = _workspace(workspace, lib.ssm_selective_scan_workspace_bytes(n, T, channels, N, n_groups), dev)
    rc = lib.ssm_selective_scan(slots, *p, 1 if dt_softplus else 0, py, *table, n, T, channels, N, n_groups, code, *s, sy, pc,
                                ws, nb, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_selective_scan")
    return y


@_placed
def ssm_selective_scan_backward(grad_y, x, dt, A, B, C, D, chunk_states, seq_starts, seq_lens, resume_flags, *, z=None,
                                dt_bias=None, dt_softplus=False, n_groups=1, grad_state=None, grad_x=None, grad_dt=None,
                                grad_A=None, grad_B=None, grad_C=None, grad_D=None, grad_z=None, grad_dt_bias=None,
                                grad_initial_state=None, workspace=None):
    """Gradients of ``ssm_selective_scan`` (``ssm_selective_scan_backward``) from the gradient of y and optionally
    of the slots after the call (grad_state [n, C, N] fp32); chunk_states as filled by the forward call.
    Outputs are allocated if not given.  Returns (grad_x, grad_dt, grad_A, grad_B, grad_C, grad_D, grad_z,
    grad_dt_bias, grad_initial_state), with None for D, z and dt_bias that are None."""
    code, dev, T, channels, N, p, s = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, n_groups)
    n, dtype = seq_lens.shape[0], x.dtype
    pg, sg = _rows(grad_y, "grad_y", dtype, dev, x.shape)
    lib = load()
    pc = _flat(chunk_states, "chunk_states", F32, dev, (lib.ssm_selective_scan_chunks(n, T), channels, N))
    table = _table(seq_starts, seq_lens, resume_flags, dev)
    pgs = _optional(grad_state, "grad_state", dev, (n, channels, N))
    for given, grad, name in ((D, grad_D, "grad_D"), (z, grad_z, "grad_z"), (dt_bias, grad_dt_bias, "grad_dt_bias")):
        if given is None and grad is not None:
            raise ValueError(f"{name} needs {name[5:]}")
    handle = _raw_stream(dev.index)
    grad_x, qx, tx = _rows_out(grad_x, "grad_x", dtype, dev, x.shape)
    grad_dt, qdt, tdt = _rows_out(grad_dt, "grad_dt", dtype, dev, x.shape)
    grad_B, qB, tB = _rows_out(grad_B, "grad_B", dtype, dev, (T, n_groups * N))
    grad_C, qC, tC = _rows_out(grad_C, "grad_C", dtype, dev, (T, n_groups * N))
    grad_A, qA = _flat_out(grad_A, "grad_A", F32, dev, (channels, N))
    qD, qz, tz, qb = None, None, 0, None
    if D is not None:
        grad_D, qD = _flat_out(grad_D, "grad_D", F32, dev, (channels,))
    if z is not None:
        grad_z, qz, tz = _rows_out(grad_z, "grad_z", dtype, dev, x.shape)
    if dt_bias is not None:
        grad_dt_bias, qb = _flat_out(grad_dt_bias, "grad_dt_bias", F32, dev, (channels,))
    grad_initial_state, q0 = _flat_out(grad_initial_state, "grad_initial_state", F32, dev, (n, channels, N))
    ws, nb, workspace = _workspace(workspace, lib.ssm_selective_scan_backward_workspace_bytes(n, T, channels, N, n_groups), dev)
    rc = lib.ssm_selective_scan_backward(pg, pgs, *p, 1 if dt_softplus else 0, pc, *table, n, T, channels, N, n_groups, code,
                                         sg, *s, qx, qdt, qA, qB, qC, qD, qz, qb, q0, tx, tdt, tB, tC, tz, ws, nb, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_selective_scan_backward")
    return grad_x, grad_dt, grad_A, grad_B, grad_C, grad_D, grad_z, grad_dt_bias, grad_initial_state


# ---- short causal convolution ----


def _conv_sizes(x, weight):
    code = _dtype(x, "x")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise TypeError("weight must be a 2-dimensional torch.Tensor [channels, kernel_size]")
    T, channels = x.shape
    return code, x.device, T, channels, weight.shape[1]


@_placed
def ssm_causal_conv(x, weight, conv_state, seq_starts, seq_lens, resume_flags, out=None, *, bias=None, silu=True):
    """Short causal convolution (``ssm_causal_conv``): ``ssm_conv1d`` for x [T, C] fp32, bf16 or fp16 with strided rows.

    weight [C, K] fp32 (K at most 8), conv_state [n, C, K-1] fp32 (updated in place), bias [C] fp32 or None;
    silu=False leaves the activation out.  Returns out [T, C] (allocated if not given)."""
    code, dev, T, channels, K = _conv_sizes(x, weight)
    n = seq_lens.shape[0]
    px, sx = _rows(x, "x", x.dtype, dev, x.shape)
    pw = _flat(weight, "weight", F32, dev, (channels, K))
    slots = _flat(conv_state, "conv_state", F32, dev, (n, channels, K - 1))
    pb = _optional(bias, "bias", dev, (channels,))
    table = _table(seq_starts, seq_lens, resume_flags, dev)
    handle = _raw_stream(dev.index)
    out, po, so = _rows_out(out, "out", x.dtype, dev, x.shape)
    rc = load().ssm_causal_conv(px, pw, pb, slots or None, po, *table, n, T, channels, K, 1 if silu else 0, code, sx, so, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_causal_conv")
    return out


def causal_conv_backward_workspace_bytes(n_seqs, n_tokens, channels, kernel_size) -> int:
    """Bytes of workspace of ``ssm_causal_conv_backward``."""
    return int(load().ssm_causal_conv_backward_workspace_bytes(int(n_seqs), int(n_tokens), int(channels), int(kernel_size)))


@_placed
def ssm_causal_conv_backward(grad_out, x, weight, seq_starts, seq_lens, resume_flags=None, *, bias=None, silu=True,
                             initial_state=None, grad_state=None, grad_x=None, grad_weight=None, grad_bias=None,
                             grad_initial_state=None, workspace=None):
    """Gradients of ``ssm_causal_conv`` (``ssm_causal_conv_backward``).  initial_state [n, C, K-1] fp32: what the
    slots held before the forward call, with resume_flags; without both every sequence was fresh.  grad_state: the
    gradient of the slots after the call, or None.  Outputs are allocated if not given.  Returns (grad_x [T, C],
    grad_weight [C, K] fp32, grad_bias [C] fp32 or None without bias, grad_initial_state, None without initial_state)."""
    code, dev, T, channels, K = _conv_sizes(x, weight)
    if not isinstance(seq_lens, torch.Tensor):
        raise TypeError("seq_lens must be a torch.Tensor")
    n, slots = seq_lens.shape[0], (seq_lens.shape[0], channels, K - 1)
    if (initial_state is None) != (resume_flags is None):
        raise ValueError("initial_state and resume_flags go together: without them every sequence is fresh")
    if bias is None and grad_bias is not None:
        raise ValueError("grad_bias needs bias")
    if initial_state is None and grad_initial_state is not None:
        raise ValueError("grad_initial_state needs initial_state")
    pg, sg = _rows(grad_out, "grad_out", x.dtype, dev, x.shape)
    px, sx = _rows(x, "x", x.dtype, dev, x.shape)
    pw = _flat(weight, "weight", F32, dev, (channels, K))
    pb = _optional(bias, "bias", dev, (channels,))
    ps, pl = _flat(seq_starts, "seq_starts", I32, dev, (n,)), _flat(seq_lens, "seq_lens", I32, dev, (n,))
    p0, pr = _optional(initial_state, "initial_state", dev, slots), None
    if resume_flags is not None:
        pr = _flat(resume_flags, "resume_flags", I32, dev, (n,))
    pgs = _optional(grad_state, "grad_state", dev, slots)
    lib = load()
    handle = _raw_stream(dev.index)
    grad_x, qx, tx = _rows_out(grad_x, "grad_x", x.dtype, dev, x.shape)
    grad_weight, qw = _flat_out(grad_weight, "grad_weight", F32, dev, (channels, K))
    qb, q0 = None, None
    if bias is not None:
        grad_bias, qb = _flat_out(grad_bias, "grad_bias", F32, dev, (channels,))
    if initial_state is not None:
        grad_initial_state, q0 = _flat_out(grad_initial_state, "grad_initial_state", F32, dev, slots)
    ws, nb, workspace = _workspace(workspace, lib.ssm_causal_conv_backward_workspace_bytes(n, T, channels, K), dev)
    rc = lib.ssm_causal_conv_backward(pg, pgs or None, px, pw, pb, p0 or None, ps, pl, pr, n, T, channels, K, 1 if silu else 0,
                                      code, sg, sx, qx, qw, qb, q0 or None, tx, ws, nb, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_causal_conv_backward")
    return grad_x, grad_weight, grad_bias, grad_initial_state


# ---- cross entropy of a projection onto a large vocabulary ----


def linear_cross_entropy_workspace_bytes(hidden, weight, *, backward=False) -> int:
    """Bytes of workspace of ``ssm_linear_cross_entropy``, or of its backward pass, for these operands (the weight's
    address and stride count)."""
    for t, name in ((hidden, "hidden"), (weight, "weight")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise TypeError(f"{name} must be a 2-dimensional torch.Tensor")
    rows, width = hidden.shape
    pw, sw = _rows(weight, "weight", hidden.dtype, hidden.device, (weight.shape[0], width))
    return int(load().ssm_linear_cross_entropy_workspace_bytes(pw, rows, weight.shape[0], width, sw, 1 if backward else 0))


def _loss_inputs(hidden, weight, targets):
    code = _dtype(hidden, "hidden")
    dev, dtype = hidden.device, hidden.dtype
    if dtype == F32:
        raise TypeError("hidden must be bfloat16 or float16, got torch.float32")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise TypeError("weight must be a 2-dimensional torch.Tensor [vocab, width]")
    T, D = hidden.shape
    V = weight.shape[0]
    ph, sh = _rows(hidden, "hidden", dtype, dev, (T, D))
    pw, sw = _rows(weight, "weight", dtype, dev, (V, D))
    if not isinstance(targets, torch.Tensor) or targets.dtype not in (torch.int64, I32):
        raise TypeError("targets must be an int64 or int32 torch.Tensor")
    pt = _flat(targets, "targets", targets.dtype, dev, (T,))
    return code, dev, T, V, D, ph, sh, pw, sw, pt, 1 if targets.dtype == torch.int64 else 0


@_placed
def ssm_linear_cross_entropy(hidden, weight, targets, *, ignore_index=-100, loss=None, lse=None, workspace=None):
    """Softmax cross entropy of the logits hidden weight^T, which are not kept (``ssm_linear_cross_entropy``).

    hidden [T, D] and weight [V, D] bf16 or fp16, targets [T] int64 or int32.  Returns (loss [T], lse [T]) fp32:
    loss = lse - the target's logit, lse the log of the sum of the logits' exponentials; both 0 where the target is
    ignore_index."""
    code, dev, T, V, D, ph, sh, pw, sw, pt, wide = _loss_inputs(hidden, weight, targets)
    lib = load()
    handle = _raw_stream(dev.index)
    loss, pl = _flat_out(loss, "loss", F32, dev, (T,))
    lse, pe = _flat_out(lse, "lse", F32, dev, (T,))
    ws, nb, workspace = _workspace(workspace, lib.ssm_linear_cross_entropy_workspace_bytes(pw, T, V, D, sw, 0), dev)
    rc = lib.ssm_linear_cross_entropy(ph, pw, pt, wide, int(ignore_index), pl, pe, T, V, D, code, sh, sw, ws, nb, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_linear_cross_entropy")
    return loss, lse


@_placed
def ssm_linear_cross_entropy_backward(grad_loss, hidden, weight, targets, lse, *, ignore_index=-100, grad_hidden=None,
                                      grad_weight=None, need_weight=True, workspace=None):
    """Gradients of ``ssm_linear_cross_entropy``'s loss (``ssm_linear_cross_entropy_backward``): grad_loss [T] fp32, lse as
    the forward call returned it.  need_weight=False leaves the weight's gradient out (a frozen projection).
    Returns (grad_hidden [T, D], grad_weight [V, D] or None), both in hidden's type (allocated if not given)."""
    code, dev, T, V, D, ph, sh, pw, sw, pt, wide = _loss_inputs(hidden, weight, targets)
    pg, pe = _flat(grad_loss, "grad_loss", F32, dev, (T,)), _flat(lse, "lse", F32, dev, (T,))
    if not need_weight and grad_weight is not None:
        raise ValueError("grad_weight is given but need_weight is False")
    lib = load()
    handle = _raw_stream(dev.index)
    grad_hidden, qh, th = _rows_out(grad_hidden, "grad_hidden", hidden.dtype, dev, (T, D))
    qw, tw = None, 0
    if need_weight:
        grad_weight, qw, tw = _rows_out(grad_weight, "grad_weight", hidden.dtype, dev, (V, D))
    ws, nb, workspace = _workspace(workspace, lib.ssm_linear_cross_entropy_workspace_bytes(pw, T, V, D, sw, 1), dev)
    rc = lib.ssm_linear_cross_entropy_backward(pg, ph, pw, pt, wide, int(ignore_index), pe, qh, qw, T, V, D, code, sh, sw, th, tw,
                                               ws, nb, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_linear_cross_entropy_backward")
    return grad_hidden, grad_weight
