"""ctypes binding of the layer operators around the scan (argument marshalling only).

The gated linear recurrence, the RMS norm with the residual's addition, the row
quantiser and the 8-bit integer matrix product of ``libssmscan.so`` on torch
tensors.  Every function runs on the current CUDA stream of its tensors' device,
or on its keyword argument ``stream``; what it allocates (outputs not given, workspaces) belongs to
that stream.  Tensors are [rows, width] with contiguous rows; rows may be further
apart than their width (slices of a wider tensor).  Formulas and rules are those
of ``include/ssmscan.h``.

No function here is recorded by torch's autograd: outputs never require a gradient, also where an
input does, so a training step calls the backward functions itself (as ``examples/gated_layer.py``
does).  A ``workspace=`` that is given has to hold at least what the operator's
``..._workspace_bytes`` says; calls that overlap on the GPU need one each.
"""
from __future__ import annotations

import contextlib
import functools
import inspect

import torch

from .binding import SSM_OK, SsmScanError, load

# torch's own short ways to the current device and stream (a stream object takes 2 us to make)
_current_device = getattr(torch._C, "_cuda_getDevice", lambda: -2)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0)

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _bad(t, name, dtype, dev, shape):
    """Why `t` is not a tensor of this type, device and shape with contiguous rows."""
    if not isinstance(t, torch.Tensor):
        return TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        return TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        return ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.shape != shape:
        return ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return ValueError(f"{name} must have contiguous rows that do not overlap, got strides {t.stride()}")


def _rows(t, name, dtype, dev, shape):
    """(pointer, row stride) of a checked [rows, width] tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev or t.shape != shape:
        raise _bad(t, name, dtype, dev, shape)
    s0, s1 = t.stride()
    if s1 != 1 or s0 < shape[1]:
        rows, width = shape
        if rows <= 1:
            s0 = max(s0, width)                   # a single row's stride says nothing
        if (s1 != 1 and width > 1) or s0 < width:
            raise _bad(t, name, dtype, dev, shape)
    return t.data_ptr(), s0


def _flat(t, name, dtype, dev, shape):
    """Pointer of a checked contiguous tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev or t.shape != shape or not t.is_contiguous():
        raise _bad(t, name, dtype, dev, shape)
    return t.data_ptr()


def _dtype(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("the operators run on CUDA tensors only")
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, width], got {t.dim()} dimensions")
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return code


@contextlib.contextmanager
def _on(dev, stream):
    """The tensors' device and the launching stream made current: what is allocated inside belongs
    to that stream."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        with torch.cuda.stream(stream):
            yield


def _placed(fn):
    """Adds ``stream=None`` to an operator whose first argument says the device: the call itself runs
    with that device and stream current."""
    name = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if (not isinstance(first, torch.Tensor) or not first.is_cuda or
                (stream is None and first.get_device() == _current_device())):
            return fn(*args, **kw)                # (what is no CUDA tensor is refused there)
        with _on(first.device, stream):
            return fn(*args, **kw)
    return call


def _rows_out(t, name, dtype, dev, shape):
    """(tensor, pointer, row stride): `t` checked, or a new tensor."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t, t.data_ptr(), shape[1]
    return (t, *_rows(t, name, dtype, dev, shape))


def _flat_out(t, name, dtype, dev, shape):
    """(tensor, pointer): `t` checked, or a new tensor."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t, t.data_ptr()
    return t, _flat(t, name, dtype, dev, shape)


def _workspace(given, need, dev):
    """(pointer, bytes, tensor to keep): `given` if it is large enough (else an error), or a new one."""
    if given is not None:
        if given.device != dev or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the operator's device")
        return given.data_ptr(), given.numel() * given.element_size(), given
    if need == 0:
        return None, 0, None
    w = torch.empty(need, dtype=torch.uint8, device=dev)
    return w.data_ptr(), need, w


# ---- gated linear recurrence ----


def gated_scan_backward_workspace_bytes(n_seqs, n_tokens, channels) -> int:
    """Bytes of workspace of ``ssm_gated_scan_backward``."""
    return int(load().ssm_gated_scan_backward_workspace_bytes(int(n_seqs), int(n_tokens), int(channels)))


def gated_scan_chunk_states(n_seqs, n_tokens, channels, device="cuda"):
    """An empty chunk_states tensor [chunks, channels] fp32 for these sizes."""
    chunks = int(load().ssm_gated_scan_chunks(int(n_seqs), int(n_tokens), int(channels)))
    return torch.empty((chunks, int(channels)), dtype=torch.float32, device=device)


@_placed
def ssm_gated_scan(state_slots, x, gate_a, gate_x, lam, seq_starts, seq_lens, resume_flags, y=None, *,
                   decay_scale=8.0, chunk_states=None):
    """Gated linear recurrence (``ssm_gated_scan``): with r = sigmoid(gate_a), i = sigmoid(gate_x),
    a = exp(-decay_scale softplus(lam) r),

        h_t = a h_{t-1} + sqrt(1 - a^2) i x_t,   y_t = h_t

    at every token, a fresh sequence's first one too.
    state_slots [n, C] fp32 (updated in place); x, gate_a, gate_x [T, C] fp32, bf16 or fp16 (slices
    of one projection are fine); lam [C] fp32; seq_starts, seq_lens, resume_flags [n] int32.
    chunk_states: a tensor of ``gated_scan_chunk_states`` to fill for the backward pass.
    Returns y [T, C] (allocated if not given)."""
    code = _dtype(x, "x")
    dev, shape, dt = x.device, x.shape, x.dtype
    T, C = shape
    n = seq_lens.shape[0]
    f32, i32, one = torch.float32, torch.int32, (n,)
    px, sx = _rows(x, "x", dt, dev, shape)
    pa, sa = _rows(gate_a, "gate_a", dt, dev, shape)
    pg, sg = _rows(gate_x, "gate_x", dt, dev, shape)
    slots = _flat(state_slots, "state_slots", f32, dev, (n, C))
    plam = _flat(lam, "lam", f32, dev, (C,))
    ps, pl, pr = (_flat(seq_starts, "seq_starts", i32, dev, one), _flat(seq_lens, "seq_lens", i32, dev, one),
                  _flat(resume_flags, "resume_flags", i32, dev, one))
    lib = load()
    pc = None
    if chunk_states is not None:
        pc = _flat(chunk_states, "chunk_states", f32, dev, (lib.ssm_gated_scan_chunks(n, T, C), C))
    handle = _raw_stream(dev.index)
    y, py, sy = _rows_out(y, "y", dt, dev, shape)
    rc = lib.ssm_gated_scan(slots, px, pa, pg, plam, decay_scale, py, ps, pl, pr, n, T, C, code, sx, sa, sg, sy,
                            pc, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_gated_scan")
    return y


@_placed
def ssm_gated_scan_backward(grad_y, x, gate_a, gate_x, lam, chunk_states, seq_starts, seq_lens, resume_flags, *,
                            decay_scale=8.0, grad_state=None, grad_x=None, grad_gate_a=None, grad_gate_x=None,
                            grad_lam=None, grad_initial_state=None, workspace=None):
    """Gradients of ``ssm_gated_scan`` (``ssm_gated_scan_backward``) from the gradient of y and
    optionally of the slots after the call (grad_state [n, C] fp32); chunk_states as filled by the
    forward call.  Outputs are allocated if not given.  Returns
    (grad_x, grad_gate_a, grad_gate_x, grad_lam, grad_initial_state)."""
    code = _dtype(x, "x")
    dev, shape, dt = x.device, x.shape, x.dtype
    T, C = shape
    n = seq_lens.shape[0]
    f32, i32, one = torch.float32, torch.int32, (n,)
    px, sx = _rows(x, "x", dt, dev, shape)
    pa, sa = _rows(gate_a, "gate_a", dt, dev, shape)
    pg, sg = _rows(gate_x, "gate_x", dt, dev, shape)
    py, sy = _rows(grad_y, "grad_y", dt, dev, shape)
    lib = load()
    pc = _flat(chunk_states, "chunk_states", f32, dev, (lib.ssm_gated_scan_chunks(n, T, C), C))
    plam = _flat(lam, "lam", f32, dev, (C,))
    ps, pl, pr = (_flat(seq_starts, "seq_starts", i32, dev, one), _flat(seq_lens, "seq_lens", i32, dev, one),
                  _flat(resume_flags, "resume_flags", i32, dev, one))
    pgs = None if grad_state is None else _flat(grad_state, "grad_state", f32, dev, (n, C))
    handle = _raw_stream(dev.index)
    grad_x, qx, tx = _rows_out(grad_x, "grad_x", dt, dev, shape)
    grad_gate_a, qa, ta = _rows_out(grad_gate_a, "grad_gate_a", dt, dev, shape)
    grad_gate_x, qg, tg = _rows_out(grad_gate_x, "grad_gate_x", dt, dev, shape)
    grad_lam, ql = _flat_out(grad_lam, "grad_lam", f32, dev, (C,))
    grad_initial_state, q0 = _flat_out(grad_initial_state, "grad_initial_state", f32, dev, (n, C))
    ws, nb, workspace = _workspace(workspace, lib.ssm_gated_scan_backward_workspace_bytes(n, T, C), dev)
    rc = lib.ssm_gated_scan_backward(py, pgs, px, pa, pg, plam, decay_scale, pc, ps, pl, pr, n, T, C, code,
                                     sx, sa, sg, sy, qx, qa, qg, tx, ta, tg, ql, q0, ws, nb, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_gated_scan_backward")
    return grad_x, grad_gate_a, grad_gate_x, grad_lam, grad_initial_state


# ---- RMS norm with the residual's addition; row quantiser ----


@_placed
def ssm_add_norm(x, weight, residual=None, *, eps=1e-6, quant=None, residual_out=None, out=None, scales=None):
    """RMS norm with the residual's addition (``ssm_add_norm``): h = x + residual in the residual's
    type, y = h / sqrt(mean(h^2) + eps) * weight per row.

    x [T, D] fp32, bf16 or fp16; weight [D] fp32; residual [T, D] of x's type or fp32, or None
    (h = x).  residual_out: where h goes (allocated if not given; residual itself is fine).
    Returns (y, h), or with quant="int8" (codes int8, scales [T] fp32, h), codes * scales being y.
    h is x when there is no residual."""
    code = _dtype(x, "x")
    dev, shape, dt = x.device, x.shape, x.dtype
    T, D = shape
    if quant not in (None, "int8"):
        raise ValueError(f"quant must be None or 'int8', got {quant!r}")
    px, sx = _rows(x, "x", dt, dev, shape)
    pw = _flat(weight, "weight", torch.float32, dev, (D,))
    pr, sr, rdt, rcode = None, 0, dt, code
    if residual is not None:
        rdt, rcode = residual.dtype, _dtype(residual, "residual")
        pr, sr = _rows(residual, "residual", rdt, dev, shape)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    handle = _raw_stream(dev.index)
    ph, sh, h = None, 0, x
    if residual is not None:
        h, ph, sh = _rows_out(residual_out, "residual_out", rdt, dev, shape)
    py, pc, ps = None, None, None
    if quant is None:
        out, py, so = _rows_out(out, "out", dt, dev, shape)
    else:
        out, pc, so = _rows_out(out, "out", torch.int8, dev, shape)
        scales, ps = _flat_out(scales, "scales", torch.float32, dev, (T,))
    rc = load().ssm_add_norm(px, pr, pw, eps, ph, py, pc, ps, T, D, code, rcode, sx, sr, sh, so, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_add_norm")
    return (out, h) if quant is None else (out, scales, h)


def add_norm_backward_workspace_bytes(rows, width) -> int:
    """Bytes of workspace of ``ssm_add_norm_backward``."""
    return int(load().ssm_add_norm_backward_workspace_bytes(int(rows), int(width)))


@_placed
def ssm_add_norm_backward(grad_y, h, weight, *, grad_h=None, eps=1e-6, grad_in=None, grad_weight=None, workspace=None):
    """Gradient of ``ssm_add_norm`` (``ssm_add_norm_backward``): grad_y [T, D] in y's type, h as the
    forward call returned it, grad_h (h's type) the gradient that reaches h from elsewhere.
    Returns (grad_in [T, D] in h's type: the gradient of x and of residual alike, grad_weight [D] fp32)."""
    code, hcode = _dtype(grad_y, "grad_y"), _dtype(h, "h")
    dev, shape, dt, hdt = grad_y.device, grad_y.shape, grad_y.dtype, h.dtype
    T, D = shape
    pg, sg = _rows(grad_y, "grad_y", dt, dev, shape)
    ph, sh = _rows(h, "h", hdt, dev, shape)
    pw = _flat(weight, "weight", torch.float32, dev, (D,))
    pr, sr = (None, 0) if grad_h is None else _rows(grad_h, "grad_h", hdt, dev, shape)
    lib = load()
    handle = _raw_stream(dev.index)
    grad_in, pi, si = _rows_out(grad_in, "grad_in", hdt, dev, shape)
    grad_weight, pq = _flat_out(grad_weight, "grad_weight", torch.float32, dev, (D,))
    ws, nb, workspace = _workspace(workspace, lib.ssm_add_norm_backward_workspace_bytes(T, D), dev)
    rc = lib.ssm_add_norm_backward(pg, ph, pw, eps, pr, pi, pq, T, D, code, hcode, sg, sh, sr, si, ws, nb, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_add_norm_backward")
    return grad_in, grad_weight


@_placed
def ssm_quantize_rows(x, codes=None, scales=None):
    """Rows in 8 bits with a scale each (``ssm_quantize_rows``): x [T, D] fp32, bf16 or fp16.
    Returns (codes [T, D] int8, scales [T] fp32), codes * scales being x to half a step."""
    code = _dtype(x, "x")
    dev, shape = x.device, x.shape
    T, D = shape
    px, sx = _rows(x, "x", x.dtype, dev, shape)
    handle = _raw_stream(dev.index)
    codes, pc, sc = _rows_out(codes, "codes", torch.int8, dev, shape)
    scales, ps = _flat_out(scales, "scales", torch.float32, dev, (T,))
    rc = load().ssm_quantize_rows(px, pc, ps, T, D, code, sx, sc, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_quantize_rows")
    return codes, scales


# ---- 8-bit integer matrix product ----


def int8_matmul_workspace_bytes(x, w) -> int:
    """Bytes of workspace of ``ssm_int8_matmul`` for these operands (their addresses and strides count; 0: none)."""
    for t, name in ((x, "x"), (w, "w")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise TypeError(f"{name} must be a 2-dimensional torch.Tensor")
    px, sx = _rows(x, "x", torch.int8, x.device, x.shape)
    pw, sw = _rows(w, "w", torch.int8, x.device, (w.shape[0], x.shape[1]))
    return int(load().ssm_int8_matmul_workspace_bytes(px, pw, x.shape[0], w.shape[0], x.shape[1], sx, sw))


@_placed
def ssm_int8_matmul(x, x_scales, w, w_scales, *, bias=None, out=None, out_dtype=torch.bfloat16, workspace=None):
    """8-bit integer matrix product (``ssm_int8_matmul``):
    out[t, n] = (sum_k x[t, k] w[n, k]) x_scales[t] w_scales[n] + bias[n].

    x [T, K] and w [N, K] int8, x_scales [T], w_scales [N] and bias [N] fp32.  Returns out [T, N]
    (out_dtype fp32, bf16 or fp16; allocated if not given)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise TypeError("x and w must be 2-dimensional torch.Tensors")
    dev, i8, f32 = x.device, torch.int8, torch.float32
    if dev.type != "cuda":
        raise ValueError("the operators run on CUDA tensors only")
    T, K = x.shape
    N = w.shape[0]
    if out is not None:
        out_dtype = out.dtype
    code = DTYPES.get(out_dtype)
    if code is None:
        raise TypeError(f"out must be float32, bfloat16 or float16, got {out_dtype}")
    px, sx = _rows(x, "x", i8, dev, x.shape)
    pw, sw = _rows(w, "w", i8, dev, (N, K))
    pxs, pws = _flat(x_scales, "x_scales", f32, dev, (T,)), _flat(w_scales, "w_scales", f32, dev, (N,))
    pb = None if bias is None else _flat(bias, "bias", f32, dev, (N,))
    lib = load()
    handle = _raw_stream(dev.index)
    out, po, so = _rows_out(out, "out", out_dtype, dev, (T, N))
    ws, nb, workspace = _workspace(workspace, lib.ssm_int8_matmul_workspace_bytes(px, pw, T, N, K, sx, sw), dev)
    rc = lib.ssm_int8_matmul(px, pxs, pw, pws, pb, po, T, N, K, code, sx, sw, so, ws, nb, handle)
    if rc != SSM_OK:
        raise SsmScanError(rc, "ssm_int8_matmul")
    return out
