"""The layer operators around the scan in plain float64 NumPy (no code shared with the CUDA path).

Written token by token and row by row from the definitions; the 8-bit codes are
float32 values by definition (a float32 product, quotient and rounding), the rest
is float64.
"""
from __future__ import annotations

import numpy as np

FLT_MAX = np.finfo(np.float32).max


def sigmoid(v):
    v = np.asarray(v, dtype=np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def softplus(v):
    v = np.asarray(v, dtype=np.float64)
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def gated_gates(x, gate_a, gate_x, lam, decay_scale):
    """(r, i, log a, a, m) of every token and channel."""
    r, i = sigmoid(gate_a), sigmoid(gate_x)
    la = -decay_scale * softplus(lam)[None, :] * r
    return r, i, la, np.exp(la), np.sqrt(-np.expm1(2.0 * la))


def gated_scan(slots, x, gate_a, gate_x, lam, starts, lens, resume, decay_scale):
    """(y, slots after): y is NaN for tokens of no sequence."""
    x = np.asarray(x, dtype=np.float64)
    r, i, la, a, m = gated_gates(x, gate_a, gate_x, lam, decay_scale)
    y, out = np.full_like(x, np.nan), np.zeros((len(lens), x.shape[1]))
    for k, (s, n) in enumerate(zip(starts, lens)):
        h = np.asarray(slots[k], dtype=np.float64).copy() if resume[k] else np.zeros(x.shape[1])
        for t in range(s, s + n):
            h = a[t] * h + m[t] * i[t] * x[t]
            y[t] = h
        out[k] = h
    return y, out


def gated_scan_backward(grad_y, grad_state, slots, x, gate_a, gate_x, lam, starts, lens, resume, decay_scale):
    """(dx, dgate_a, dgate_x, dlam, d slots before); NaN for tokens of no sequence."""
    x, grad_y = np.asarray(x, dtype=np.float64), np.asarray(grad_y, dtype=np.float64)
    r, i, la, a, m = gated_gates(x, gate_a, gate_x, lam, decay_scale)
    y, _ = gated_scan(slots, x, gate_a, gate_x, lam, starts, lens, resume, decay_scale)
    dx, da, dg = (np.full_like(x, np.nan) for _ in range(3))
    drate, d0 = np.zeros(x.shape[1]), np.zeros((len(lens), x.shape[1]))
    for k, (s, n) in enumerate(zip(starts, lens)):
        first = np.asarray(slots[k], dtype=np.float64) if resume[k] else np.zeros(x.shape[1])
        e = np.asarray(grad_state[k], dtype=np.float64) if grad_state is not None else np.zeros(x.shape[1])
        for t in range(s + n - 1, s - 1, -1):
            g = grad_y[t] + e
            before = y[t - 1] if t > s else first
            with np.errstate(divide="ignore", invalid="ignore"):
                slope = np.where(m[t] > 0, a[t] ** 2 / m[t], 0.0)     # -dm / d log a; the gate is shut where m = 0
            dla = g * (a[t] * before - slope * i[t] * x[t])
            dx[t] = g * m[t] * i[t]
            dg[t] = g * m[t] * x[t] * i[t] * (1.0 - i[t])
            da[t] = dla * la[t] * (1.0 - r[t])
            drate += dla * r[t]
            e = a[t] * g
        d0[k] = e if resume[k] else 0.0
    return dx, da, dg, -decay_scale * sigmoid(lam) * drate, d0


def quantize_rows(v):
    """(codes, factor) of float32 rows: factor = min(127 / max|v|, FLT_MAX), codes = rint(v factor), in float32."""
    v = np.asarray(v, dtype=np.float32)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        f = np.minimum(np.float32(127.0) / np.max(np.abs(v), axis=1), FLT_MAX)
        q = np.rint(v * f[:, None])
    return q, f


def add_norm(h, weight, eps):
    """(inv, y) of rows h (the sum, already in the residual's type)."""
    h = np.asarray(h, dtype=np.float64)
    inv = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return inv, h * inv[:, None] * np.asarray(weight, dtype=np.float64)


def add_norm_backward(grad_y, h, weight, grad_h, eps):
    """(grad_in, grad_weight)."""
    h, gy, w = (np.asarray(v, dtype=np.float64) for v in (h, grad_y, weight))
    inv, _ = add_norm(h, w, eps)
    n, gn = h * inv[:, None], gy * w
    gin = inv[:, None] * (gn - n * np.mean(n * gn, axis=1, keepdims=True))
    if grad_h is not None:
        gin = gin + np.asarray(grad_h, dtype=np.float64)
    return gin, np.sum(gy * n, axis=0)


def int8_matmul(x, xs, w, ws, bias):
    acc = np.asarray(x, dtype=np.int64) @ np.asarray(w, dtype=np.int64).T
    out = acc.astype(np.float64) * np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)[None, :]
    return out if bias is None else out + np.asarray(bias, np.float64)[None, :]
