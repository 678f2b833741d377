"""The operators of a selective-scan model in plain float64 NumPy (no code shared with the CUDA path):
the selective scan with a decay for each channel and state, the short causal convolution, and the
cross entropy of a projection, with their gradients.  Written token by token from the definitions;
tokens that belong to no sequence are NaN in the outputs.
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(over="ignore"):
        e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def step_of(dt, dt_bias, softplus):
    """(v, step, d step / d v)."""
    v = np.asarray(dt, dtype=np.float64) + (0.0 if dt_bias is None else np.asarray(dt_bias, dtype=np.float64))
    if not softplus:
        return v, v, np.ones_like(v)
    with np.errstate(over="ignore"):
        step = np.where(v > 20, v, np.log1p(np.exp(np.minimum(v, 20.0))))
    return v, step, np.where(v > 20, 1.0, sigmoid(v))


def _groups(rows, channels, groups):
    """[T, G N] as [T, C, N]."""
    T = rows.shape[0]
    r = np.asarray(rows, dtype=np.float64).reshape(T, groups, -1)
    return np.repeat(r, channels // groups, axis=1)


def selective_scan(slots, x, dt, A, B, C, D, starts, lens, resume, z=None, dt_bias=None, softplus=False, groups=1):
    """(y, slots after, states before every token {sequence: [len, C, N]})."""
    x, A = np.asarray(x, dtype=np.float64), np.asarray(A, dtype=np.float64)
    T, channels = x.shape
    _, step, _ = step_of(dt, dt_bias, softplus)
    Bc, Cc = _groups(B, channels, groups), _groups(C, channels, groups)
    d = np.zeros(channels) if D is None else np.asarray(D, dtype=np.float64)
    y, out, before = np.full_like(x, np.nan), np.zeros((len(lens),) + A.shape), {}
    for k, (s, n) in enumerate(zip(starts, lens)):
        h = np.asarray(slots[k], dtype=np.float64).copy() if resume[k] else np.zeros(A.shape)
        before[k] = np.zeros((n,) + A.shape)
        for t in range(s, s + n):
            before[k][t - s] = h
            h = np.exp(step[t][:, None] * A) * h + (step[t] * x[t])[:, None] * Bc[t]
            y[t] = (h * Cc[t]).sum(1) + d * x[t]
            if z is not None:
                y[t] *= z[t] * sigmoid(z[t])
        out[k] = h
    return y, out, before


def selective_scan_backward(grad_y, grad_state, slots, x, dt, A, B, C, D, starts, lens, resume, z=None, dt_bias=None,
                            softplus=False, groups=1):
    """Gradients by name: x, dt, A, B, C, D, z, dt_bias, initial_state."""
    x, A, grad_y = (np.asarray(v, dtype=np.float64) for v in (x, A, grad_y))
    T, channels = x.shape
    N = A.shape[1]
    _, step, slope = step_of(dt, dt_bias, softplus)
    Bc, Cc = _groups(B, channels, groups), _groups(C, channels, groups)
    d = np.zeros(channels) if D is None else np.asarray(D, dtype=np.float64)
    _, _, before = selective_scan(slots, x, dt, A, B, C, D, starts, lens, resume, None, dt_bias, softplus, groups)
    g = {k: np.full_like(x, np.nan) for k in ("x", "dt", "z")}
    g.update({k: np.full((T, groups * N), np.nan) for k in ("B", "C")})
    g.update(A=np.zeros_like(A), D=np.zeros(channels), dt_bias=np.zeros(channels), initial_state=np.zeros((len(lens),) + A.shape))
    for k, (s, n) in enumerate(zip(starts, lens)):
        e = np.zeros(A.shape) if grad_state is None else np.asarray(grad_state[k], dtype=np.float64).copy()
        for t in range(s + n - 1, s - 1, -1):
            decay = np.exp(step[t][:, None] * A)
            kept = decay * before[k][t - s]
            h = kept + (step[t] * x[t])[:, None] * Bc[t]
            p = (h * Cc[t]).sum(1) + d * x[t]
            gp = grad_y[t]
            if z is not None:
                sg = sigmoid(z[t])
                g["z"][t] = grad_y[t] * p * sg * (1 + z[t] * (1 - sg))
                gp = grad_y[t] * z[t] * sg
            e = e + gp[:, None] * Cc[t]
            eb = (e * Bc[t]).sum(1)
            g["x"][t] = d * gp + step[t] * eb
            g["dt"][t] = ((e * kept * A).sum(1) + x[t] * eb) * slope[t]
            g["A"] += e * kept * step[t][:, None]
            g["D"] += gp * x[t]
            g["dt_bias"] += g["dt"][t]
            g["B"][t] = (e * (step[t] * x[t])[:, None]).reshape(groups, -1, N).sum(1).ravel()
            g["C"][t] = (h * gp[:, None]).reshape(groups, -1, N).sum(1).ravel()
            e = e * decay
        g["initial_state"][k] = e if resume[k] else 0.0
    return g


def causal_conv(x, weight, slots, starts, lens, resume, bias=None, silu=True):
    """(out, slots after, v)."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    T, channels = x.shape
    K = w.shape[1]
    b = np.zeros(channels) if bias is None else np.asarray(bias, dtype=np.float64)
    out, pre, after = np.full_like(x, np.nan), np.full_like(x, np.nan), np.zeros((len(lens), channels, K - 1))
    for k, (s, n) in enumerate(zip(starts, lens)):
        head = np.asarray(slots[k], dtype=np.float64).T if resume is not None and resume[k] else np.zeros((K - 1, channels))
        stream = np.concatenate([head, x[s:s + n]])
        for t in range(n):
            v = b + sum(w[:, u] * stream[t + u] for u in range(K))
            pre[s + t] = v
            out[s + t] = v * sigmoid(v) if silu else v
        after[k] = stream[n:].T
    return out, after, pre


def causal_conv_backward(grad_out, grad_state, x, weight, slots, starts, lens, resume, bias=None, silu=True):
    """Gradients by name: x, weight, bias, initial_state."""
    x, w, grad_out = (np.asarray(v, dtype=np.float64) for v in (x, weight, grad_out))
    T, channels = x.shape
    K = w.shape[1]
    _, _, pre = causal_conv(x, weight, slots, starts, lens, resume, bias, silu)
    g = dict(x=np.full_like(x, np.nan), weight=np.zeros_like(w), bias=np.zeros(channels),
             initial_state=np.zeros((len(lens), channels, K - 1)))
    for k, (s, n) in enumerate(zip(starts, lens)):
        resumed = resume is not None and resume[k]
        head = np.asarray(slots[k], dtype=np.float64).T if resumed else np.zeros((K - 1, channels))
        stream = np.concatenate([head, x[s:s + n]])
        gs = np.zeros_like(stream)
        if grad_state is not None:
            gs[n:] = np.asarray(grad_state[k], dtype=np.float64).T
        for t in range(n):
            gv = grad_out[s + t]
            if silu:
                sg = sigmoid(pre[s + t])
                gv = gv * (sg + pre[s + t] * sg * (1 - sg))
            g["bias"] += gv
            for u in range(K):
                gs[t + u] += w[:, u] * gv
                g["weight"][:, u] += gv * stream[t + u]
        g["x"][s:s + n] = gs[K - 1:]
        if resumed:
            g["initial_state"][k] = gs[:K - 1].T
    return g


def linear_cross_entropy(hidden, weight, targets, ignore_index=-100):
    """(loss, lse) of every row; 0 where it is ignored."""
    h, w = np.asarray(hidden, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    loss, lse = np.zeros(len(h)), np.zeros(len(h))
    for t, v in enumerate(targets):
        if v == ignore_index:
            continue
        logits = w @ h[t]
        top = logits.max()
        lse[t] = top + np.log(np.exp(logits - top).sum())
        loss[t] = lse[t] - logits[v] if 0 <= v < len(w) else np.nan
    return loss, lse


def linear_cross_entropy_backward(grad_loss, hidden, weight, targets, ignore_index=-100):
    """(grad_hidden, grad_weight, G): G [T, V] the gradient of the logits."""
    h, w = np.asarray(hidden, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    G = np.zeros((len(h), len(w)))
    for t, v in enumerate(targets):
        if v == ignore_index:
            continue
        logits = w @ h[t]
        p = np.exp(logits - logits.max())
        G[t] = p / p.sum() * grad_loss[t]
        G[t, v] -= grad_loss[t]
    hz = np.where((np.asarray(targets) != ignore_index)[:, None], h, 0.0)
    return G @ w, G.T @ hz, G
