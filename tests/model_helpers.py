"""Error bounds of the selective-scan model's operators on the GPU, from the count of roundings (u = 2^-24
for one to fp32).

Hardware 2^x and 1/x: 4u and 2u (2 ulp, 1 ulp).  exp(w) as 2^(w log2 e): the constant's and the product's
rounding move the argument by 2|w|u, so exp is within (2|w| + 4)u.
 * sigmoid(v) = 1 / (1 + exp(-v)): (2|v| + 8)u.
 * step = softplus(v): v's own rounding |v|u, e = exp(-|v|), a quotient (5u), a series (4u) and three
   roundings: (3|v| + 18)u relative; without softplus the sum's u.
 * decay = 2^(step A log2 e): with X = |step A|, the exponent's relative error (the step's and 3u) times X, and 4u.
   Where a sequence is cut into segments, a segment's whole decay comes from the sum of its steps, whose
   rounding is at most one u a token relative: n X u more, n the sequence's length.
 * states and their gradients follow their recurrences with 4u a step; sums over N states or n tokens add a u a
   term (in whatever order), sums over channels 24u (four channels in a lane, five exchanges, four warps, up to
   eleven blocks; `blocks` says if there are more).
The tensor cores add products in fp32 with truncation: 2u of the sum of magnitudes a term.
"""
import numpy as np
import torch

from oracle import model as om
from tests.layer_helpers import DTYPES, U, close, half_step, np64, tiny_step  # noqa: F401


def sig_err(v):
    return (2 * np.abs(v) + 8) * U


def _rep(rows, channels, groups):
    return om._groups(rows, channels, groups)


def scan_bounds(slots, x, dt, A, B, C, D, starts, lens, resume, z=None, dt_bias=None, softplus=False, groups=1,
                grad_y=None, grad_state=None, blocks=11):
    """Bounds (float64 arrays by name) of y and the slots, and with grad_y of the gradients."""
    T, channels = x.shape
    N = A.shape[1]
    v, step, slope = om.step_of(dt, dt_bias, softplus)
    # above the threshold the step is v itself; exp(-inf) is exactly 0, and so is the step
    with np.errstate(invalid="ignore"):
        es = np.where(v > 20, 2 * U, np.where(np.isinf(v), 0.0, (3 * np.abs(v) + 18) * U)) if softplus else np.full_like(v, 2 * U)
    Ba, Ca = np.abs(_rep(B, channels, groups)), np.abs(_rep(C, channels, groups))
    d = np.zeros(channels) if D is None else np.abs(D)
    sg = om.sigmoid(z) if z is not None else None
    gate = np.abs(z * sg) if z is not None else np.ones_like(x)
    over = (15 + blocks) * U                                  # a sum over channels
    eg = sig_err(z) + 4 * U if z is not None else np.zeros_like(x)
    u, ax = np.abs(step * x), np.abs(x)
    out = {"y": np.zeros_like(x), "slots": np.zeros((len(lens),) + A.shape)}
    back = grad_y is not None
    if back:
        gp = np.abs(grad_y) * gate
        for k in ("grad_x", "grad_dt", "grad_z"):
            out[k] = np.zeros_like(x)
        for k in ("grad_B", "grad_C"):
            out[k] = np.zeros((T, groups * N))
        gA_m, out["grad_A"] = np.zeros_like(A), np.zeros_like(A)
        gD_m, out["grad_D"] = np.zeros(channels), np.zeros(channels)
        gb_m, out["grad_dt_bias"] = np.zeros(channels), np.zeros(channels)
        out["grad_slots"] = np.zeros((len(lens),) + A.shape)
        eslope = np.where((v > 20) | np.isinf(v), 0.0, (3 * np.abs(v) + 8) * U) if softplus else np.zeros_like(v)

    def fold(m):
        return m.reshape(groups, -1, N).sum(1).ravel()

    for k, (s, n) in enumerate(zip(starts, lens)):
        M = np.abs(slots[k]) if resume[k] else np.zeros(A.shape)
        E = np.zeros(A.shape)
        keep = []
        for t in range(s, s + n):
            X = np.abs(step[t][:, None] * A)
            a = np.exp(step[t][:, None] * A)
            ea = X * (es[t][:, None] + (3 + n) * U) + 4 * U
            b = u[t][:, None] * Ba[t]
            kM, kE = a * M, a * E + a * M * (ea + 2 * U)
            E = kE + 2 * U * kM + (es[t][:, None] + 4 * U) * b
            M = kM + b
            keep.append((a, ea, kM, kE, M, E))
            pm = (M * Ca[t]).sum(1) + d * ax[t]
            pe = (E * Ca[t]).sum(1) + (N + 3) * U * (M * Ca[t]).sum(1) + 2 * U * d * ax[t]
            out["y"][t] = gate[t] * (pe + pm * (eg[t] + 4 * U))
            if back and z is not None:
                sz = sg[t] + np.abs(z[t]) * sg[t] * (1 - sg[t])
                e1 = sig_err(z[t])
                esz = sg[t] * e1 + np.abs(z[t]) * sg[t] * ((1 - sg[t]) * (e1 + 3 * U) + sg[t] * e1 + U)
                out["grad_z"][t] = np.abs(grad_y[t]) * (pe * sz + pm * (esz + 3 * U * sz))
        out["slots"][k] = E
        if not back:
            continue
        eM = np.abs(grad_state[k]) if grad_state is not None else np.zeros(A.shape)
        eE = np.zeros(A.shape)
        for t in range(s + n - 1, s - 1, -1):
            a, ea, kM, kE, hM, hE = keep[t - s]
            g = gp[t][:, None] * Ca[t]
            eE = eE + g * (eg[t][:, None] + 3 * U) + 2 * U * (eM + g)
            eM = eM + g
            st, Aa = np.abs(step[t])[:, None], np.abs(A)
            wM, wE = eM * kM, eM * kE + eE * kM + eE * kE + U * eM * kM
            ebM = (eM * Ba[t]).sum(1)
            ebE = (eE * Ba[t]).sum(1) + (N + 2) * U * ebM
            out["grad_x"][t] = d * gp[t] * (eg[t] + 3 * U) + np.abs(step[t]) * (ebE + ebM * (es[t] + 3 * U))
            gsM = (wM * Aa).sum(1) + ax[t] * ebM
            gsE = (wE * Aa).sum(1) + (N + 6) * U * (wM * Aa).sum(1) + ax[t] * (ebE + 2 * U * ebM)
            out["grad_dt"][t] = slope[t] * (gsE + gsM * (eslope[t] + 3 * U))
            out["grad_A"] += st * (wE + wM * (es[t][:, None] + 2 * U))
            gA_m += st * wM
            out["grad_D"] += gp[t] * ax[t] * (eg[t] + 2 * U)
            gD_m += gp[t] * ax[t]
            out["grad_dt_bias"] += out["grad_dt"][t]
            gb_m += slope[t] * gsM
            ue = u[t][:, None] * eM
            out["grad_B"][t] = fold(u[t][:, None] * eE + ue * (es[t][:, None] + over))
            out["grad_C"][t] = fold(gp[t][:, None] * hE + gp[t][:, None] * hM * (eg[t][:, None] + over))
            eE = a * eE + a * eM * (ea + 2 * U)
            eM = a * eM
        out["grad_slots"][k] = eE if resume[k] else 0.0
    if back:
        out["grad_A"] += (T + 8) * U * gA_m
        out["grad_D"] += (T + 8) * U * gD_m
        out["grad_dt_bias"] += (T + 8) * U * gb_m
    return out


def state_range(slots, x, dt, A, B, C, D, starts, lens, resume, z=None, dt_bias=None, softplus=False, groups=1, grad_y=None,
                grad_state=None):
    """Largest magnitude [n_seqs, C] that a state, its gradient or a product of the two reaches."""
    channels = x.shape[1]
    _, step, _ = om.step_of(dt, dt_bias, softplus)
    Ba, Ca = np.abs(_rep(B, channels, groups)), np.abs(_rep(C, channels, groups))
    gate = np.abs(z * om.sigmoid(z)) if z is not None else np.ones_like(x)
    most = np.zeros((len(lens), channels))
    with np.errstate(over="ignore", invalid="ignore"):
        for k, (s, n) in enumerate(zip(starts, lens)):
            h = np.abs(slots[k]) if resume[k] else np.zeros(A.shape)
            hs = []
            for t in range(s, s + n):
                h = np.exp(step[t][:, None] * A) * h + np.abs(step[t] * x[t])[:, None] * Ba[t]
                hs.append(h)
                most[k] = np.maximum(most[k], (h * Ca[t]).sum(1) + h.max(1))
            if grad_y is None:
                continue
            e = np.abs(grad_state[k]) if grad_state is not None else np.zeros(A.shape)
            for t in range(s + n - 1, s - 1, -1):
                e = e + (np.abs(grad_y[t]) * gate[t])[:, None] * Ca[t]
                most[k] = np.maximum(most[k], (e * (hs[t - s] + 1) * (1 + np.abs(A))).sum(1) * n * (1 + np.abs(step[t])))
                e = e * np.exp(step[t][:, None] * A)
                most[k] = np.maximum(most[k], e.max(1))
    return np.where(np.isfinite(most), most, np.inf)


def conv_bounds(x, weight, slots, starts, lens, resume, bias=None, silu=True, grad_out=None, grad_state=None):
    """Bounds of out, and with grad_out of the gradients."""
    T, channels = x.shape
    K = weight.shape[1]
    w, b = np.abs(weight), 0.0 if bias is None else np.abs(bias)
    _, _, pre = om.causal_conv(x, weight, slots, starts, lens, resume, bias, silu)
    out = {"out": np.zeros_like(x)}
    if grad_out is not None:
        out.update(grad_x=np.zeros_like(x), grad_weight=np.zeros_like(w), grad_bias=np.zeros(channels),
                   grad_slots=np.zeros((len(lens), channels, K - 1)))
        mw, mb = np.zeros_like(w), np.zeros(channels)
    for k, (s, n) in enumerate(zip(starts, lens)):
        resumed = resume is not None and resume[k]
        head = np.abs(slots[k]).T if resumed else np.zeros((K - 1, channels))
        stream = np.concatenate([head, np.abs(x[s:s + n])])
        gsE, gsM = np.zeros_like(stream), np.zeros_like(stream)
        if grad_out is not None and grad_state is not None:
            gsM[n:] = np.abs(grad_state[k]).T
        for t in range(n):
            m = b + sum(w[:, u] * stream[t + u] for u in range(K))
            ev = (K + 2) * U * m
            v = pre[s + t]
            sg, e1 = om.sigmoid(v), sig_err(v)
            out["out"][s + t] = 1.1 * ev + np.abs(v) * sg * (e1 + 3 * U) if silu else ev
            if grad_out is None:
                continue
            go = np.abs(grad_out[s + t])
            if silu:
                sl = np.abs(sg + v * sg * (1 - sg))
                esl = sg * e1 + np.abs(v) * sg * ((1 - sg) * (e1 + 3 * U) + sg * e1 + U) + 0.5 * ev
                gm, ge = go * sl, go * (esl + 2 * U * sl)
            else:
                gm, ge = go, np.zeros(channels)
            out["grad_bias"] += ge
            mb += gm
            for u in range(K):
                gsE[t + u] += w[:, u] * ge
                gsM[t + u] += w[:, u] * gm
                out["grad_weight"][:, u] += ge * stream[t + u]
                mw[:, u] += gm * stream[t + u]
        if grad_out is not None:
            e = gsE + (K + 2) * U * gsM
            out["grad_x"][s:s + n] = e[K - 1:]
            out["grad_slots"][k] = e[:K - 1].T if resumed else 0.0
    if grad_out is not None:
        out["grad_weight"] += (T + 8) * U * mw
        out["grad_bias"] += (T + 8) * U * mb
    return out


def loss_bounds(hidden, weight, targets, ignore, dtype, grad_loss=None):
    """Bounds of loss and lse, and with grad_loss of the gradients."""
    T, D = hidden.shape
    V = weight.shape[0]
    keep = targets != ignore
    h = np.where(keep[:, None], hidden, 0.0)
    mag = np.abs(h) @ np.abs(weight).T
    el = 2 * (D + 8) * U * mag                                            # of a logit
    _, lse = om.linear_cross_entropy(hidden, weight, targets, ignore)
    # exponentials of l - top (2^x of one rounded product and sum), sums of 32, then of the parts, a logarithm
    logits = h @ weight.T
    spread = logits.max(1) - logits.min(1)
    elog = el.max(1) + (2 * spread + 4 + 40 + V / 128 / 32 + 16) * U + 4 * U * np.abs(lse) + 2 * U * np.abs(logits).max(1)
    out = {"lse": np.where(keep, elog, 0.0), "loss": np.where(keep, 2 * elog, 0.0)}
    if grad_loss is None:
        return out
    _, _, G = om.linear_cross_entropy_backward(grad_loss, hidden, weight, targets, ignore)
    p = np.exp(logits - lse[:, None]) * keep[:, None]
    ep = p * (np.exp(el + elog[:, None]) - 1 + (2 * np.abs(logits) + 2 * np.abs(lse)[:, None] + 8) * U) + U
    top = np.abs(grad_loss[keep]).max() if keep.any() else 0.0
    step = tiny_step(dtype) * top / (32768.0 if dtype == torch.float16 else 1.0)
    eG = np.abs(grad_loss)[:, None] * keep[:, None] * ep + (half_step(dtype) + 4 * U) * np.abs(G) * (1 + 1e-2) + step
    eG *= keep[:, None]
    aG = np.abs(G) + eG
    out["grad_hidden"] = eG @ np.abs(weight) + 2 * (V + 8) * U * (aG @ np.abs(weight))
    out["grad_weight"] = eG.T @ np.abs(h) + 2 * (T + 8) * U * (aG.T @ np.abs(h))
    return out
