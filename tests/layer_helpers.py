"""Error bounds of the layer operators on the GPU, from the count of fp32 roundings (u = 2^-24 each).

Per gate: __expf carries 2 ulp (4u) and its argument's rounding, 1.5 |v| u, and the
shared reciprocal of four denominators 7 u, so a sigmoid is within (1.5 |v| + 12) u; log a adds softplus and two
products (8 u); a = exp(log a) has |log a| times that plus 6 u; m = sqrt(1 - a^2) has
half the relative error of 1 - a^2: that of 2 log a (series, 2 log a < 1/4) or of a^2
times a^2 / (1 - a^2) <= 3.6 (above), plus 8 u.  The state's error follows the
recurrence; composing chunks adds three roundings to a term, so 4 u a step cover it.
"""
import numpy as np
import torch

from oracle import layers as ol

U = 2.0 ** -24
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dtype):
    """Rounding to `dtype`: half a step relative to the value (zero for fp32: counted with the sums)."""
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def tiny_step(dtype):
    """Absolute error of a rounding below the type's normal range."""
    return {torch.float32: 0.0, torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25}[dtype]


def np64(t):
    return t.detach().double().cpu().numpy()


def gate_errors(gate_a, gate_x, la, a):
    """Relative errors (in units of 1) of r, i, log a, a and m."""
    with np.errstate(invalid="ignore"):
        er = np.where(np.isfinite(gate_a), (1.5 * np.abs(gate_a) + 12) * U, 12 * U)
        ei = np.where(np.isfinite(gate_x), (1.5 * np.abs(gate_x) + 12) * U, 12 * U)
    el = er + 8 * U
    ea = np.abs(la) * (el + 2 * U) + 6 * U
    em = 0.5 * np.maximum(el, np.minimum(3.6, a * a / np.maximum(1 - a * a, 1e-30)) * 2 * ea) + 8 * U
    return er, ei, el, ea, em


def gated_bounds(slots, x, ga, gx, lam, starts, lens, resume, c0, grad_y=None, grad_state=None):
    """Bounds on the fp32 errors of y and the slots, and of the gradients (dict), all float64 arrays."""
    r, i, la, a, m = ol.gated_gates(x, ga, gx, lam, c0)
    er, ei, el, ea, em = gate_errors(ga, gx, la, a)
    b, eb = np.abs(m * i * x), em + ei + 4 * U
    T, C = x.shape
    M, E, M0 = np.zeros((T, C)), np.zeros((T, C)), np.zeros((T, C))     # |h|, its error, |h before|
    E0 = np.zeros((T, C))
    sM, sE = np.zeros((len(lens), C)), np.zeros((len(lens), C))
    for k, (s, n) in enumerate(zip(starts, lens)):
        h = np.abs(slots[k]) if resume[k] else np.zeros(C)
        e = np.zeros(C)
        for t in range(s, s + n):
            M0[t], E0[t] = h, e
            e = a[t] * e + (ea[t] + 4 * U) * a[t] * h + (eb[t] + 4 * U) * b[t]
            h = a[t] * h + b[t]
            M[t], E[t] = h, e
        sM[k], sE[k] = h, e
    out = {"y": E + U * M, "slots": sE}
    if grad_y is None:
        return out
    slope = np.where(m > 0, a * a / np.where(m > 0, m, 1), 0.0)
    with np.errstate(invalid="ignore"):
        oi, orr = 1 - i, 1 - r
        # 1 - i in fp32: the absolute error of i and a rounding, relative to 1 - i
        eoi = np.where(oi > 0, (ei * i + 2 * U) / np.where(oi > 0, oi, 1), 0.0)
        eor = np.where(orr > 0, (er * r + 2 * U) / np.where(orr > 0, orr, 1), 0.0)
    for name in ("grad_x", "grad_gate_x", "grad_gate_a"):
        out[name] = np.zeros((T, C))
    lam_e, g0 = np.zeros(C), np.zeros((len(lens), C))
    lam_m = np.zeros(C)
    for k, (s, n) in enumerate(zip(starts, lens)):
        g = np.abs(grad_state[k]) if grad_state is not None else np.zeros(C)
        e = np.zeros(C)
        for t in range(s + n - 1, s - 1, -1):
            G, eG = g + np.abs(grad_y[t]), e + 4 * U * (g + np.abs(grad_y[t]))
            ix = np.abs(i[t] * x[t])
            out["grad_x"][t] = m[t] * i[t] * (eG + G * (em[t] + ei[t] + 4 * U))
            out["grad_gate_x"][t] = m[t] * ix * np.abs(oi[t]) * (eG + G * (em[t] + ei[t] + eoi[t] + 6 * U))
            D = a[t] * M0[t] + slope[t] * ix
            eD = (a[t] * E0[t] + a[t] * M0[t] * (ea[t] + 4 * U) +
                  slope[t] * ix * (2 * ea[t] + em[t] + ei[t] + 8 * U))
            eL = eG * D + G * eD
            out["grad_gate_a"][t] = np.abs(la[t] * orr[t]) * (eL + G * D * (el[t] + eor[t] + 4 * U))
            lam_e += r[t] * (eL + G * D * (er[t] + 4 * U))
            lam_m += r[t] * G * D
            e = a[t] * eG + a[t] * G * (ea[t] + 4 * U)
            g = a[t] * G
        g0[k] = e if resume[k] else 0.0
    # the sum over tokens: runs of 8 in a thread, 8 runs, then the chunks 8 ways; at most T / 512 + 24 roundings a term
    scale = c0 * ol.sigmoid(lam)
    out["grad_lam"] = scale * (lam_e + lam_m * (T / 512 + 24 + 12) * U)
    out["grad_slots"] = g0
    return out


def close(got, ref, bound, dtype=torch.float32):
    """got (tensor) within bound plus the rounding to dtype of ref; the worst excess in the message."""
    got = np64(got)
    tol = bound + half_step(dtype) * (np.abs(ref) + bound) + tiny_step(dtype) + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / tol)), np.argwhere(bad)[:4].tolist())
