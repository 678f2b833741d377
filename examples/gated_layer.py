"""A layer around the gated linear recurrence, from the library's operators (needs a GB300).

    python examples/gated_layer.py [--channels 2048] [--tokens 2048] [--steps 4]

Serving: the residual stream is added and normalised into 8 bits (``ssm_add_norm``), one 8-bit
product gives the recurrence's input and both gates (``ssm_int8_matmul``), the recurrence runs on
their slices with its state in per-sequence slots (``ssm_gated_scan``), and its output goes through
the row quantiser and a second product back into the stream.  A prompt is prefilled, then decoded
token by token; the decoded rows are checked against one pass over the whole sequence.

Training: forward with saved chunk states, and the gradients of the recurrence and of the norm
(``ssm_gated_scan_backward``, ``ssm_add_norm_backward``), with the projections in torch; the
gradient of the loss along a random direction is checked against a difference.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import state_space_model_ssm_gb300 as ssm  # noqa: E402


class GatedLayer:
    """Weights of one layer: fp32 masters, and their 8-bit rows for serving."""

    def __init__(self, channels, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.channels = channels
        self.w_in = torch.randn(3 * channels, channels, generator=g, device=device) / math.sqrt(channels)
        self.w_out = torch.randn(channels, channels, generator=g, device=device) / math.sqrt(channels)
        self.norm = torch.ones(channels, device=device)
        a0 = torch.rand(channels, generator=g, device=device) * 0.099 + 0.9
        self.lam = torch.log(torch.expm1(-torch.log(a0)))
        self.q_in, self.s_in = ssm.ssm_quantize_rows(self.w_in)
        self.q_out, self.s_out = ssm.ssm_quantize_rows(self.w_out)

    def serve(self, x, residual, slots, starts, lens, resume):
        """One serving step: (the layer's output, the residual stream), slots updated in place."""
        C = self.channels
        codes, scales, h = ssm.ssm_add_norm(x, self.norm, residual, quant="int8")
        proj = ssm.ssm_int8_matmul(codes, scales, self.q_in, self.s_in, out_dtype=x.dtype)
        y = ssm.ssm_gated_scan(slots, proj[:, :C], proj[:, C:2 * C], proj[:, 2 * C:], self.lam, starts, lens, resume)
        codes, scales = ssm.ssm_quantize_rows(y)
        return ssm.ssm_int8_matmul(codes, scales, self.q_out, self.s_out, out_dtype=x.dtype), h

    def loss(self, x, residual, target, slots, meta, save=False):
        """0.5 |layer(x) - target|^2 in fp32, and with `save` what the gradients need."""
        C = self.channels
        n, h = ssm.ssm_add_norm(x, self.norm, residual)
        proj = n @ self.w_in.t()
        chunks = ssm.gated_scan_chunk_states(len(slots), *x.shape, device=x.device)
        y = ssm.ssm_gated_scan(slots, proj[:, :C], proj[:, C:2 * C], proj[:, 2 * C:], self.lam, *meta, chunk_states=chunks)
        diff = y @ self.w_out.t() + h - target
        return (0.5 * diff.double().square().sum(), (n, h, proj, chunks, y, diff)) if save else 0.5 * diff.double().square().sum()

    def gradients(self, saved, meta):
        """Gradients of the loss: input (x and residual alike), norm, lam, both projections."""
        C = self.channels
        n, h, proj, chunks, y, diff = saved
        g_proj = torch.empty_like(proj)                       # the three gradients side by side, like proj
        parts = [g_proj[:, k * C:(k + 1) * C] for k in range(3)]
        *_, g_lam, _ = ssm.ssm_gated_scan_backward(
            diff @ self.w_out, proj[:, :C], proj[:, C:2 * C], proj[:, 2 * C:], self.lam, chunks, *meta,
            grad_x=parts[0], grad_gate_a=parts[1], grad_gate_x=parts[2])
        g_in, g_norm = ssm.ssm_add_norm_backward(g_proj @ self.w_in, h, self.norm, grad_h=diff)
        return {"input": g_in, "norm": g_norm, "lam": g_lam, "w_in": g_proj.t() @ n, "w_out": diff.t() @ y}


def table(lens, resume, device="cuda"):
    i32 = dict(dtype=torch.int32, device=device)
    starts = [sum(lens[:k]) for k in range(len(lens))]
    return torch.tensor(starts, **i32), torch.tensor(lens, **i32), torch.tensor(resume, **i32)


def serve(layer, tokens, steps):
    C = layer.channels
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(tokens + steps, C, generator=g, device="cuda").bfloat16() for _ in range(2))
    slots = torch.zeros(1, C, device="cuda")
    whole, _ = layer.serve(x, r, slots, *table([tokens + steps], [0]))
    out, _ = layer.serve(x[:tokens], r[:tokens], slots, *table([tokens], [0]))
    meta = table([1], [1])
    rows = [out] + [layer.serve(x[t:t + 1], r[t:t + 1], slots, *meta)[0] for t in range(tokens, tokens + steps)]
    err = (torch.cat(rows).float() - whole.float()).norm() / whole.float().norm()
    return float(err)


def train(layer, tokens):
    C = layer.channels
    g = torch.Generator(device="cuda").manual_seed(2)
    x, r, target, d = (torch.randn(tokens, C, generator=g, device="cuda") for _ in range(4))
    lens = [tokens - tokens // 3, tokens // 3]
    meta = table(lens, [0, 0])
    slots = torch.zeros(2, C, device="cuda")
    _, saved = layer.loss(x, r, target, slots, meta, save=True)
    slope = float((layer.gradients(saved, meta)["input"].double() * d.double()).sum())
    step = 1e-2
    up, down = (layer.loss(x + s * step * d, r, target, slots, meta) for s in (1, -1))
    return slope, float(up - down) / (2 * step)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--channels", type=int, default=2048)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    layer = GatedLayer(a.channels)
    print(f"serving: prefill {a.tokens} + {a.steps} decode steps, relative difference from one pass "
          f"{serve(layer, a.tokens, a.steps):.2e}")
    slope, difference = train(layer, a.tokens)
    print(f"training: directional derivative {slope:.6g}, central difference {difference:.6g}")


if __name__ == "__main__":
    main()
