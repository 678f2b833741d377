"""A small language model on a selective scan, from the library's operators (needs a GB300).

    python examples/selective_lm.py [--channels 512] [--vocab 8000] [--tokens 512] [--steps 4]

One layer: RMS norm, a projection into the mixer's input and gate, the short causal convolution, a projection of its
output onto the scan's step (low rank), B and C, the selective scan with its gate, a projection back into the stream, and the
cross entropy of the projection onto the vocabulary.  The projections are torch products on 16-bit activations.

Serving: a prompt is prefilled, then decoded token by token from the slots; the decoded rows are checked against one
pass over the whole sequence.

Training: the loss of a batch of two sequences (prompt tokens ignored) and its gradients by the backward functions; the
gradient along a direction of some parameters is checked against differences of the loss.  The check runs in fp16: with
bf16 the activations' roundings (2^-9) change the loss by up to 6 % of such a difference.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import state_space_model_ssm_gb300 as ssm  # noqa: E402

RANK, STATES, TAPS = 16, 16, 4


class SelectiveLM:
    """fp32 masters of one layer and the vocabulary; the products run on 16-bit copies."""

    def __init__(self, channels, vocab, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device=device) * scale

        inner = 2 * channels
        self.channels, self.inner, self.dtype = channels, inner, dtype
        start = torch.exp(torch.rand(inner, generator=g, device=device) * math.log(100.0)) * 1e-3
        self.p = dict(
            norm=torch.ones(channels, device=device), w_in=normal(2 * inner, channels, scale=channels ** -0.5),
            conv=normal(inner, TAPS, scale=TAPS ** -0.5), conv_bias=normal(inner, scale=0.1),
            w_x=normal(RANK + 2 * STATES, inner, scale=inner ** -0.5), w_dt=normal(inner, RANK, scale=0.1),
            dt_bias=torch.log(torch.expm1(start)), A_log=torch.log(torch.arange(1, STATES + 1, device=device).float()).repeat(inner, 1),
            D=torch.ones(inner, device=device), w_out=normal(channels, inner, scale=inner ** -0.5),
            head=normal(vocab, channels, scale=channels ** -0.5))

    def slots(self, n, device="cuda"):
        return (torch.zeros(n, self.inner, TAPS - 1, device=device), torch.zeros(n, self.inner, STATES, device=device))

    def forward(self, x, slots, meta, p=None, train=False):
        """(the stream after the layer, what the gradients need); slots (conv, scan) are updated in place."""
        p = self.p if p is None else p
        half = {k: v.to(self.dtype) for k, v in p.items() if k.startswith("w_")}
        n, _ = ssm.ssm_add_norm(x, p["norm"])
        proj = n @ half["w_in"].t()
        u = ssm.ssm_causal_conv(proj[:, :self.inner], p["conv"], slots[0], *meta, bias=p["conv_bias"])
        low = u @ half["w_x"].t()
        dt = low[:, :RANK] @ half["w_dt"].t()
        B, C = low[:, RANK:RANK + STATES], low[:, RANK + STATES:]
        A = -torch.exp(p["A_log"])
        chunks = ssm.selective_scan_chunk_states(len(slots[0]), x.shape[0], *A.shape, device=x.device) if train else None
        y = ssm.ssm_selective_scan(slots[1], u, dt, A, B, C, p["D"], *meta, z=proj[:, self.inner:], dt_bias=p["dt_bias"],
                                   dt_softplus=True, chunk_states=chunks)
        out = x + y @ half["w_out"].t()
        return out, (n, proj, u, low, dt, A, chunks, y, half)

    def loss(self, x, targets, meta, p=None):
        """Mean loss over the tokens that count."""
        p = self.p if p is None else p
        out, _ = self.forward(x, self.slots(len(meta[0])), meta, p)
        loss, _ = ssm.ssm_linear_cross_entropy(out, p["head"].to(self.dtype), targets)
        return loss.double().sum() / (targets != -100).sum()

    def gradients(self, x, targets, meta):
        """Gradients of ``loss`` by name."""
        p, E = self.p, self.inner
        out, (n, proj, u, low, dt, A, chunks, y, half) = self.forward(x, self.slots(len(meta[0])), meta, train=True)
        head = p["head"].to(self.dtype)
        _, lse = ssm.ssm_linear_cross_entropy(out, head, targets)
        mean = (1.0 / (targets != -100).sum()).expand(len(targets)).float().contiguous()
        g_out, g_head = ssm.ssm_linear_cross_entropy_backward(mean, out, head, targets, lse)
        g_proj, g_low = torch.empty_like(proj), torch.empty_like(low)       # gradients side by side, like the projections
        B, C = low[:, RANK:RANK + STATES], low[:, RANK + STATES:]
        g_u, g_dt, g_A, _, _, g_D, _, g_bias, _ = ssm.ssm_selective_scan_backward(
            g_out @ half["w_out"], u, dt, A, B, C, p["D"], chunks, *meta, z=proj[:, E:], dt_bias=p["dt_bias"], dt_softplus=True,
            grad_B=g_low[:, RANK:RANK + STATES], grad_C=g_low[:, RANK + STATES:], grad_z=g_proj[:, E:])
        g_low[:, :RANK] = g_dt @ half["w_dt"]
        g_u = g_u + g_low @ half["w_x"]
        _, g_conv, g_cb, _ = ssm.ssm_causal_conv_backward(g_u, proj[:, :E], p["conv"], *meta[:2], bias=p["conv_bias"],
                                                          grad_x=g_proj[:, :E])
        _, g_norm = ssm.ssm_add_norm_backward(g_proj @ half["w_in"], x, p["norm"])
        f = torch.Tensor.float
        return dict(norm=g_norm, w_in=f(g_proj).t() @ f(n), conv=g_conv, conv_bias=g_cb, w_x=f(g_low).t() @ f(u),
                    w_dt=f(g_dt).t() @ f(low[:, :RANK]), dt_bias=g_bias, A_log=g_A * A, D=g_D, w_out=f(g_out).t() @ f(y),
                    head=f(g_head))


def table(lens, resume, device="cuda"):
    i32 = dict(dtype=torch.int32, device=device)
    starts = [sum(lens[:k]) for k in range(len(lens))]
    return torch.tensor(starts, **i32), torch.tensor(lens, **i32), torch.tensor(resume, **i32)


def serve(model, tokens, steps):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens + steps, model.channels, generator=g, device="cuda").to(model.dtype)
    whole, _ = model.forward(x, model.slots(1), table([tokens + steps], [0]))
    slots, meta = model.slots(1), table([1], [1])
    rows = [model.forward(x[:tokens], slots, table([tokens], [0]))[0]]
    rows += [model.forward(x[t:t + 1], slots, meta)[0] for t in range(tokens, tokens + steps)]
    return float((torch.cat(rows).float() - whole.float()).norm() / whole.float().norm())


def train(model, tokens, vocab):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(tokens, model.channels, generator=g, device="cuda").to(model.dtype)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    meta = table([tokens - tokens // 3, tokens // 3], [0, 0])
    targets[:tokens // 4] = -100                              # a prompt
    grads = model.gradients(x, targets, meta)
    report = []
    for name in ("conv", "dt_bias", "A_log", "D", "norm", "w_dt"):
        d = torch.sign(grads[name])                           # a direction along which the loss does change
        slope = float((grads[name].double() * d).sum())
        step = 5e-3 / max(slope, 1e-2)                        # a change well above the roundings of the losses
        up, down = (float(model.loss(x, targets, meta, {**model.p, name: model.p[name] + s * step * d})) for s in (1, -1))
        report.append((name, slope, (up - down) / (2 * step)))
    return float(model.loss(x, targets, meta)), report


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--channels", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=8000)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    model = SelectiveLM(a.channels, a.vocab)
    print(f"serving: prefill {a.tokens} + {a.steps} decode steps, relative difference {serve(model, a.tokens, a.steps):.2e} from one pass")
    loss, report = train(SelectiveLM(a.channels, a.vocab, torch.float16), a.tokens, a.vocab)
    print(f"training: loss {loss:.4f}")
    for name, slope, diff in report:
        print(f"  gradient of {name}: {slope:.6g}, difference {diff:.6g}")


if __name__ == "__main__":
    main()
