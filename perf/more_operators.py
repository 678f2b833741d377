"""Cases of the operators a selective-scan language model is trained and served with: the
selective scan with a decay for each channel and state (forward, and forward with backward),
the short causal convolution in front of it (the same two), and the softmax cross entropy of a
projection onto a large vocabulary (the loss, and the loss with its gradients).

A case is a dict of plain values.  ``prepare`` draws its inputs on the GPU,
``run`` makes one pass (``own``: through the library's entry points; else in
elementary torch operations in 32 bits), ``exact`` gives the same outputs from the
definitions in 64 bits and ``work`` the bytes and operations a pass cannot do without.

The formulas (tokens t of one sequence, channels c, states n, group g of c, row elements k):

scan   v = dt + dt_bias, step = v if v > 20 else log1p(exp(v));  a = exp(step A[c,n])
       h_t = a h_{t-1} + step x_t B[t,g,n];  p_t = sum_n h_t C[t,g,n] + D[c] x_t;  y_t = p_t z sigmoid(z)
conv   s = the slot's K - 1 inputs, then the tokens;  v_t = bias + sum_u w[c,u] s_{t+u};  out_t = v sigmoid(v)
loss   l = hidden weight^T;  lse = log sum_v exp(l);  loss = lse - l[target], and 0 where the target is ignored
"""
import math

import numpy as np
import torch

own = False

IGNORE = -100
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


def listed():
    return [
        # One decode step of a small batch: latency, and the states' traffic.
        {"name": "scan_decode_16x1", "op": "scan", "channels": 4096, "states": 16, "groups": 1,
         "lens": ",".join(["1"] * 16), "dtype": "bf16", "gate": True},
        # A serving batch with prompts of every length beside single tokens (the ragged batch of the scan's benchmark).
        {"name": "scan_ragged_12", "op": "scan", "channels": 4096, "states": 16, "groups": 1,
         "lens": "1,1,1,1,3,25,26,150,513,1024,2048,4096", "dtype": "bf16", "gate": True},
        # A training step of one long sequence.
        {"name": "scan_train_1x4096", "op": "scan_train", "channels": 4096, "states": 16, "groups": 1, "lens": "4096",
         "dtype": "bf16", "gate": True},
        # A training step of a small model, odd lengths, channels and states, full precision, no gate.
        {"name": "scan_train_4x777", "op": "scan_train", "channels": 1001, "states": 13, "groups": 1,
         "lens": "777,777,777,777", "dtype": "fp32", "gate": False},
        # The convolution of a decode step.
        {"name": "conv_decode_64x1", "op": "conv", "channels": 4096, "kernel": 4, "lens": ",".join(["1"] * 64),
         "dtype": "bf16", "bias": True},
        # The convolution of a prefill batch, ragged, out of a projection.
        {"name": "conv_ragged_12", "op": "conv", "channels": 8192, "kernel": 4,
         "lens": "1,1,1,1,3,25,26,150,513,1024,2048,4096", "dtype": "bf16", "bias": True},
        # A training step of it.
        {"name": "conv_train_2x4096", "op": "conv_train", "channels": 8192, "kernel": 4, "lens": "4096,4096",
         "dtype": "bf16", "bias": True},
        # The same of a small model, odd sizes, full precision, no bias.
        {"name": "conv_train_4x777", "op": "conv_train", "channels": 1001, "kernel": 3, "lens": "777,777,777,777",
         "dtype": "fp32", "bias": False},
        # The loss of a few tokens (scoring one answer): reads the vocabulary's rows.
        {"name": "loss_16", "op": "loss", "rows": 16, "vocab": 32000, "width": 4096, "dtype": "bf16", "ignored": 0.0},
        # The loss of an evaluation batch, vocabulary of odd size.
        {"name": "loss_8192", "op": "loss", "rows": 8192, "vocab": 50257, "width": 1024, "dtype": "bf16", "ignored": 0.1},
        # A training step's loss, the largest.
        {"name": "loss_train_4096", "op": "loss_train", "rows": 4096, "vocab": 64000, "width": 2048, "dtype": "bf16",
         "ignored": 0.0},
        # A short training step of odd sizes in which the prompt's tokens are ignored.
        {"name": "loss_train_777", "op": "loss_train", "rows": 777, "vocab": 32003, "width": 1001, "dtype": "fp16",
         "ignored": 0.4},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total):
    """Sequence lengths of about `total` tokens: equal ones, ragged ones or single tokens."""
    kind = rng.randrange(3)
    if kind == 0:
        n = _log_int(rng, 1, 16)
        return [max(1, total // n)] * n
    if kind == 1:
        lens, left = [], total
        while left > 0 and len(lens) < 64:
            lens.append(min(left, _log_int(rng, 1, max(1, total))))
            left -= lens[-1]
        return lens
    return [1] * max(1, min(512, total // 8))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_train", "conv", "conv_train", "loss", "loss_train", "loss_train"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("loss", "loss_train"):
        rows, vocab = _log_int(rng, 1, 8192), _log_int(rng, 100, 131072)
        width = _log_int(rng, 64, 4096)
        if rng.random() < 0.7:
            vocab, width = max(64, vocab // 64 * 64), max(64, width // 64 * 64)
        while rows * vocab * max(width, 2048) > 4096 * 64000 * 2048:
            rows //= 2
        return {"op": op, "rows": rows, "vocab": vocab, "width": width, "dtype": rng.choice(["bf16", "bf16", "fp16"]),
                "ignored": rng.choice([0.0, 0.0, 0.1, 0.5, 0.9])}
    channels = _log_int(rng, 48, 8192)
    if rng.random() < 0.7:
        channels = max(64, channels // 64 * 64)
    if op in ("conv", "conv_train"):
        lens = _lens(rng, _log_int(rng, 1, min(32768, (64 << 20) // channels)))
        return {"op": op, "channels": channels, "kernel": rng.choice([2, 3, 4, 4, 4, 5, 8]), "lens": ",".join(map(str, lens)),
                "dtype": dtype, "bias": rng.random() < 0.7}
    states = rng.choice([16, 16, 16, 8, 32, 64, 128, rng.randrange(1, 65)])
    lens = _lens(rng, _log_int(rng, 1, min(16384, (256 << 20) // (channels * states))))
    groups = rng.choice([g for g in (1, 1, 1, 2, 4) if channels % g == 0])
    return {"op": op, "channels": channels, "states": states, "groups": groups, "lens": ",".join(map(str, lens)),
            "dtype": dtype, "gate": rng.random() < 0.6}


def _case_lens(case):
    return [int(v) for v in case["lens"].split(",")]


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op in ("loss", "loss_train"):
        T, V, D = case["rows"], case["vocab"], case["width"]
        T = round(T * (1 - case["ignored"]))          # what is ignored needs no work
        b, f = (T + V) * D * e + 16 * T, 2 * T * V * D
        if op == "loss_train":                        # hidden, weight and lse again, both gradients; the logits again, since they are not kept
            b, f = 2 * b + (T + V) * D * e, 4 * f
        return {"bytes": b, "flops": f}
    lens, C = _case_lens(case), case["channels"]
    T, n = sum(lens), len(lens)
    if op in ("conv", "conv_train"):
        K = case["kernel"]
        b, f = 2 * T * C * e + 8 * n * C * (K - 1) + 4 * C * K, T * C * (2 * K + 4)
        if op == "conv_train":
            b, f = b + 3 * T * C * e + 12 * n * C * (K - 1) + 8 * C * K, f + T * C * (6 * K + 10)
        return {"bytes": b, "flops": f}
    N, G, tensors = case["states"], case["groups"], 4 if case["gate"] else 3
    b = T * (tensors * C + 2 * G * N) * e + 8 * n * C * N + 4 * C * N
    f = 7 * T * C * N + 15 * T * C
    if op == "scan_train":
        b += T * ((2 * tensors - 1) * C + 4 * G * N) * e + 8 * n * C * N + 8 * C * N
        f += 25 * T * C * N + 40 * T * C
    return {"bytes": b, "flops": f}


# ---- inputs ----


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, op = TYPES[case["dtype"]], case["op"]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    if op in ("loss", "loss_train"):
        T, V, D = case["rows"], case["vocab"], case["width"]
        target = torch.randint(0, V, (T,), generator=g, device="cuda")
        order = torch.argsort(uniform(T))
        target[order[round(T * (1 - case["ignored"])):]] = IGNORE
        s = dict(op=op, hidden=normal(T, D), weight=normal(V, D, scale=1.5 / math.sqrt(D)), target=target)
        if op == "loss_train":                        # of the mean over the tokens that count, scaled as 16-bit training does
            scale = 1024.0 if case["dtype"] == "fp16" else 1.0
            s["grad_loss"] = torch.full((T,), scale / max(1, round(T * (1 - case["ignored"]))), device="cuda")
        return s
    lens, C = _case_lens(case), case["channels"]
    n, T = len(lens), sum(lens)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(op=op, longest=max(lens), starts=torch.tensor(np.cumsum([0] + lens[:-1]), **i32), lens=torch.tensor(lens, **i32),
             resume=torch.tensor([k % 2 for k in range(n)], **i32))
    wide = normal(T, 2 * C)                           # one projection gives the mixer's input and its gate
    if op in ("conv", "conv_train"):
        K = case["kernel"]
        s.update(x=wide[:, :C], weight=normal(C, K, dtype=torch.float32, scale=1.0 / math.sqrt(K)),
                 bias=normal(C, dtype=torch.float32, scale=0.1) if case["bias"] else None,
                 slots=normal(n, C, K - 1).float())
        if op == "conv_train":
            s["grad_out"] = normal(T, C)
            s["grad_slots"] = normal(n, C, K - 1, dtype=torch.float32)
        return s
    N, G = case["states"], case["groups"]
    bc = normal(T, 32 + 2 * G * N)                    # one projection gives the step's low-rank part, B and C
    start = torch.exp(uniform(C) * math.log(100.0)) * 1e-3            # steps of 1e-3 to 1e-1 at dt = 0
    s.update(x=normal(T, C), z=wide[:, C:] if case["gate"] else None, dt=normal(T, C, scale=0.5),
             B=bc[:, 32:32 + G * N], C=bc[:, 32 + G * N:], groups=G, dt_bias=torch.log(torch.expm1(start)),
             A=-torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * normal(C, N, dtype=torch.float32)),
             D=1.0 + 0.1 * normal(C, dtype=torch.float32), slots=normal(n, C, N, dtype=torch.float32, scale=0.5))
    if op == "scan_train":
        s["grad_y"] = normal(T, C)
        s["grad_slots"] = normal(n, C, N, dtype=torch.float32, scale=0.1)
    return s


# ---- one pass ----


def run(s):
    return RUN[s["op"]](s)


def _linear_scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t over the rows (a is 0 where a sequence begins), by doubling the reach of each row."""
    step = 1
    while step < longest:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _sequences(s):
    first = s["starts"].long()
    return first, first + s["lens"].long() - 1


def _per_channel(v, s):
    """[T, G N] as [T, C, N] (each group's row for each of its channels)."""
    C, N = s["A"].shape
    return v.float().view(-1, s["groups"], 1, N).expand(-1, -1, C // s["groups"], -1).reshape(-1, C, N)


def _silu(v):
    """v sigmoid(v) and its derivative."""
    sg = 1.0 / (1.0 + torch.exp(-v))
    return v * sg, sg * (1.0 + v * (1.0 - sg))


def _scan_forward(s):
    x, v = s["x"].float(), s["dt"].float() + s["dt_bias"]
    step = torch.where(v > 20, v, torch.log1p(torch.exp(v)))
    a = torch.exp(step[:, :, None] * s["A"])
    first, last = _sequences(s)
    h0 = s["slots"] * (s["resume"] != 0)[:, None, None]
    b = (step * x)[:, :, None] * _per_channel(s["B"], s)
    b[first] += a[first] * h0
    c = a.clone()
    c[first] = 0
    h = _linear_scan(c, b, s["longest"])
    s["slots"].copy_(h[last])
    p = (h * _per_channel(s["C"], s)).sum(2) + s["D"] * x
    gate, slope = (1.0, 0.0) if s["z"] is None else _silu(s["z"].float())
    return x, v, step, a, h0, h, p, gate, slope


def _own_scan(s, chunk_states=None):
    from state_space_model_ssm_gb300 import ssm_selective_scan
    return ssm_selective_scan(s["slots"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["starts"], s["lens"], s["resume"],
                              z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True, n_groups=s["groups"], chunk_states=chunk_states)


def _scan(s):
    if own:
        return {"y": _own_scan(s), "slots": s["slots"]}
    *_, p, gate, _ = _scan_forward(s)
    return {"y": (p * gate).to(s["x"].dtype), "slots": s["slots"]}


NAMES = ("grad_x", "grad_dt", "grad_A", "grad_B", "grad_C", "grad_D", "grad_z", "grad_dt_bias", "grad_slots")


def _scan_train(s):
    if own:
        from state_space_model_ssm_gb300 import selective_scan_chunk_states, ssm_selective_scan_backward
        n, C, N = s["slots"].shape
        chunks = selective_scan_chunk_states(n, s["x"].shape[0], C, N, device=s["x"].device)
        y = _own_scan(s, chunks)
        grads = ssm_selective_scan_backward(
            s["grad_y"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], chunks, s["starts"], s["lens"], s["resume"], z=s["z"],
            dt_bias=s["dt_bias"], dt_softplus=True, n_groups=s["groups"], grad_state=s["grad_slots"])
        return {"y": y, "slots": s["slots"], **{k: v for k, v in zip(NAMES, grads) if v is not None}}
    first, last = _sequences(s)
    x, v, step, a, h0, h, p, gate, slope = _scan_forward(s)
    B, C = _per_channel(s["B"], s), _per_channel(s["C"], s)
    dt, gy = s["x"].dtype, s["grad_y"].float()
    gp = gy * gate
    e = gp[:, :, None] * C
    e[last] += s["grad_slots"]
    c = torch.cat([a[1:], a[:1]])
    c[last] = 0
    e = _linear_scan(c.flip(0), e.flip(0), s["longest"]).flip(0)
    before = torch.cat([h[:1], h[:-1]])
    before[first] = h0
    before *= a                                       # what the step before left of the state
    eb, ea = (e * B).sum(2), e * before
    gdt = ((ea * s["A"]).sum(2) + x * eb) * torch.where(v > 20, 1.0, 1.0 / (1.0 + torch.exp(-v)))
    T, G, N = x.shape[0], s["groups"], s["A"].shape[1]
    out = {"y": (p * gate).to(dt), "slots": s["slots"], "grad_x": (s["D"] * gp + step * eb).to(dt), "grad_dt": gdt.to(dt),
           "grad_A": (ea * step[:, :, None]).sum(0),
           "grad_B": (e * (step * x)[:, :, None]).view(T, G, -1, N).sum(2).reshape(T, G * N).to(dt),
           "grad_C": (h * gp[:, :, None]).view(T, G, -1, N).sum(2).reshape(T, G * N).to(dt),
           "grad_D": (gp * x).sum(0), "grad_dt_bias": gdt.sum(0),
           "grad_slots": a[first] * e[first] * (s["resume"] != 0)[:, None, None]}
    if s["z"] is not None:
        out["grad_z"] = (gy * p * slope).to(dt)
    return out


def _stream(s):
    """The stream of inputs of every sequence back to back, [T + n (K - 1), C], and the row of each token in it."""
    K1, T = s["weight"].shape[1] - 1, s["x"].shape[0]
    n = s["slots"].shape[0]
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), s["lens"].long(), output_size=T)
    rows = torch.arange(T, device="cuda") + (seq + 1) * K1
    head = (s["starts"].long() + torch.arange(n, device="cuda") * K1)[:, None] + torch.arange(K1, device="cuda")
    stream = torch.empty(T + n * K1, s["x"].shape[1], device="cuda")
    stream[rows] = s["x"].float()
    stream[head] = (s["slots"] * (s["resume"] != 0)[:, None, None]).transpose(1, 2)
    return stream, rows, head, head + s["lens"].long()[:, None]


def _conv_forward(s):
    stream, rows, head, tail = _stream(s)
    w = s["weight"]
    K = w.shape[1]
    v = stream[rows] * w[:, K - 1] + sum(stream[rows - u] * w[:, K - 1 - u] for u in range(1, K))
    if s["bias"] is not None:
        v = v + s["bias"]
    return stream, rows, head, tail, v


def _conv(s):
    if own:
        from state_space_model_ssm_gb300 import ssm_causal_conv
        out = ssm_causal_conv(s["x"], s["weight"], s["slots"], s["starts"], s["lens"], s["resume"], bias=s["bias"])
        return {"out": out, "slots": s["slots"]}
    stream, _, _, tail, v = _conv_forward(s)
    s["slots"].copy_(stream[tail].transpose(1, 2))
    return {"out": _silu(v)[0].to(s["x"].dtype), "slots": s["slots"]}


def _conv_train(s):
    if own:
        from state_space_model_ssm_gb300 import ssm_causal_conv, ssm_causal_conv_backward
        slots = s["slots"].clone()                    # the backward pass reads what the slots held before
        out = ssm_causal_conv(s["x"], s["weight"], slots, s["starts"], s["lens"], s["resume"], bias=s["bias"])
        gx, gw, gb, gs = ssm_causal_conv_backward(s["grad_out"], s["x"], s["weight"], s["starts"], s["lens"], s["resume"],
                                                  bias=s["bias"], initial_state=s["slots"], grad_state=s["grad_slots"])
        return {"out": out, "slots": slots, "grad_x": gx, "grad_weight": gw, "grad_slots": gs,
                **({} if s["bias"] is None else {"grad_bias": gb})}
    stream, rows, head, tail, v = _conv_forward(s)
    slots = stream[tail].transpose(1, 2).contiguous()
    w, K, dt = s["weight"], s["weight"].shape[1], s["x"].dtype
    y, slope = _silu(v)
    gv = s["grad_out"].float() * slope
    gs = torch.zeros_like(stream)
    gs.index_put_((tail,), s["grad_slots"].transpose(1, 2), accumulate=True)
    gw = torch.empty_like(w)
    for u in range(K):
        gs.index_put_((rows - u,), gv * w[:, K - 1 - u], accumulate=True)
        gw[:, K - 1 - u] = (gv * stream[rows - u]).sum(0)
    out = {"out": y.to(dt), "slots": slots, "grad_x": gs[rows].to(dt), "grad_weight": gw,
           "grad_slots": gs[head].transpose(1, 2) * (s["resume"] != 0)[:, None, None]}
    if s["bias"] is not None:
        out["grad_bias"] = gv.sum(0)
    return out


def _loss_forward(s):
    h, w = s["hidden"].float(), s["weight"].float()
    counts = s["target"] != IGNORE
    target = torch.where(counts, s["target"], 0)[:, None]
    logits = h @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))
    loss = torch.where(counts, (lse - logits.gather(1, target))[:, 0], 0.0)
    return h, w, counts, target, logits, lse, loss


def _loss(s):
    if own:
        from state_space_model_ssm_gb300 import ssm_linear_cross_entropy
        loss, lse = ssm_linear_cross_entropy(s["hidden"], s["weight"], s["target"], ignore_index=IGNORE)
        return {"loss": loss, "lse": lse}
    _, _, counts, _, _, lse, loss = _loss_forward(s)
    return {"loss": loss, "lse": torch.where(counts, lse[:, 0], 0.0)}


def _loss_train(s):
    if own:
        from state_space_model_ssm_gb300 import ssm_linear_cross_entropy, ssm_linear_cross_entropy_backward
        loss, lse = ssm_linear_cross_entropy(s["hidden"], s["weight"], s["target"], ignore_index=IGNORE)
        gh, gw = ssm_linear_cross_entropy_backward(s["grad_loss"], s["hidden"], s["weight"], s["target"], lse,
                                                   ignore_index=IGNORE)
        return {"loss": loss, "lse": lse, "grad_hidden": gh, "grad_weight": gw}
    h, w, counts, target, logits, lse, loss = _loss_forward(s)
    p = torch.exp(logits - lse)
    p.scatter_add_(1, target, torch.full_like(target, -1, dtype=p.dtype))
    p *= torch.where(counts, s["grad_loss"], 0.0)[:, None]
    dt = s["hidden"].dtype
    return {"loss": loss, "lse": torch.where(counts, lse[:, 0], 0.0), "grad_hidden": (p @ w).to(dt),
            "grad_weight": (p.t() @ h).to(dt)}


RUN = {"scan": _scan, "scan_train": _scan_train, "conv": _conv, "conv_train": _conv_train, "loss": _loss,
       "loss_train": _loss_train}


# ---- the definitions in 64 bits ----


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("loss", "loss_train"):
        return _exact_loss(case, s)
    return (_exact_scan if s["op"] in ("scan", "scan_train") else _exact_conv)(case, s)


def _exact_loss(case, s):
    """Row by row of the tokens that count, a few hundred at a time."""
    T, V, D = case["rows"], case["vocab"], case["width"]
    if T * V * D * (3 if s["op"] == "loss_train" else 1) > 3e12:      # 64-bit products are slow here
        return None
    d = torch.float64
    w = s["weight"].to(d)
    out = {"loss": torch.zeros(T, dtype=d, device="cuda"), "lse": torch.zeros(T, dtype=d, device="cuda")}
    if s["op"] == "loss_train":
        out.update(grad_hidden=torch.zeros(T, D, dtype=d, device="cuda"), grad_weight=torch.zeros(V, D, dtype=d, device="cuda"))
    for rows in torch.nonzero(s["target"] != IGNORE)[:, 0].split(512):
        h, t = s["hidden"][rows].to(d), s["target"][rows]
        logits = torch.einsum("td,vd->tv", h, w)
        out["lse"][rows] = torch.logsumexp(logits, 1)
        logp = torch.log_softmax(logits, 1)
        at = torch.arange(len(rows), device="cuda")
        out["loss"][rows] = -logp[at, t]
        if s["op"] == "loss_train":
            g = torch.exp(logp)
            g[at, t] -= 1.0
            g = g * s["grad_loss"][rows].to(d)[:, None]
            out["grad_hidden"][rows] = torch.einsum("tv,vd->td", g, w)
            out["grad_weight"] += torch.einsum("tv,td->vd", g, h)
    return out


def _exact_conv(case, s):
    """Sequence by sequence, by the definition's sum over the taps."""
    d, K = torch.float64, case["kernel"]
    w = s["weight"].to(d)
    out = {"out": torch.empty(s["x"].shape, dtype=d, device="cuda"), "slots": torch.empty_like(s["slots"], dtype=d)}
    train = s["op"] == "conv_train"
    if train:
        out.update(grad_x=torch.empty_like(out["out"]), grad_weight=torch.zeros_like(w), grad_slots=torch.zeros_like(out["slots"]))
        if s["bias"] is not None:
            out["grad_bias"] = torch.zeros(w.shape[0], dtype=d, device="cuda")
    at = 0
    for k, n in enumerate(_case_lens(case)):
        head = s["slots"][k].to(d).t() if k % 2 else torch.zeros(K - 1, w.shape[0], dtype=d, device="cuda")
        stream = torch.cat([head, s["x"][at:at + n].to(d)])
        windows = stream.unfold(0, K, 1)                              # [n, C, K]
        v = torch.einsum("tcu,cu->tc", windows, w)
        if s["bias"] is not None:
            v = v + s["bias"].to(d)
        sg = torch.special.expit(v)
        out["out"][at:at + n], out["slots"][k] = v * sg, stream[n:].t()
        if train:
            gv = s["grad_out"][at:at + n].to(d) * (sg + v * sg * (1 - sg))
            gs = torch.zeros_like(stream)
            gs[n:] = s["grad_slots"][k].to(d).t()
            for u in range(K):
                gs[u:u + n] += gv * w[:, u]
            out["grad_x"][at:at + n] = gs[K - 1:]
            out["grad_slots"][k] = gs[:K - 1].t() * (k % 2)
            out["grad_weight"] += torch.einsum("tc,tcu->cu", gv, windows)
            if s["bias"] is not None:
                out["grad_bias"] += gv.sum(0)
        at += n
    return out


def _exact_scan(case, s):
    """Token by token; the sequences side by side, each as long as the longest."""
    d, lens = torch.float64, _case_lens(case)
    n, L, C, N, G = len(lens), max(lens), case["channels"], case["states"], case["groups"]
    train = s["op"] == "scan_train"
    if n * L * C * (1 + N * train) > (1 << 30) or n * C * N > (1 << 28):
        return None
    place = torch.tensor([k * L + t for k, v in enumerate(lens) for t in range(v)], device="cuda")
    live = torch.zeros(n * L, dtype=d, device="cuda").index_fill_(0, place, 1.0).view(n, L)

    def wide(v):                                                      # past a sequence's end: zeros
        return torch.zeros(n * L, v.shape[1], dtype=d, device="cuda").index_copy_(0, place, v.to(d)).view(n, L, v.shape[1])

    def packed(v):
        return v.reshape(n * L, -1)[place]

    v = wide(s["dt"].to(d) + s["dt_bias"].to(d))
    # the definition's threshold: above 20 the step is v itself
    step = torch.where(v > 20, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0)))) * live[:, :, None]
    x, B, Cm = wide(s["x"]), wide(s["B"]).view(n, L, G, 1, N), wide(s["C"]).view(n, L, G, 1, N)
    A, D = s["A"].to(d), s["D"].to(d)
    flag = (s["resume"] != 0)[:, None, None]
    h = s["slots"].to(d) * flag
    p = torch.empty(n, L, C, dtype=d, device="cuda")
    hs = torch.empty(n, L + 1, C, N, dtype=d, device="cuda") if train else None
    if train:
        hs[:, 0] = h
    for t in range(L):                                                # a step of 0 leaves the state as it is
        u = (step[:, t] * x[:, t]).view(n, G, -1, 1) * B[:, t]
        h = torch.exp(step[:, t, :, None] * A) * h + u.reshape(n, C, N)
        p[:, t] = torch.einsum("igcm,igm->igc", h.view(n, G, -1, N), Cm[:, t, :, 0]).reshape(n, C)
        if train:
            hs[:, t + 1] = h
    p += D * x
    gate, slope = torch.ones((), dtype=d, device="cuda"), None
    if s["z"] is not None:
        z = wide(s["z"])
        sg = torch.special.expit(z)
        gate, slope = z * sg, sg + z * sg * (1 - sg)
    out = {"y": packed(p * gate), "slots": h}
    if not train:
        return out
    gy = wide(s["grad_y"])
    gp = gy * gate
    e = s["grad_slots"].to(d)
    gA = torch.zeros(C, N, dtype=d, device="cuda")
    gx, gstep = torch.empty_like(p), torch.empty_like(p)
    gB, gC = (torch.zeros(n, L, G, N, dtype=d, device="cuda") for _ in range(2))
    for t in range(L - 1, -1, -1):
        e = e + (gp[:, t].view(n, G, -1, 1) * Cm[:, t]).reshape(n, C, N)
        st = step[:, t, :, None]
        decay = torch.exp(st * A)
        kept = decay * hs[:, t] * e
        eg = e.view(n, G, -1, N)
        eb = torch.einsum("igcm,igm->igc", eg, B[:, t, :, 0]).reshape(n, C)
        gx[:, t] = gp[:, t] * D + step[:, t] * eb
        gstep[:, t] = (kept * A).sum(2) + x[:, t] * eb
        gA += (kept * st).sum(0)
        gB[:, t] = torch.einsum("igcm,igc->igm", eg, (step[:, t] * x[:, t]).view(n, G, -1))
        gC[:, t] = torch.einsum("igcm,igc->igm", hs[:, t + 1].view(n, G, -1, N), gp[:, t].view(n, G, -1))
        e = e * decay
    gdt = gstep * torch.where(v > 20, 1.0, torch.special.expit(v)) * live[:, :, None]
    out.update(grad_x=packed(gx), grad_dt=packed(gdt), grad_A=gA, grad_B=packed(gB), grad_C=packed(gC),
               grad_D=(gp * x).sum((0, 1)), grad_dt_bias=gdt.sum((0, 1)), grad_slots=e * flag)
    if s["z"] is not None:
        out["grad_z"] = packed(gy * p * slope)
    return out
