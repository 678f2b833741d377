"""Cases of the operators around the scan: the gated linear recurrence (forward, and
forward with backward), the RMS norm with the residual's addition (8-bit output, and
forward with backward), the row quantiser and the 8-bit integer matrix product.

A case is a dict of plain values.  ``prepare`` draws its inputs on the GPU,
``run`` makes one pass (``own``: through the library's entry points; else in
elementary torch operations in 32 bits), ``exact`` gives the same outputs from the
definitions in 64 bits and ``work`` the bytes and operations a pass cannot do without.

The formulas (sums over tokens t of one sequence, channels c, row elements k):

gated scan   r = sigmoid(gate_a), i = sigmoid(gate_x), log a = -decay_scale softplus(lam) r,
             a = exp(log a), m = sqrt(1 - a^2);   h_t = a_t h_{t-1} + m_t i_t x_t;   y_t = h_t
add + norm   h = x + residual rounded to the residual's type; inv = 1/sqrt(mean(h^2) + eps);
             y = h inv weight, or in 8 bits: v = h weight (fp32), f = min(127 / max|v|, FLT_MAX)
             (fp32), code = rint(v f), scale = inv / f
quantiser    the same codes with v = x and inv = 1
int8 product out[t,n] = (sum_k xq[t,k] wq[n,k]) xs[t] ws[n] + bias[n]
"""
import math

import numpy as np
import torch

own = False

DECAY_SCALE = 8.0
EPS = 1e-6
FLT_MAX = 3.4028234663852886e38
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


def listed():
    return [
        # One decode step of a small batch: latency.
        {"name": "scan_decode_16x1", "op": "scan", "channels": 4096, "lens": ",".join(["1"] * 16), "dtype": "bf16",
         "fused": True},
        # A serving batch with prompts of every length beside single tokens (the ragged batch of the scan's benchmark).
        {"name": "scan_ragged_12", "op": "scan", "channels": 4096,
         "lens": "1,1,1,1,3,25,26,150,513,1024,2048,4096", "dtype": "bf16", "fused": True},
        # Long documents, the largest: four sequences of 16384 tokens, fp32.
        {"name": "scan_long_4x16384", "op": "scan", "channels": 2048, "lens": "16384,16384,16384,16384", "dtype": "fp32",
         "fused": False},
        # A training step of one long sequence.
        {"name": "scan_train_1x4096", "op": "scan_train", "channels": 4096, "lens": "4096", "dtype": "bf16", "fused": True},
        # A training step of a small model, odd lengths and channels, full precision.
        {"name": "scan_train_4x777", "op": "scan_train", "channels": 1001, "lens": "777,777,777,777", "dtype": "fp32",
         "fused": False},
        # In front of a projection, one decode step.
        {"name": "norm_int8_16", "op": "norm_int8", "rows": 16, "width": 4096, "dtype": "bf16", "residual": "bf16"},
        # In front of a projection, a prefill batch with the residual stream in fp32.
        {"name": "norm_int8_7889", "op": "norm_int8", "rows": 7889, "width": 4096, "dtype": "bf16", "residual": "fp32"},
        # Training step of the norm.
        {"name": "norm_train_4096", "op": "norm_train", "rows": 4096, "width": 4096, "dtype": "bf16", "residual": "bf16"},
        # What enters the projection out of the mixer, odd width.
        {"name": "quantize_4108x6145", "op": "quantize", "rows": 4108, "width": 6145, "dtype": "fp16"},
        # The projection into the mixer (x and both gates), one decode step: reads the weights.
        {"name": "matmul_16", "op": "matmul", "rows": 16, "out": 12288, "inner": 4096, "dtype": "bf16", "bias": False},
        # A short prompt through a layer of odd sizes.
        {"name": "matmul_777_odd", "op": "matmul", "rows": 777, "out": 2501, "inner": 1000, "dtype": "fp32", "bias": True},
        # The projection into the mixer, a prefill batch: the largest product.
        {"name": "matmul_8192", "op": "matmul", "rows": 8192, "out": 12288, "inner": 4096, "dtype": "bf16", "bias": False},
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
    op = rng.choice(["scan", "scan", "scan_train", "norm_int8", "norm_train", "quantize", "matmul", "matmul"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("scan", "scan_train"):
        channels = _log_int(rng, 48, 8192)
        if rng.random() < 0.7:
            channels = max(64, channels // 64 * 64)
        most = min(16384, (64 << 20) // channels)
        lens = _lens(rng, _log_int(rng, 1, most))
        return {"op": op, "channels": channels, "lens": ",".join(map(str, lens)), "dtype": dtype, "fused": rng.random() < 0.5}
    if op in ("norm_int8", "norm_train", "quantize"):
        width = _log_int(rng, 48, 16384)
        if rng.random() < 0.7:
            width = max(64, width // 64 * 64)
        rows = _log_int(rng, 1, min(16384, (64 << 20) // width))
        c = {"op": op, "rows": rows, "width": width, "dtype": dtype}
        if op != "quantize":
            c["residual"] = rng.choice([dtype, dtype, "fp32"])
        return c
    rows, out, inner = _log_int(rng, 1, 8192), _log_int(rng, 64, 12288), _log_int(rng, 64, 8192)
    if rng.random() < 0.7:
        out, inner = max(64, out // 64 * 64), max(64, inner // 64 * 64)
    while rows * out * inner > 8192 * 12288 * 4096:
        rows //= 2
    return {"op": op, "rows": rows, "out": out, "inner": inner, "dtype": dtype, "bias": rng.random() < 0.5}


def _case_lens(case):
    return [int(v) for v in case["lens"].split(",")]


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op in ("scan", "scan_train"):
        lens, C = _case_lens(case), case["channels"]
        T, n = sum(lens), len(lens)
        b, f = 4 * T * C * e + 8 * n * C, 25 * T * C
        if op == "scan_train":
            b, f = b + 7 * T * C * e + 8 * n * C, f + 55 * T * C
        return {"bytes": b, "flops": f}
    if op == "matmul":
        T, N, K = case["rows"], case["out"], case["inner"]
        return {"bytes": T * K + N * K + T * N * e + 4 * (T + N), "flops": 2 * T * N * K}
    T, D = case["rows"], case["width"]
    if op == "quantize":
        return {"bytes": T * D * (e + 1) + 4 * T, "flops": 4 * T * D}
    er = SIZE[case["residual"]]
    if op == "norm_int8":
        return {"bytes": T * D * (e + 2 * er + 1) + 4 * T + 4 * D, "flops": 8 * T * D}
    return {"bytes": T * D * (2 * e + 2 * er) + T * D * (e + 3 * er) + 8 * D, "flops": 20 * T * D}


# ---- inputs ----


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, op = TYPES[case["dtype"]], case["op"]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    if op in ("scan", "scan_train"):
        lens, C = _case_lens(case), case["channels"]
        n, T = len(lens), sum(lens)
        starts = np.cumsum([0] + lens[:-1])
        i32 = dict(dtype=torch.int32, device="cuda")
        if case["fused"]:                       # one projection gives the input and both gates
            proj = normal(T, 3 * C)
            x, ga, gx = proj[:, :C], proj[:, C:2 * C], proj[:, 2 * C:]
        else:
            x, ga, gx = normal(T, C), normal(T, C), normal(T, C)
        a0 = torch.rand(C, generator=g, device="cuda") * 0.099 + 0.9      # decay at an open gate: a0 ** DECAY_SCALE
        lam = torch.log(torch.expm1(-torch.log(a0)))
        s = dict(op=op, x=x, gate_a=ga, gate_x=gx, lam=lam, longest=max(lens),
                 slots=normal(n, C, dtype=torch.float32, scale=0.5),
                 starts=torch.tensor(starts, **i32), lens=torch.tensor(lens, **i32),
                 resume=torch.tensor([k % 2 for k in range(n)], **i32))
        if op == "scan_train":
            s["grad_y"] = normal(T, C)
            s["grad_slots"] = normal(n, C, dtype=torch.float32)
        return s
    if op == "matmul":
        T, N, K = case["rows"], case["out"], case["inner"]

        def codes(rows):                        # rows quantised to their largest value
            v = torch.randn(rows, K, generator=g, device="cuda")
            top = v.abs().amax(1, keepdim=True)
            return torch.round(v * (127.0 / top)).to(torch.int8), (top[:, 0] / 127.0)

        xq, xs = codes(T)
        wq, ws = codes(N)
        return dict(op=op, xq=xq, xs=xs, wq=wq, ws=ws / math.sqrt(K), dtype=dt,
                    bias=normal(N, dtype=torch.float32) if case["bias"] else None)
    T, D = case["rows"], case["width"]
    s = dict(op=op, x=normal(T, D))
    if op != "quantize":
        rd = TYPES[case["residual"]]
        s["residual"] = normal(T, D, dtype=rd, scale=2.0)
        s["weight"] = 1.0 + 0.2 * normal(D, dtype=torch.float32)
        if op == "norm_train":
            s["grad_y"] = normal(T, D)
            s["grad_h"] = normal(T, D, dtype=rd)
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


def _gates(s):
    x, r, i = s["x"].float(), torch.sigmoid(s["gate_a"].float()), torch.sigmoid(s["gate_x"].float())
    lam = s["lam"]
    rate = DECAY_SCALE * (torch.clamp(lam, min=0) + torch.log1p(torch.exp(-lam.abs())))
    loga = -rate * r
    return x, r, i, loga, torch.exp(loga), torch.sqrt(-torch.expm1(2 * loga))


def _scan_forward(s):
    x, r, i, loga, a, m = _gates(s)
    first = s["starts"].long()
    last = first + s["lens"].long() - 1
    h0 = s["slots"] * (s["resume"] != 0)[:, None]
    b = m * i * x
    b[first] += a[first] * h0
    c = a.clone()
    c[first] = 0
    h = _linear_scan(c, b, s["longest"])
    s["slots"].copy_(h[last])
    return (x, r, i, loga, a, m), first, last, h0, h


def _scan(s):
    if own:
        from state_space_model_ssm_gb300 import ssm_gated_scan
        y = ssm_gated_scan(s["slots"], s["x"], s["gate_a"], s["gate_x"], s["lam"], s["starts"], s["lens"], s["resume"],
                           decay_scale=DECAY_SCALE)
        return {"y": y, "slots": s["slots"]}
    h = _scan_forward(s)[-1]
    return {"y": h.to(s["x"].dtype), "slots": s["slots"]}


def _scan_train(s):
    if own:
        from state_space_model_ssm_gb300 import gated_scan_chunk_states, ssm_gated_scan, ssm_gated_scan_backward
        T, C = s["x"].shape
        chunks = gated_scan_chunk_states(s["slots"].shape[0], T, C, device=s["x"].device)
        y = ssm_gated_scan(s["slots"], s["x"], s["gate_a"], s["gate_x"], s["lam"], s["starts"], s["lens"], s["resume"],
                           decay_scale=DECAY_SCALE, chunk_states=chunks)
        gx, gga, ggx, glam, gslots = ssm_gated_scan_backward(
            s["grad_y"], s["x"], s["gate_a"], s["gate_x"], s["lam"], chunks, s["starts"], s["lens"], s["resume"],
            decay_scale=DECAY_SCALE, grad_state=s["grad_slots"])
        return {"y": y, "slots": s["slots"], "grad_x": gx, "grad_gate_a": gga, "grad_gate_x": ggx, "grad_lam": glam,
                "grad_slots": gslots}
    (x, r, i, loga, a, m), first, last, h0, h = _scan_forward(s)
    before = torch.cat([h[:1], h[:-1]])
    before[first] = h0
    c = torch.cat([a[1:], a[:1]])
    c[last] = 0
    gy = s["grad_y"].to(torch.float32, copy=True)
    gy[last] += s["grad_slots"]
    g = _linear_scan(c.flip(0), gy.flip(0), s["longest"]).flip(0)
    dloga = g * (a * before - torch.where(m > 0, a * a / m, 0.0) * i * x)
    dt = s["x"].dtype
    return {"y": h.to(dt), "slots": s["slots"],
            "grad_x": (g * m * i).to(dt),
            "grad_gate_a": (dloga * loga * (1 - r)).to(dt),
            "grad_gate_x": (g * m * x * i * (1 - i)).to(dt),
            "grad_lam": (-DECAY_SCALE * torch.sigmoid(s["lam"])) * (dloga * r).sum(0),
            "grad_slots": a[first] * g[first] * (s["resume"] != 0)[:, None]}


def _codes(v):
    """(codes, factor): v in 8 bits a row."""
    top = v.abs().amax(1, keepdim=True)
    f = torch.clamp(torch.full_like(top, 127.0) / top, max=FLT_MAX)
    return torch.round(v * f).to(torch.int8), f


def _sum_and_inverse(s):
    h = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    hf = h.float()
    return h, hf, 1.0 / torch.sqrt((hf * hf).mean(1, keepdim=True) + EPS)


def _norm_int8(s):
    if own:
        from state_space_model_ssm_gb300 import ssm_add_norm
        q, scale, h = ssm_add_norm(s["x"], s["weight"], s["residual"], eps=EPS, quant="int8")
    else:
        h, hf, inv = _sum_and_inverse(s)
        q, f = _codes(hf * s["weight"])
        scale = (inv / f)[:, 0]
    return {"h": h, "scale": scale, "values": q * scale[:, None]}


def _norm_train(s):
    if own:
        from state_space_model_ssm_gb300 import ssm_add_norm, ssm_add_norm_backward
        y, h = ssm_add_norm(s["x"], s["weight"], s["residual"], eps=EPS)
        gin, gw = ssm_add_norm_backward(s["grad_y"], h, s["weight"], grad_h=s["grad_h"], eps=EPS)
        return {"y": y, "h": h, "grad_in": gin, "grad_weight": gw}
    h, hf, inv = _sum_and_inverse(s)
    w, gy = s["weight"], s["grad_y"].float()
    gw = gy * w
    gin = s["grad_h"].float() + inv * gw - hf * inv ** 3 * (hf * gw).mean(1, keepdim=True)
    return {"y": (hf * inv * w).to(s["x"].dtype), "h": h, "grad_in": gin.to(h.dtype),
            "grad_weight": (gy * hf * inv).sum(0)}


def _quantize(s):
    if own:
        from state_space_model_ssm_gb300 import ssm_quantize_rows
        q, scale = ssm_quantize_rows(s["x"])
    else:
        q, f = _codes(s["x"].float())
        scale = (1.0 / f)[:, 0]
    return {"scale": scale, "values": q * scale[:, None]}


def _matmul(s):
    if own:
        from state_space_model_ssm_gb300 import ssm_int8_matmul
        return ssm_int8_matmul(s["xq"], s["xs"], s["wq"], s["ws"], bias=s["bias"], out_dtype=s["dtype"])
    out = (s["xq"].float() @ s["wq"].float().t()) * s["xs"][:, None] * s["ws"]
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(s["dtype"])


RUN = {"scan": _scan, "scan_train": _scan_train, "norm_int8": _norm_int8, "norm_train": _norm_train,
       "quantize": _quantize, "matmul": _matmul}


# ---- the definitions in 64 bits ----


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("scan", "scan_train"):
        return _exact_scan(case, s)
    d = torch.float64
    if s["op"] == "matmul":
        out = torch.einsum("tk,nk->tn", s["xq"].to(d), s["wq"].to(d)) * s["ws"].to(d)
        out *= s["xs"].to(d)[:, None]
        return out if s["bias"] is None else out + s["bias"].to(d)
    if s["op"] == "quantize":
        v, inv, out = s["x"].float(), 1.0, {}
    else:
        h = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)      # h is held in the residual's type
        inv = torch.rsqrt(h.to(d).square().mean(1) + EPS)
        v, out = h.float() * s["weight"], {"h": h.to(d)}
    if s["op"] == "norm_train":
        hn = h.to(d) * inv[:, None]                                               # gradients through n = h inv
        gn = s["grad_y"].to(d) * s["weight"].to(d)
        out["y"] = hn * s["weight"].to(d)
        out["grad_weight"] = torch.einsum("tk,tk->k", s["grad_y"].to(d), hn)
        out["grad_in"] = s["grad_h"].to(d) + inv[:, None] * (gn - hn * torch.einsum("tk,tk->t", gn, hn)[:, None] / case["width"])
        return out
    # v and the factor are 32-bit values by definition: the codes are theirs
    v = v.cpu().numpy()
    f = np.minimum(np.float32(127) / np.abs(v).max(1), np.float32(FLT_MAX))
    q = np.rint(v * f[:, None]).astype(np.float64)
    scale = (inv.cpu().numpy() if s["op"] == "norm_int8" else 1.0) / f.astype(np.float64)
    out["scale"], out["values"] = torch.from_numpy(scale), torch.from_numpy(q * scale[:, None])
    return out


def _exact_scan(case, s):
    """Token by token; the sequences side by side, each as long as the longest."""
    d, lens = torch.float64, _case_lens(case)
    n, L, C = len(lens), max(lens), case["channels"]
    if n * L * C > (224 << 20):
        return None
    place = torch.tensor([k * L + t for k, v in enumerate(lens) for t in range(v)], device="cuda")
    inside = torch.zeros(n * L, dtype=torch.bool, device="cuda").index_fill_(0, place, True).view(n, L)

    def wide(v):
        return torch.zeros(n * L, C, dtype=d, device="cuda").index_copy_(0, place, v.to(d)).view(n, L, C)

    def packed(v):
        return v.reshape(n * L, C)[place]

    r, i = torch.special.expit(wide(s["gate_a"])), torch.special.expit(wide(s["gate_x"]))
    lam = s["lam"].to(d)
    rate = DECAY_SCALE * torch.nn.functional.softplus(lam)
    a = torch.exp(-rate * r)
    v = torch.sqrt(-torch.expm1(-2 * rate * r)) * i * wide(s["x"])
    a.masked_fill_(~inside[:, :, None], 1.0)                        # past a sequence's end the state stays
    v.masked_fill_(~inside[:, :, None], 0.0)
    h = s["slots"].to(d) * (s["resume"] != 0)[:, None]
    hs = torch.empty(n, L + 1, C, dtype=d, device="cuda")
    hs[:, 0] = h
    for t in range(L):
        h = torch.addcmul(v[:, t], a[:, t], h)
        hs[:, t + 1] = h
    out = {"y": packed(hs[:, 1:]), "slots": h}
    if s["op"] == "scan":
        return out
    gy, g = wide(s["grad_y"]), s["grad_slots"].to(d)
    gs = torch.empty(n, L, C, dtype=d, device="cuda")
    for t in range(L - 1, -1, -1):
        g = g + gy[:, t]
        gs[:, t] = g
        g = g * a[:, t]
    x, m = wide(s["x"]), torch.sqrt(-torch.expm1(-2 * rate * r))
    da = gs * (hs[:, :-1] - a / m * i * x)                          # through a = exp(-rate r) and m = sqrt(1 - a^2)
    dr = da * a * -rate
    gate = inside[:, :, None]
    out["grad_x"] = packed(gs * m * i)
    out["grad_gate_x"] = packed(gs * m * x * i * (1 - i))
    out["grad_gate_a"] = packed(dr * r * (1 - r))
    out["grad_lam"] = (da * a * r * gate).sum((0, 1)) * -DECAY_SCALE * torch.special.expit(lam)
    out["grad_slots"] = g * (s["resume"] != 0)[:, None]
    return out
