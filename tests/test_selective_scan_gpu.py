"""Parity of the selective scan with a decay for each channel and state (forward, backward) with the float64
oracle (needs a GB300).  Bounds: ``model_helpers.scan_bounds``."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from oracle import model as om
from tests.model_helpers import DTYPES, close, np64, scan_bounds, state_range

pytestmark = pytest.mark.gpu
NAMES = ("grad_x", "grad_dt", "grad_A", "grad_B", "grad_C", "grad_D", "grad_z", "grad_dt_bias", "grad_slots")


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _case(C, N, lens, resume=None, dtype=torch.float32, seed=0, groups=1, gate=True, skip=True, bias=True, softplus=True,
          starts=None, n_tokens=None):
    g = torch.Generator().manual_seed(seed)
    n = len(lens)
    starts = list(starts) if starts is not None else [int(v) for v in np.cumsum([0] + list(lens[:-1]))]
    T = n_tokens if n_tokens is not None else sum(lens)
    wide, bc = torch.randn(T, 2 * C, generator=g).to(dtype).cuda(), torch.randn(T, 6 + 2 * groups * N, generator=g).to(dtype).cuda()
    resume = [k % 2 for k in range(n)] if resume is None else resume
    slots = torch.randn(n, C, N, generator=g)
    for k, f in enumerate(resume):
        if not f:
            slots[k] = float("nan")                       # never read
    dt = torch.randn(T, C, generator=g) * 0.7
    dt = dt if softplus else dt.abs() * 0.2
    i32 = dict(dtype=torch.int32, device="cuda")
    c = dict(x=wide[:, :C], dt=dt.to(dtype).cuda(), z=wide[:, C:] if gate else None, B=bc[:, 6:6 + groups * N],
             C=bc[:, 6 + groups * N:], A=(-torch.exp(torch.randn(C, N, generator=g) * 0.7)).cuda(), slots=slots.cuda(),
             D=torch.randn(C, generator=g).cuda() if skip else None,
             dt_bias=(torch.randn(C, generator=g) - 1).cuda() if bias else None)
    c.update(starts=torch.tensor(starts, **i32), lens=torch.tensor(list(lens), **i32), resume=torch.tensor(resume, **i32),
             host=(starts, list(lens), resume), softplus=softplus, groups=groups,
             grad_y=torch.randn(T, C, generator=g).to(dtype).cuda(), grad_state=torch.randn(n, C, N, generator=g).cuda())
    return c


def _options(c):
    return dict(z=c["z"], dt_bias=c["dt_bias"], dt_softplus=c["softplus"], n_groups=c["groups"])


def _forward(c, train=False, y=None, **kw):
    slots = c["slots"].clone()
    if y is None:
        y = torch.full(c["x"].shape, float("nan"), dtype=c["x"].dtype, device="cuda")
    ch = pkg.selective_scan_chunk_states(slots.shape[0], c["x"].shape[0], *c["A"].shape) if train else None
    pkg.ssm_selective_scan(slots, c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["starts"], c["lens"], c["resume"], y,
                           chunk_states=ch, **_options(c), **kw)
    return y, slots, ch


def _backward(c, ch, **kw):
    nan = {k: torch.full_like(v, float("nan")) for k, v in (("grad_x", c["grad_y"]), ("grad_dt", c["grad_y"]))}
    nan.update({k: torch.full(c["B"].shape, float("nan"), dtype=c["x"].dtype, device="cuda") for k in ("grad_B", "grad_C")})
    if c["z"] is not None:
        nan["grad_z"] = torch.full_like(c["grad_y"], float("nan"))
    nan.update(kw)
    out = pkg.ssm_selective_scan_backward(c["grad_y"], c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], ch, c["starts"],
                                          c["lens"], c["resume"], grad_state=c["grad_state"], **_options(c), **nan)
    return dict(zip(NAMES, out))


def _ref(c):
    a = {k: None if c[k] is None else np64(c[k]) for k in ("slots", "x", "dt", "A", "B", "C", "D", "z", "dt_bias")}
    return [a[k] for k in ("slots", "x", "dt", "A", "B", "C", "D")] + list(c["host"]), dict(
        z=a["z"], dt_bias=a["dt_bias"], softplus=c["softplus"], groups=c["groups"])


def _check(c, y, slots, grads=None, blocks=11):
    args, kw = _ref(c)
    y_ref, s_ref, _ = om.selective_scan(*args, **kw)
    gy, gs = (np64(c["grad_y"]), np64(c["grad_state"])) if grads is not None else (None, None)
    b = scan_bounds(*args, **kw, grad_y=gy, grad_state=gs, blocks=blocks)
    own = ~np.isnan(y_ref[:, 0])
    rows, dtype = torch.from_numpy(own), c["x"].dtype
    # Without softplus a step may be negative and a state grow without bound.  What passes through a state or a state's
    # gradient above the largest fp32 value (3.4e38) has no fp32 value: those channels are not compared, nor sums
    # over channels of their sequences' tokens.
    held = np.ones((len(c["host"][0]), c["x"].shape[1]), dtype=bool)
    if not c["softplus"]:
        held = state_range(*args, **kw, grad_y=gy, grad_state=gs) < 3.4e38
    t_held = np.ones(c["x"].shape, dtype=bool)
    for k, (s, n) in enumerate(zip(*c["host"][:2])):
        t_held[s:s + n] = held[k]
    assert held.mean() > 0.5

    def compare(got, ref, bound, mask, dtype=torch.float32):
        got = torch.where(torch.from_numpy(mask).to(got.device), got, torch.zeros((), dtype=got.dtype, device=got.device))
        close(got, np.where(mask, ref, 0.0), np.where(mask, bound, 0.0), dtype)

    compare(y[rows], y_ref[own], b["y"][own], t_held[own], dtype)
    compare(slots, s_ref, b["slots"], np.broadcast_to(held[:, :, None], s_ref.shape))
    assert torch.isnan(y[~rows]).all()
    if grads is None:
        return
    g = om.selective_scan_backward(gy, gs, *args, **kw)
    g["slots"] = g.pop("initial_state")
    for name, got in grads.items():
        ref = g[name[5:]]
        if got is None:
            continue
        if name in ("grad_A", "grad_D", "grad_dt_bias"):
            compare(got, ref, b[name], np.broadcast_to(held.all(0)[:, None] if ref.ndim == 2 else held.all(0), ref.shape))
        elif name == "grad_slots":
            compare(got, ref, b[name], np.broadcast_to(held[:, :, None], ref.shape))
        else:
            mask = t_held if name in ("grad_x", "grad_dt", "grad_z") else np.broadcast_to(t_held.all(1)[:, None], ref.shape)
            compare(got[rows], ref[own], b[name][own], mask[own], dtype)
            assert torch.isnan(got[~rows]).all(), name


LENS = {"one": [1], "decode": [1] * 5, "edges": [7, 8, 9, 15, 16, 17], "empty": [0, 3, 0, 1], "segments": [300],
        "ragged": [1, 3, 25, 130, 64, 0, 200]}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("C,N", [(1, 1), (6, 16), (33, 5), (70, 13), (64, 16), (36, 32), (20, 64), (9, 100), (8, 128)])
@pytest.mark.parametrize("lens", list(LENS))
def test_both_directions(lens, C, N, dtype):
    c = _case(C, N, LENS[lens], dtype=DTYPES[dtype], seed=C + N)
    y, slots, ch = _forward(c, train=True)
    _check(c, y, slots, _backward(c, ch))


@pytest.mark.parametrize("gate,skip,bias,softplus", [(0, 0, 0, 0), (0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0)])
def test_options(gate, skip, bias, softplus):
    c = _case(40, 16, [50, 20], seed=11, gate=bool(gate), skip=bool(skip), bias=bool(bias), softplus=bool(softplus))
    y, slots, ch = _forward(c, train=True)
    grads = _backward(c, ch)
    assert (grads["grad_z"] is None) == (not gate) and (grads["grad_D"] is None) == (not skip)
    assert (grads["grad_dt_bias"] is None) == (not bias)
    _check(c, y, slots, grads)


@pytest.mark.parametrize("groups,C", [(2, 70), (4, 36), (5, 15)])
def test_groups(groups, C):
    c = _case(C, 16, [90, 33], dtype=torch.bfloat16, seed=12, groups=groups)
    y, slots, ch = _forward(c, train=True)
    _check(c, y, slots, _backward(c, ch))


def test_unowned_tokens_and_order():
    """Sequences out of order with gaps between them, all resuming: rows of no sequence stay as they were."""
    for C in (34, 96):
        c = _case(C, 16, [70, 5, 130], resume=[1, 1, 1], seed=3, starts=[140, 2, 8], n_tokens=215, dtype=torch.bfloat16)
        y, slots, ch = _forward(c, train=True)
        _check(c, y, slots, _backward(c, ch))


@pytest.mark.parametrize("which", ["x", "dt", "z", "grad_y", "y", "B"])
def test_odd_pointers(which):
    """One tensor starts at an odd element, so no two of its channels are an aligned word."""
    c = _case(64, 16, [40], dtype=torch.bfloat16, seed=5)
    width = 16 if which == "B" else 64
    wide = torch.zeros(40, width + 3, dtype=torch.bfloat16, device="cuda")
    part = wide[:, 1:1 + width]
    if which != "y":
        part.copy_(c[which])
        c[which] = part
    y, slots, ch = _forward(c, train=True, y=part if which == "y" else None)
    _check(c, y, slots, _backward(c, ch))
    assert (wide[:, 0] == 0).all() and (wide[:, 1 + width:] == 0).all()


def test_many_segments_and_long_sequences():
    """One long sequence with few channels (dozens of segments a pass), and a long one among short ones."""
    assert pkg.selective_scan_workspace_bytes(1, 5000, 24, 16) > 0
    c = _case(24, 16, [5000], resume=[1], seed=9)
    y, slots, ch = _forward(c, train=True)
    _check(c, y, slots, _backward(c, ch))
    c = _case(16, 8, [1] * 7 + [2000], seed=10, dtype=torch.bfloat16)
    y, slots, ch = _forward(c, train=True)
    _check(c, y, slots, _backward(c, ch))


def test_many_sequences_none_of_them_cut():
    c = _case(320, 16, [70] * 400, seed=13)
    y, slots, ch = _forward(c, train=True)
    grads = _backward(c, ch)
    for k in (0, 7, 399):                                  # sequences by themselves
        s = dict(c, host=([0], [70], [c["host"][2][k]]))
        rows = slice(70 * k, 70 * k + 70)
        for name in ("x", "dt", "z", "B", "C", "grad_y"):
            s[name] = c[name][rows]
        s["slots"], s["grad_state"] = c["slots"][k:k + 1], c["grad_state"][k:k + 1]
        part = {n: v[rows] for n, v in grads.items() if n in ("grad_x", "grad_dt", "grad_z", "grad_B", "grad_C")}
        part["grad_slots"] = grads["grad_slots"][k:k + 1]
        _check(s, y[rows], slots[k:k + 1], part)


def test_a_long_sequence_among_single_tokens():
    """Most sequences are left whole, one is cut."""
    lens = [1] * 120 + [900] + [1] * 80 + [0, 130]
    c = _case(48, 16, lens, seed=17, dtype=torch.bfloat16)
    y, slots, ch = _forward(c, train=True)
    _check(c, y, slots, _backward(c, ch))


def test_step_by_step_equals_one_call():
    c = _case(128, 16, [40], resume=[1], seed=6)
    s = c["slots"].clone()
    one, zero = (torch.full((1,), v, dtype=torch.int32, device="cuda") for v in (1, 0))
    row = lambda name, t: c[name][t:t + 1]                 # noqa: E731
    ys = [pkg.ssm_selective_scan(s, row("x", t), row("dt", t), c["A"], row("B", t), row("C", t), c["D"], zero, one, one,
                                 z=row("z", t), dt_bias=c["dt_bias"], dt_softplus=True) for t in range(40)]
    _check(c, torch.cat(ys), s)


@pytest.mark.parametrize("N", [13, 16])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_no_number_stays_in_its_channel(value, N):
    """An input that is no finite number reaches its own channel's later tokens, and B's and C's gradients."""
    c = _case(70, N, [100, 100], resume=[0, 0], seed=8)
    c["x"][120, 5] = value
    y, slots, ch = _forward(c, train=True)
    bad = ~torch.isfinite(y)
    assert bad[120:200, 5].all() and int(bad.sum()) == 80
    # an infinity times B is infinite in every state (B is not 0 here); only padding would make it a NaN
    assert not torch.isfinite(slots[1, 5]).any() and int((~torch.isfinite(slots)).sum()) == N
    if value == float("inf"):
        assert torch.isinf(slots[1, 5]).all()
    g = _backward(c, ch)
    assert torch.isfinite(g["grad_x"][:100]).all() and torch.isfinite(g["grad_A"][torch.arange(70) != 5]).all()
    assert torch.isfinite(g["grad_slots"]).all() or int((~torch.isfinite(g["grad_slots"])).sum()) <= N
    clean = torch.arange(70) != 5
    assert torch.isfinite(g["grad_dt"][:, clean.cuda()]).all()


def test_steps_at_their_ends():
    """Steps of 0 (the state stays), of thousands (it is forgotten), and A = 0 (it adds up)."""
    c = _case(32, 16, [60], resume=[1], seed=7)
    c["dt"][:, 0::4] = float("-inf")
    c["dt"][:, 1::4] = 5000.0
    c["A"][2] = 0.0
    y, slots, ch = _forward(c, train=True)
    _check(c, y, slots, _backward(c, ch))
    assert torch.equal(slots[0, 0], c["slots"][0, 0])


def test_a_sequence_outside_the_rows_counts_as_empty():
    c = _case(32, 16, [20, 10], resume=[1, 1], seed=14)
    c["starts"][1] = 25                                    # 25 + 10 > 30
    y, slots, _ = _forward(c)
    assert torch.equal(slots[1], c["slots"][1]) and torch.isnan(y[20:]).all() and torch.isfinite(y[:20]).all()


def test_same_bits_every_time_and_in_two_streams():
    c = _case(200, 16, [700, 300], seed=15, dtype=torch.bfloat16)
    y, slots, ch = _forward(c, train=True)
    first = _backward(c, ch)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for s in streams * 3:                                  # overlapping calls, each with its own workspace
        with torch.cuda.stream(s):
            yy, ss, hh = _forward(c, train=True)
            got.append((yy, ss, hh, _backward(c, hh)))
    torch.cuda.synchronize()
    for yy, ss, hh, g in got:
        assert torch.equal(yy, y) and torch.equal(ss, slots)
        assert all(torch.equal(g[k], first[k]) for k in NAMES)


def test_captured_and_replayed_beside_eager_calls():
    c = _case(96, 16, [400, 77], seed=16, dtype=torch.bfloat16)
    y, slots, ch = _forward(c, train=True)
    eager = _backward(c, ch)
    s0, yg = c["slots"].clone(), torch.empty_like(y)
    ws = torch.empty(max(1, pkg.selective_scan_workspace_bytes(2, 477, 96, 16)), dtype=torch.uint8, device="cuda")
    wb = torch.empty(pkg.selective_scan_backward_workspace_bytes(2, 477, 96, 16), dtype=torch.uint8, device="cuda")
    held = _backward(c, ch, workspace=wb)                  # also loads every kernel before the capture
    slots_g, chg = s0.clone(), torch.empty_like(ch)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.ssm_selective_scan(slots_g, c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["starts"], c["lens"], c["resume"],
                               yg, chunk_states=chg, workspace=ws, **_options(c))
        _backward(c, chg, workspace=wb, **{k: held[k] for k in ("grad_x", "grad_dt", "grad_B", "grad_C", "grad_z")})
    for _ in range(3):
        slots_g.copy_(s0)
        held["grad_x"].zero_()
        graph.replay()
        again = _backward(c, ch)                           # an eager call of the same tensors in between
        torch.cuda.synchronize()
        assert torch.equal(yg, y) and torch.equal(slots_g, slots) and torch.equal(held["grad_x"], eager["grad_x"])
        assert all(torch.equal(again[k], eager[k]) for k in NAMES)


@pytest.mark.parametrize("N", [13, 16])
@pytest.mark.parametrize("left", [0.0, 1e-35])
def test_segments_whose_decay_overflows(left, N):
    """Decays that grow (A above 0): over a segment of 64 tokens by 2^130, which fp32 does not hold, on states of `left`.
    Token by token everything is finite; so it is in segments.  Sequences: growth on small states, ordinary tokens, growth
    behind the last gradient."""
    lens = [256, 320]
    c = _case(12, N, lens, resume=[1, 1], seed=18, softplus=False, bias=False, gate=False)
    assert pkg.selective_scan_workspace_bytes(2, 576, 12, N) > 0
    g = torch.Generator().manual_seed(19)
    c["A"] = (0.7 + 0.01 * torch.rand(12, N, generator=g)).cuda()
    c["dt"] = torch.full((576, 12), -0.3, device="cuda")
    c["x"] = c["x"] * 1e-8
    c["grad_y"] *= 1e-8
    c["slots"], c["grad_state"] = c["slots"].clone(), c["grad_state"] * left
    c["slots"][:] = left * torch.randn(2, 12, N, generator=g).cuda()
    for start, n in zip((0, 256), lens):
        for part in (slice(start, start + 64), slice(start + n - 64, start + n)):
            c["dt"][part] = 130 * 0.6931471805599453 / 64 / 0.7     # 130 / 64 of an exponent of 2 a token at least
            c["x"][part] = 0.0
            c["grad_y"][part] = 0.0
    y, slots, ch = _forward(c, train=True)
    grads = _backward(c, ch)
    assert torch.isfinite(slots).all() and all(torch.isfinite(v).all() for v in grads.values() if v is not None)
    _check(c, y, slots, grads)
