"""Parity of the gated linear recurrence (forward, backward) with the float64 oracle (needs a GB300)."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from oracle import layers as ol
from state_space_model_ssm_gb300 import layers
from tests.layer_helpers import DTYPES, close, gated_bounds, np64

pytestmark = pytest.mark.gpu
C0 = 8.0


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _case(C, lens, resume=None, dtype=torch.float32, seed=0, fused=False, starts=None, n_tokens=None, gate=1.0):
    g = torch.Generator().manual_seed(seed)
    n = len(lens)
    starts = list(starts) if starts is not None else [int(v) for v in np.cumsum([0] + list(lens[:-1]))]
    T = n_tokens if n_tokens is not None else sum(lens)
    wide = torch.randn(T, 3 * C, generator=g)
    wide[:, C:] *= gate
    wide = wide.to(dtype).cuda()
    parts = [wide[:, k * C:(k + 1) * C] for k in range(3)]
    if not fused:
        parts = [p.contiguous() for p in parts]
    lam = torch.log(torch.expm1(-torch.log(torch.rand(C, generator=g) * 0.099 + 0.9)))
    resume = [k % 2 for k in range(n)] if resume is None else resume
    slots = torch.randn(n, C, generator=g)
    for k, f in enumerate(resume):
        if not f:
            slots[k] = float("nan")                       # never read
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(x=parts[0], gate_a=parts[1], gate_x=parts[2], lam=lam.cuda(), slots=slots.cuda(),
                starts=torch.tensor(starts, **i32), lens=torch.tensor(list(lens), **i32),
                resume=torch.tensor(resume, **i32), host=(starts, list(lens), resume),
                grad_y=torch.randn(T, C, generator=g).to(dtype).cuda(), grad_state=torch.randn(n, C, generator=g).cuda())


def _forward(c, train=False, **kw):
    slots = c["slots"].clone()
    y = torch.full(c["x"].shape, float("nan"), dtype=c["x"].dtype, device="cuda")
    ch = pkg.gated_scan_chunk_states(slots.shape[0], *c["x"].shape) if train else None
    pkg.ssm_gated_scan(slots, c["x"], c["gate_a"], c["gate_x"], c["lam"], c["starts"], c["lens"], c["resume"], y,
                       decay_scale=C0, chunk_states=ch, **kw)
    return y, slots, ch


def _ref_args(c):
    return [np64(c["slots"])] + [np64(c[k]) for k in ("x", "gate_a", "gate_x", "lam")] + list(c["host"]) + [C0]


def _check_forward(c, y, slots):
    args = _ref_args(c)
    y_ref, s_ref = ol.gated_scan(*args)
    b = gated_bounds(*args)
    own = ~np.isnan(y_ref[:, 0])
    close(y[torch.from_numpy(own)], y_ref[own], b["y"][own], c["x"].dtype)
    assert torch.isnan(y[torch.from_numpy(~own)]).all()
    close(slots, s_ref, b["slots"])


LENS = {
    "one": [1], "two": [2], "decode": [1] * 5, "edge_of_run": [7, 8, 9], "edge_of_chunk": [63, 64, 65],
    "empty": [0, 3, 0, 1], "long": [1000], "ragged": [1, 3, 25, 150, 513, 64, 0, 200],
}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("C", [1, 31, 64, 66, 200])
@pytest.mark.parametrize("lens", list(LENS))
def test_forward(lens, C, dtype):
    c = _case(C, LENS[lens], dtype=DTYPES[dtype], seed=C)
    _check_forward(c, *_forward(c)[:2])


@pytest.mark.parametrize("train", [False, True])
def test_forward_fused_views_and_unowned_tokens(train):
    """Slices of one projection (token stride 3C), sequences out of order with gaps, all resuming."""
    for C in (33, 96):
        c = _case(C, [70, 5, 130], resume=[1, 1, 1], seed=3, fused=True, starts=[140, 2, 8], n_tokens=215)
        _check_forward(c, *_forward(c, train)[:2])


@pytest.mark.parametrize("where", ["x", "gate_a", "gate_x", "y"])
def test_forward_odd_pointer(where):
    """One tensor starts at an odd element: the pairwise path must not be taken."""
    c = _case(64, [100], dtype=torch.bfloat16, seed=5)
    wide = torch.zeros(100, 67, dtype=torch.bfloat16, device="cuda")
    if where == "y":
        slots = c["slots"].clone()
        y = wide[:, 1:65]
        pkg.ssm_gated_scan(slots, c["x"], c["gate_a"], c["gate_x"], c["lam"], c["starts"], c["lens"], c["resume"], y)
        _check_forward(c, y, slots)
        assert (wide[:, 0] == 0).all() and (wide[:, 65:] == 0).all()
    else:
        wide[:, 1:65] = c[where]
        c[where] = wide[:, 1:65]
        _check_forward(c, *_forward(c)[:2])


def test_step_by_step_equals_one_call_within_bounds():
    c = _case(128, [40], resume=[1], seed=6)
    y, slots, _ = _forward(c)
    s = c["slots"].clone()
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    ys = [pkg.ssm_gated_scan(s, c["x"][t:t + 1], c["gate_a"][t:t + 1], c["gate_x"][t:t + 1], c["lam"], zero, one, one)
          for t in range(40)]
    _check_forward(c, torch.cat(ys), s)


def test_gates_at_their_ends():
    """Shut and open gates and far logits: finite, and the state kept where the recurrence gate is shut."""
    c = _case(64, [90], resume=[1], seed=7)
    c["gate_a"][:, 0::4] = float("-inf")
    c["gate_a"][:, 1::4] = 80.0
    c["gate_x"][:, 2::4] = float("-inf")
    c["gate_a"][:, 3::4] = -30.0
    y, slots, ch = _forward(c, train=True)
    _check_forward(c, y, slots)
    assert torch.equal(slots[0, 0::4], c["slots"][0, 0::4])
    grads = _backward(c, ch)
    assert all(torch.isfinite(v).all() for v in grads)
    _check_backward(c, grads)


def test_nan_stays_in_its_sequence_and_channel():
    c = _case(64, [100, 100], resume=[0, 0], seed=8)
    c["x"][120, 5] = float("nan")
    y, slots, _ = _forward(c)
    bad = torch.isnan(y)
    assert bad[120:, 5].all() and int(bad.sum()) == 80
    assert torch.isnan(slots[1, 5]) and int(torch.isnan(slots).sum()) == 1


def test_long_sequence_passes_its_state():
    """Hundreds of chunks in a row: 40000 tokens, and beside it a batch of 300 short ones."""
    c = _case(64, [40000], resume=[1], seed=9)
    _check_forward(c, *_forward(c)[:2])
    c = _case(32, [17] * 300, seed=10)
    _check_forward(c, *_forward(c)[:2])


def test_invalid_range_counts_as_empty():
    c = _case(32, [10, 10], resume=[1, 1], seed=11)
    c["starts"][1] = 15                                    # 15 + 10 > 20
    y, slots, _ = _forward(c)
    assert torch.isnan(y[10:]).all() and torch.equal(slots[1], c["slots"][1])
    assert not torch.isnan(y[:10]).any()


# ---- backward ----


def _backward(c, ch, **kw):
    return pkg.ssm_gated_scan_backward(c["grad_y"], c["x"], c["gate_a"], c["gate_x"], c["lam"], ch, c["starts"],
                                       c["lens"], c["resume"], decay_scale=C0, grad_state=c["grad_state"], **kw)


def _check_backward(c, grads):
    args = _ref_args(c)
    gy, gs = np64(c["grad_y"]), np64(c["grad_state"])
    ref = ol.gated_scan_backward(gy, gs, *args)
    b = gated_bounds(*args, grad_y=gy, grad_state=gs)
    own = ~np.isnan(ref[0][:, 0])
    sel = torch.from_numpy(own)
    dt = c["x"].dtype
    close(grads[0][sel], ref[0][own], b["grad_x"][own], dt)
    close(grads[1][sel], ref[1][own], b["grad_gate_a"][own], dt)
    close(grads[2][sel], ref[2][own], b["grad_gate_x"][own], dt)
    close(grads[3], ref[3], b["grad_lam"])
    close(grads[4], ref[4], b["grad_slots"])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("C", [1, 31, 64, 200])
@pytest.mark.parametrize("lens", list(LENS))
def test_backward(lens, C, dtype):
    c = _case(C, LENS[lens], dtype=DTYPES[dtype], seed=C + 1)
    _, _, ch = _forward(c, train=True)
    _check_backward(c, _backward(c, ch))


def test_backward_views_gaps_and_fixed_order():
    """Fused inputs, gradients into slices of one tensor, unowned tokens untouched; twice the same bits."""
    C = 96
    c = _case(C, [70, 5, 330], resume=[1, 0, 1], seed=13, fused=True, starts=[340, 2, 8], n_tokens=415)
    y, slots, ch = _forward(c, train=True)
    _check_forward(c, y, slots)
    wide = torch.full((415, 3 * C), 7.0, device="cuda")
    v = [wide[:, k * C:(k + 1) * C] for k in range(3)]
    grads = _backward(c, ch, grad_x=v[0], grad_gate_a=v[1], grad_gate_x=v[2])
    _check_backward(c, grads)
    own = torch.zeros(415, dtype=torch.bool)
    for s, n in zip(*c["host"][:2]):
        own[s:s + n] = True
    assert (wide[~own.cuda()] == 7.0).all()
    again = _backward(c, ch)
    for a, b in zip(grads[3:], again[3:]):
        assert torch.equal(a, b)


def test_backward_long_sequence():
    c = _case(64, [20000], resume=[1], seed=14)
    _, _, ch = _forward(c, train=True)
    _check_backward(c, _backward(c, ch))


def test_training_state_equals_serving_state():
    c = _case(64, [300, 40], seed=15)
    a, b = _forward(c), _forward(c, train=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_other_stream_and_graph():
    """A call on another stream than the current one, and forward and backward captured into a graph."""
    c = _case(64, [500, 77], seed=16)
    want = _forward(c, train=True)
    grads = _backward(c, want[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    slots = c["slots"].clone()
    side.wait_stream(torch.cuda.current_stream())
    y = pkg.ssm_gated_scan(slots, c["x"], c["gate_a"], c["gate_x"], c["lam"], c["starts"], c["lens"], c["resume"],
                           stream=side)
    side.synchronize()
    own = ~torch.isnan(want[0])
    assert torch.equal(y[own], want[0][own]) and torch.equal(slots, want[1])
    slots.copy_(c["slots"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    ch = pkg.gated_scan_chunk_states(2, 577, 64)
    with torch.cuda.graph(graph):
        y = pkg.ssm_gated_scan(slots, c["x"], c["gate_a"], c["gate_x"], c["lam"], c["starts"], c["lens"], c["resume"],
                               decay_scale=C0, chunk_states=ch)
        got = _backward(c, ch)
    for _ in range(2):
        slots.copy_(c["slots"])
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(slots, want[1])
    for a, b in zip(got, grads):
        assert torch.equal(a, b)


def test_refuses_small_workspace():
    c = _case(64, [100], seed=17)
    _, _, ch = _forward(c, train=True)
    ws = torch.empty(128, dtype=torch.uint8, device="cuda")
    with pytest.raises(pkg.SsmScanError) as e:
        _backward(c, ch, workspace=ws)
    assert e.value.status == -1
    need = layers.gated_scan_backward_workspace_bytes(1, 100, 64)
    _check_backward(c, _backward(c, ch, workspace=torch.empty(need, dtype=torch.uint8, device="cuda")))


@pytest.mark.parametrize("C", [30, 64, 129])
@pytest.mark.parametrize("lens", [[1024], [2100], [600, 1, 0, 1500], [64 * 8] * 3])
def test_time_shared_by_a_cluster(lens, C):
    """Few channels and long sequences: clusters of 2 to 8 blocks, lengths that leave some of them
    without a chunk, forward and backward."""
    c = _case(C, lens, resume=[1] * len(lens), seed=C + len(lens))
    y, slots, ch = _forward(c, train=True)
    _check_forward(c, y, slots)
    _check_backward(c, _backward(c, ch))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("C", [1, 33, 64])
def test_many_short_sequences_and_a_long_one(C, dtype):
    """The stepping kernels (16 tokens a sequence or fewer on average): single tokens, fours, odd
    lengths, empty sequences, and one that spans several chunks; forward and backward."""
    lens = [1, 4, 0, 7, 8, 16, 3, 0, 200, 64, 65] + [2] * 25
    c = _case(C, lens, dtype=DTYPES[dtype], seed=C + 40, fused=C == 64)
    assert sum(lens) <= 16 * len(lens)
    y, slots, ch = _forward(c, train=True)
    _check_forward(c, y, slots)
    _check_backward(c, _backward(c, ch))
