"""Parity of the short causal convolution on strided rows (forward, backward) with the float64 oracle, and with
``ssm_conv1d`` where both apply (needs a GB300).  Bounds: ``model_helpers.conv_bounds``."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from state_space_model_ssm_gb300 import binding as bd
from oracle import model as om
from tests.model_helpers import DTYPES, close, conv_bounds, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _case(C, K, lens, resume=None, dtype=torch.float32, seed=0, bias=True, silu=True, starts=None, n_tokens=None, off=0):
    g = torch.Generator().manual_seed(seed)
    n = len(lens)
    starts = list(starts) if starts is not None else [int(v) for v in np.cumsum([0] + list(lens[:-1]))]
    T = n_tokens if n_tokens is not None else sum(lens)
    resume = [k % 2 for k in range(n)] if resume is None else resume
    slots = torch.randn(n, C, K - 1, generator=g)
    for k, f in enumerate(resume):
        if not f:
            slots[k] = float("nan")
    wide = torch.randn(T, 2 * C + 4, generator=g).to(dtype).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(x=wide[:, off:off + C], weight=torch.randn(C, K, generator=g).cuda(), slots=slots.cuda(), silu=silu,
                bias=torch.randn(C, generator=g).cuda() if bias else None, host=(starts, list(lens), resume),
                starts=torch.tensor(starts, **i32), lens=torch.tensor(list(lens), **i32), resume=torch.tensor(resume, **i32),
                grad_out=torch.randn(T, C, generator=g).to(dtype).cuda(), grad_state=torch.randn(n, C, K - 1, generator=g).cuda())


def _run(c, **kw):
    slots = c["slots"].clone()
    out = torch.full(c["grad_out"].shape, float("nan"), dtype=c["x"].dtype, device="cuda")
    gx = torch.full_like(out, float("nan"))
    pkg.ssm_causal_conv(c["x"], c["weight"], slots, c["starts"], c["lens"], c["resume"], out, bias=c["bias"], silu=c["silu"])
    g = pkg.ssm_causal_conv_backward(c["grad_out"], c["x"], c["weight"], c["starts"], c["lens"], c["resume"], bias=c["bias"],
                                     silu=c["silu"], initial_state=c["slots"], grad_state=c["grad_state"], grad_x=gx, **kw)
    return out, slots, dict(zip(("x", "weight", "bias", "slots"), g))


def _check(c, out, slots, grads):
    a = {k: None if c[k] is None else np64(c[k]) for k in ("x", "weight", "slots", "bias", "grad_out", "grad_state")}
    args, kw = (a["x"], a["weight"], a["slots"], *c["host"]), dict(bias=a["bias"], silu=c["silu"])
    ref, after, _ = om.causal_conv(*args, **kw)
    b = conv_bounds(*args, **kw, grad_out=a["grad_out"], grad_state=a["grad_state"])
    own = ~np.isnan(ref[:, 0])
    rows, dtype = torch.from_numpy(own), c["x"].dtype
    close(out[rows], ref[own], b["out"][own], dtype)
    assert torch.isnan(out[~rows]).all() and torch.isnan(grads["x"][~rows]).all()
    assert np.array_equal(np64(slots), after)              # inputs as they are
    g = om.causal_conv_backward(a["grad_out"], a["grad_state"], *args, **kw)
    close(grads["x"][rows], g["x"][own], b["grad_x"][own], dtype)
    close(grads["weight"], g["weight"], b["grad_weight"])
    close(grads["slots"], g["initial_state"], b["grad_slots"])
    assert (grads["bias"] is None) == (c["bias"] is None)
    if c["bias"] is not None:
        close(grads["bias"], g["bias"], b["grad_bias"])


LENS = {"one": [1], "short": [1, 2, 3, 0, 4, 5], "runs": [7, 8, 9, 31, 32, 33], "spans": [400, 3, 70]}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("C,K", [(1, 4), (2, 1), (6, 2), (31, 3), (64, 4), (130, 5), (300, 8), (12, 6), (9, 7)])
@pytest.mark.parametrize("lens", list(LENS))
def test_both_directions(lens, C, K, dtype):
    c = _case(C, K, LENS[lens], dtype=DTYPES[dtype], seed=C + K)
    _check(c, *_run(c))


@pytest.mark.parametrize("bias,silu,off", [(0, 1, 0), (1, 0, 0), (0, 0, 1), (1, 1, 1), (1, 1, 2)])
def test_options_and_odd_pointers(bias, silu, off):
    c = _case(64, 4, [50, 20], seed=1, bias=bool(bias), silu=bool(silu), off=off, dtype=torch.bfloat16)
    _check(c, *_run(c))


def test_unowned_tokens_and_order():
    c = _case(64, 4, [70, 5, 130], resume=[1, 0, 1], seed=3, starts=[140, 2, 8], n_tokens=215, dtype=torch.bfloat16)
    _check(c, *_run(c))


def test_all_fresh_without_slots():
    c = _case(64, 4, [50, 2, 0], resume=[0, 0, 0], seed=4)
    out, slots, with_slots = _run(c)
    g = pkg.ssm_causal_conv_backward(c["grad_out"], c["x"], c["weight"], c["starts"], c["lens"], bias=c["bias"],
                                     grad_state=c["grad_state"])
    assert g[3] is None and torch.equal(g[0], with_slots["x"]) and torch.equal(g[1], with_slots["weight"])
    assert (with_slots["slots"] == 0).all()


def test_equals_conv1d():
    c = _case(192, 4, [33, 1, 257], seed=5, off=0)
    c["x"] = c["x"].contiguous()
    out, slots, _ = _run(c)
    s1 = c["slots"].clone()
    o1 = pkg.ssm_conv1d(c["x"], c["weight"], s1, c["starts"], c["lens"], c["resume"], bias=c["bias"])
    assert torch.equal(s1, slots)
    close(o1, np64(out), 2 * conv_bounds(*(np64(c[k]) for k in ("x", "weight", "slots")), *c["host"], bias=np64(c["bias"]))["out"])


def test_step_by_step_equals_one_call():
    c = _case(96, 4, [30], resume=[1], seed=6, dtype=torch.bfloat16)
    out, slots, _ = _run(c)
    s = c["slots"].clone()
    one, zero = (torch.full((1,), v, dtype=torch.int32, device="cuda") for v in (1, 0))
    rows = [pkg.ssm_causal_conv(c["x"][t:t + 1], c["weight"], s, zero, one, one, bias=c["bias"]) for t in range(30)]
    assert torch.equal(torch.cat(rows), out) and torch.equal(s, slots)


def test_nan_stays_in_its_window():
    c = _case(66, 4, [100, 100], resume=[0, 0], seed=7)
    c["x"][120, 5] = float("nan")
    out, slots, g = _run(c)
    bad = torch.isnan(out)
    assert bad[120:124, 5].all() and int(bad.sum()) == 4 and torch.isfinite(slots).all()
    clean = torch.arange(66, device="cuda") != 5
    assert torch.isfinite(g["x"][:, clean]).all() and torch.isfinite(g["weight"][clean]).all()
    assert int(torch.isnan(g["x"]).sum()) == 7             # inputs whose outputs share a window with it


def test_streams_graph_and_bits():
    c = _case(256, 4, [900, 40], seed=8, dtype=torch.bfloat16)
    out, slots, g = _run(c)
    torch.cuda.synchronize()
    ws = torch.empty(pkg.causal_conv_backward_workspace_bytes(2, 940, 256, 4), dtype=torch.uint8, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        og, sg, gg = _run(c, workspace=ws)
    graph.replay()
    with torch.cuda.stream(side):
        o2, s2, g2 = _run(c)
    torch.cuda.synchronize()
    for o, s, gr in ((og, sg, gg), (o2, s2, g2)):
        assert torch.equal(o, out) and torch.equal(s, slots) and all(torch.equal(gr[k], g[k]) for k in g)


def test_one_tap_reads_no_flags():
    """A C caller may leave resume_flags out for one tap, also where it has pointers for the (empty) slots."""
    c = _case(66, 1, [40, 7], seed=9)
    out, slots, g = _run(c)
    T, C = c["x"].shape
    spare = torch.full((2, C), 7.0, device="cuda")         # stands for slots of no values: neither read nor written
    gx, gw, gb = torch.empty_like(out), torch.empty_like(c["weight"]), torch.empty_like(c["bias"])
    ws = torch.empty(pkg.causal_conv_backward_workspace_bytes(2, T, C, 1), dtype=torch.uint8, device="cuda")
    p = torch.Tensor.data_ptr
    rc = bd.load().ssm_causal_conv_backward(p(c["grad_out"]), p(spare), p(c["x"]), p(c["weight"]), p(c["bias"]), p(spare),
                                            p(c["starts"]), p(c["lens"]), None, 2, T, C, 1, 1, 0, C, c["x"].stride(0), p(gx),
                                            p(gw), p(gb), p(spare), C, p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == bd.SSM_OK and (spare == 7.0).all()
    assert torch.equal(gx, g["x"]) and torch.equal(gw, g["weight"]) and torch.equal(gb, g["bias"])
