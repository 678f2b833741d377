"""Parity of the cross entropy of a projection (loss, gradients) with the float64 oracle (needs a GB300).
Bounds: ``model_helpers.loss_bounds``."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from oracle import model as om
from tests.model_helpers import close, loss_bounds, np64

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _case(T, V, D, dtype=torch.bfloat16, ignored=0.0, seed=0, wide=True, extra=0, off=0, logits=2.0, equal=False):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, D + extra, generator=g).to(dtype).cuda()[:, off:off + D]
    w = (torch.randn(V, D + extra, generator=g) * logits / D ** 0.5).to(dtype).cuda()[:, off:off + D]
    t = torch.randint(0, V, (T,), generator=g)
    t[torch.rand(T, generator=g) < ignored] = -100
    gl = torch.full((T,), 1.0 / max(T, 1)) if equal else torch.randn(T, generator=g)
    return dict(h=h, w=w, t=(t if wide else t.int()).cuda(), gl=gl.cuda(), ignore=-100)


def _run(c, **kw):
    loss, lse = pkg.ssm_linear_cross_entropy(c["h"], c["w"], c["t"], ignore_index=c["ignore"])
    gh, gw = pkg.ssm_linear_cross_entropy_backward(c["gl"], c["h"], c["w"], c["t"], lse, ignore_index=c["ignore"], **kw)
    return loss, lse, gh, gw


def _check(c, loss, lse, gh=None, gw=None):
    h, w, t, gl = np64(c["h"]), np64(c["w"]), c["t"].cpu().numpy().astype(np.int64), np64(c["gl"])
    dtype = c["h"].dtype
    b = loss_bounds(h, w, t, c["ignore"], dtype, gl)
    rl, re = om.linear_cross_entropy(h, w, t, c["ignore"])
    close(loss, rl, b["loss"])
    close(lse, re, b["lse"])
    rh, rw, _ = om.linear_cross_entropy_backward(gl, h, w, t, c["ignore"])
    if gh is not None:
        close(gh, rh, b["grad_hidden"], dtype)
        assert (gh[c["t"] == c["ignore"]] == 0).all()
    if gw is not None:
        close(gw, rw, b["grad_weight"], dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 300, 64), (2, 257, 8), (31, 100, 33), (128, 256, 64), (129, 513, 100),
                                   (257, 1000, 129), (300, 255, 320), (520, 700, 200)])
def test_both_directions(T, V, D, dtype):
    c = _case(T, V, D, TYPES[dtype], seed=T + V)
    _check(c, *_run(c))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("ignored", [0.1, 0.6, 0.97, 1.0])
def test_ignored_rows(ignored, dtype):
    """What stands in ignored rows reaches nothing: they hold NaN and infinities here."""
    c = _case(300, 500, 96, TYPES[dtype], ignored=ignored, seed=3)
    gone = c["t"] == -100
    clean = c["h"].clone()
    c["h"][gone] = float("nan")
    c["h"][gone, 3] = float("inf")
    c["gl"][gone] = float("nan")
    out = _run(c)
    c["h"], c["gl"] = torch.where(gone[:, None], clean, c["h"]), torch.nan_to_num(c["gl"])
    _check(c, *out)
    assert (out[0][gone] == 0).all() and (out[1][gone] == 0).all() and torch.isfinite(out[3]).all()


def test_another_ignored_index_and_32_bit_targets():
    c = _case(200, 300, 64, wide=False, seed=4)
    c["ignore"] = 7
    c["t"][::5] = 7
    _check(c, *_run(c))


@pytest.mark.parametrize("D,extra,off", [(64, 8, 0), (64, 8, 1), (61, 0, 0), (61, 3, 0), (64, 1, 0)])
def test_strides_and_odd_rows(D, extra, off):
    """Rows inside wider ones: described to the copy engine as they are, or packed first."""
    c = _case(70, 333, D, seed=5, extra=extra, off=off)
    out = torch.zeros(70, D + 5, dtype=torch.bfloat16, device="cuda")
    gw = torch.zeros(333, D + 5, dtype=torch.bfloat16, device="cuda")
    got = _run(c, grad_hidden=out[:, 1:1 + D], grad_weight=gw[:, 1:1 + D])
    _check(c, *got)
    for v in (out, gw):
        assert (v[:, 0] == 0).all() and (v[:, 1 + D:] == 0).all()


def test_a_mean_over_many_rows_and_small_probabilities():
    """Equal grad_loss of 1 / T; rows of the vocabulary that are no target have gradients of about 1 / (T V)."""
    for dtype in TYPES.values():
        c = _case(256, 2000, 64, dtype, seed=6, equal=True)
        c["gl"] *= 1024.0 if dtype == torch.float16 else 1.0
        _check(c, *_run(c))


def test_large_logits():
    c = _case(64, 400, 64, seed=7, logits=60.0)
    loss, lse, gh, gw = _run(c)
    assert torch.isfinite(loss).all() and torch.isfinite(gh).all()
    _check(c, loss, lse, gh, gw)


def test_several_pieces_of_the_vocabulary():
    """More rows than one piece of G has room for, ignored ones among them (a piece holds 256 MB here)."""
    T, V, D = 9000, 20000, 64
    c = _case(T, V, D, seed=8, ignored=0.5, equal=True)
    need = pkg.linear_cross_entropy_workspace_bytes(c["h"], c["w"], backward=True)
    assert need < 9216 * 20224 * 2                          # less than G of the whole vocabulary (79 tiles of 256)
    loss, lse, gh, gw = _run(c)
    keep = torch.nonzero(c["t"] != -100)[:, 0]
    rows = keep[::200]
    logits = c["h"].double() @ c["w"].double().t()
    p = torch.softmax(logits, 1)
    p[keep, c["t"][keep]] -= 1
    p[c["t"] == -100] = 0
    p *= c["gl"].double()[:, None]
    # the bound of a row's own terms (rows and columns of the full product are too many for the host)
    sub = dict(c, h=c["h"][rows], t=c["t"][rows], gl=c["gl"][rows])
    b = loss_bounds(np64(sub["h"]), np64(c["w"]), sub["t"].cpu().numpy(), -100, torch.bfloat16, np64(sub["gl"]))
    close(gh[rows], np64(p[rows] @ c["w"].double()), b["grad_hidden"], torch.bfloat16)
    half = 2.0 ** -9
    ref = p.t() @ c["h"].double()
    mag = p.abs().t() @ c["h"].double().abs()
    tol = (half + 1e-4) * mag * 1.01 + half * ref.abs() + 2 * (T + 8) * 2.0 ** -24 * mag
    assert ((gw.double() - ref).abs() <= tol).all()
    assert (gh[c["t"] == -100] == 0).all()


def test_target_outside_the_vocabulary():
    c = _case(40, 100, 64, seed=9)
    c["t"][3], c["t"][7] = 100, -5
    loss, lse, gh, gw = _run(c)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[3] = bad[7] = True
    assert torch.isnan(loss[bad]).all() and torch.isfinite(loss[~bad]).all() and torch.isfinite(lse).all()
    assert torch.isnan(gh[bad]).all() and torch.isfinite(gh[~bad]).all() and torch.isnan(gw).any()


def test_nan_in_a_row_that_counts():
    c = _case(40, 300, 64, seed=10)
    c["h"][5, 2] = float("nan")
    loss, lse, gh, gw = _run(c)
    assert torch.isnan(loss[5]) and int(torch.isnan(loss).sum()) == 1 and torch.isnan(gh[5]).all()
    assert int(torch.isnan(gh).any(1).sum()) == 1


def test_frozen_weight_zero_gradient_and_no_rows():
    c = _case(100, 300, 64, seed=11)
    loss, lse, gh, gw = _run(c)
    gh2, none = pkg.ssm_linear_cross_entropy_backward(c["gl"], c["h"], c["w"], c["t"], lse, need_weight=False)
    assert none is None and torch.equal(gh, gh2)
    gh0, gw0 = pkg.ssm_linear_cross_entropy_backward(c["gl"] * 0, c["h"], c["w"], c["t"], lse)
    assert (gh0 == 0).all() and (gw0 == 0).all()
    gh0, gw0 = pkg.ssm_linear_cross_entropy_backward(c["gl"][:0], c["h"][:0], c["w"], c["t"][:0], lse[:0])
    assert gh0.shape == (0, 64) and (gw0 == 0).all()


def test_same_bits_streams_and_a_graph_beside_eager_calls():
    c = _case(700, 3000, 128, seed=12, ignored=0.3)
    first = _run(c)
    nbytes = [pkg.linear_cross_entropy_workspace_bytes(c["h"], c["w"], backward=b) for b in (False, True)]
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in nbytes]
    loss, lse, gh, gw = (torch.empty_like(v) for v in first)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pkg.ssm_linear_cross_entropy(c["h"], c["w"], c["t"], loss=loss, lse=lse, workspace=ws[0])
        pkg.ssm_linear_cross_entropy_backward(c["gl"], c["h"], c["w"], c["t"], lse, grad_hidden=gh, grad_weight=gw, workspace=ws[1])
    side = torch.cuda.Stream()
    for _ in range(3):
        for v in (loss, lse, gh, gw):
            v.zero_()
        graph.replay()
        with torch.cuda.stream(side):
            other = _run(c)
        eager = _run(c)
        torch.cuda.synchronize()
        for got in ((loss, lse, gh, gw), other, eager):
            assert all(torch.equal(x, y) for x, y in zip(got, first))
    # the kept rows change between replays
    t2 = torch.randint(0, 3000, (700,), device="cuda")
    c["t"].copy_(t2)
    graph.replay()
    want = _run(c)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((loss, lse, gh, gw), want))


def test_counting_pass_of_many_rows():
    """More rows than a block counts by itself."""
    c = _case(20000, 64, 16, seed=13, ignored=0.9, equal=True)
    loss, lse, gh, gw = _run(c)
    _check(c, loss, lse, gh, gw)


def test_waits_that_give_up(monkeypatch):
    """Waits that give up at once: NaN, no hang, and the next call is right."""
    import os
    import subprocess
    import sys
    code = ("import torch, state_space_model_ssm_gb300 as p\n"
            "g = torch.Generator().manual_seed(1)\n"
            "h, w = (torch.randn(n, 64, generator=g).bfloat16().cuda() for n in (600, 700))\n"
            "t = torch.randint(0, 700, (600,), generator=g).cuda()\n"
            "loss, lse = p.ssm_linear_cross_entropy(h, w, t)\n"
            "gh, gw = p.ssm_linear_cross_entropy_backward(torch.ones(600, device='cuda'), h, w, t, torch.zeros(600, device='cuda'))\n"
            "torch.cuda.synchronize()\n"
            "assert torch.isnan(loss).all() and torch.isnan(gh).all() and torch.isnan(gw).all()\n"
            "print('gave up')\n")
    env = dict(os.environ, SSM_SCAN_TEST_FAIL_WAITS="1")
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "gave up" in r.stdout, r.stdout + r.stderr
    c = _case(600, 700, 64, seed=14)
    _check(c, *_run(c))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_of_a_warp_that_part(dtype):
    """Odd rows have logits of -inf in every other run of 32 columns (a product that overflows), even rows have none; some
    rows are NaN.  A warp's rows then take different ways between two loads of its columns."""
    big, factor = (2.0 ** 100, -2.0 ** 60) if dtype == "bf16" else (float("inf"), -2.0)
    c = _case(150, 600, 64, TYPES[dtype], seed=15)
    gone = (torch.arange(600, device="cuda") // 32) % 2 == 1
    part = torch.arange(150, device="cuda") % 2 == 1
    c["h"][:, 0] = 0.0
    c["w"][:, 0] = -2.0 if dtype == "fp16" else 0.0         # (inf times 0 is a NaN: fp16 rows of inf are all -inf)
    c["w"][gone, 0] = factor
    c["t"] %= 32                                            # targets in columns that stay
    clean = dict(c, h=c["h"].clone())
    c["h"][part, 0] = big
    c["h"][40:44] = float("nan")
    loss, lse, gh, gw = _run(c)
    assert torch.isnan(loss[40:44]).all() and torch.isnan(lse[40:44]).all() and torch.isnan(gh[40:44]).all()
    fine = torch.ones(150, dtype=torch.bool, device="cuda")
    fine[40:44] = False
    if dtype == "fp16":                                     # rows without a finite logit: lse -inf, the loss no number
        assert (lse[part & fine] == float("-inf")).all() and torch.isnan(loss[part & fine]).all()
        fine &= ~part
    for rows, cols in ((fine & ~part, slice(None)), (fine & part, ~gone)):
        if not rows.any():
            continue
        h, w = np64(clean["h"][rows]), np64(c["w"][cols])
        h[:, 0] = w[:, 0] = 0.0
        t = c["t"][rows].cpu().numpy()                      # (the first 32 columns are the first of either choice)
        gl = np64(c["gl"][rows])
        b = loss_bounds(h, w, t, -100, TYPES[dtype], gl)
        rl, re = om.linear_cross_entropy(h, w, t, -100)
        close(loss[rows], rl, b["loss"])
        close(lse[rows], re, b["lse"])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,V,D", [(60, 300, 64), (200, 5000, 200), (9000, 64, 16)])
def test_infinite_gradients_stay_in_their_rows(T, V, D, dtype):
    """Rows whose grad_loss is infinite or no number leave the other rows' gradients as they are."""
    c = _case(T, V, D, TYPES[dtype], seed=16)
    c["gl"][5], c["gl"][17], c["gl"][30] = float("inf"), float("nan"), float("-inf")
    fine = torch.isfinite(c["gl"])
    loss, lse, gh, gw = _run(c)
    assert not torch.isfinite(gh[~fine]).any() and not torch.isfinite(gw).any()
    sub = dict(c, h=c["h"][fine], t=c["t"][fine], gl=c["gl"][fine])
    _check(sub, loss[fine], lse[fine], gh[fine])
    c["gl"][fine] = 0.0                                     # nothing finite to be relative to
    _, _, gh, gw = _run(c)
    assert (gh[fine] == 0).all() and not torch.isfinite(gh[~fine]).any()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_infinite_logits(dtype):
    """A logit that overflows makes its row's lse and loss infinite, wherever among the columns it stands; NaN stays NaN."""
    c = _case(70, 900, 64, TYPES[dtype], seed=17)
    big, one = (2.0 ** 100, 2.0 ** 60) if dtype == "bf16" else (float("inf"), 1.0)
    c["h"][:, 0] = 0.0
    c["w"][:, 0] = 0.0 if dtype == "bf16" else -1.0
    up = torch.tensor([0, 40, 41, 300, 899], device="cuda")
    c["t"] = torch.where(torch.isin(c["t"], up), c["t"] + 1, c["t"]) % 899
    c["t"][c["t"] == 41] = 42
    c["t"][c["t"] == 0] = 1
    clean = dict(c, w=c["w"].clone())
    c["w"][up, 0] = one
    c["h"][::3, 0] = big
    c["h"][3, 5] = float("nan")
    loss, lse, gh, gw = _run(c)
    inf = torch.arange(70, device="cuda") % 3 == 0
    inf[3] = False
    assert (lse[inf] == float("inf")).all() and (loss[inf] == float("inf")).all()
    assert torch.isnan(lse[3]) and torch.isnan(loss[3])
    rest = torch.arange(70, device="cuda") % 3 != 0
    _check(dict(clean, h=c["h"][rest], t=c["t"][rest], gl=c["gl"][rest]), loss[rest], lse[rest])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,V,D,ignored", [(100, 9000, 1000, 0.0), (300, 20000, 1024, 0.5), (64, 8000, 4096, 0.2),
                                           (513, 5000, 2048, 0.1), (40, 40000, 300, 0.3), (256, 17000, 200, 0.97)])
def test_terms_shared_by_several_pairs(T, V, D, ignored, dtype):
    """Few tiles of grad hidden: 3 to 16 pairs share each one's terms (fewer where ignored rows leave whole tiles out), at
    widths of real models and with a grad_loss of every size."""
    c = _case(T, V, D, TYPES[dtype], ignored=ignored, seed=18)
    _check(c, *_run(c))
