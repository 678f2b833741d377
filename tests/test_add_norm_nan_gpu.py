"""What is no number in the norm's 8-bit output: a row with a NaN or an infinity in h or in h * weight
has scale NaN, and the other rows are as they are without it (needs a GB300)."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from oracle import layers as ol
from tests.layer_helpers import DTYPES, close, np64
from tests.test_add_norm_gpu import EPS, PAIRS, U, _inputs, _inv_error, _sum

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
# width, place of the value: one and several warps a row, whole and cut slots, one and more slots a thread
PLACES = [(40, 0), (40, 39), (256, 5), (1000, 999), (4096, 2049), (4100, 4099), (16384, 12345)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _rows_are(rows, q, s, h, w):
    inv, _ = ol.add_norm(np64(h)[rows], np64(w), EPS)
    codes, f = ol.quantize_rows(h.float().cpu().numpy()[rows] * w.cpu().numpy()[None, :])
    assert np.array_equal(q.cpu().numpy()[rows], codes.astype(np.int8))
    close(s[rows], inv / f, inv / f * (_inv_error(h.shape[1]) + 2 * U))


@pytest.mark.parametrize("pair", PAIRS, ids=["-".join(p) for p in PAIRS])
@pytest.mark.parametrize("D,at", PLACES)
def test_nan_weight(D, at, pair):
    x, r, w = _inputs(5, D, *(DTYPES[k] for k in pair), seed=D)
    w[at] = NAN
    _, s, h = pkg.ssm_add_norm(x, w, r, eps=EPS, quant="int8")
    assert torch.equal(h, _sum(x, r)) and torch.isnan(s).all()
    y, _ = pkg.ssm_add_norm(x, w, r, eps=EPS)
    assert torch.isnan(y[:, at]).all() and int(torch.isnan(y).sum()) == 5


@pytest.mark.parametrize("pair", PAIRS, ids=["-".join(p) for p in PAIRS])
@pytest.mark.parametrize("D,at", PLACES)
def test_infinite_weight(D, at, pair):
    """Infinity times a number, and times zero."""
    x, r, w = _inputs(5, D, *(DTYPES[k] for k in pair), seed=D + 1)
    x[::2, at], r[::2, at] = 0, 0
    w[at] = INF
    _, s, _ = pkg.ssm_add_norm(x, w, r, eps=EPS, quant="int8")
    assert torch.isnan(s).all()


@pytest.mark.parametrize("pair", PAIRS, ids=["-".join(p) for p in PAIRS])
@pytest.mark.parametrize("D,at", PLACES)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("weight", [0.0, 1.5])
def test_value_that_is_no_number(D, at, value, weight, pair):
    x, r, w = _inputs(6, D, *(DTYPES[k] for k in pair), seed=D + 2)
    w[at] = weight
    x[1, at] = value
    r[4, at] = value
    q, s, h = pkg.ssm_add_norm(x, w, r, eps=EPS, quant="int8")
    assert torch.isnan(s[[1, 4]]).all()
    _rows_are([0, 2, 3, 5], q, s, h, w)


@pytest.mark.parametrize("D,at", PLACES)
@pytest.mark.parametrize("off", [1, 3])
def test_rows_off_the_boundary(D, at, off):
    x, r, w = _inputs(4, D, torch.bfloat16, torch.bfloat16, seed=D + 3)
    wide = torch.zeros(4, D + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, off:off + D] = x
    w[at] = NAN
    for res in (r, wide[:, off:off + D].clone()):           # rows that lie unlike x's; see below for alike
        _, s, _ = pkg.ssm_add_norm(wide[:, off:off + D], w, res, eps=EPS, quant="int8")
        assert torch.isnan(s).all()
    alike = torch.zeros_like(wide)
    alike[:, off:off + D] = r
    _, s, _ = pkg.ssm_add_norm(wide[:, off:off + D], w, alike[:, off:off + D], eps=EPS, quant="int8",
                               residual_out=alike[:, off:off + D])
    assert torch.isnan(s).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D,at", PLACES)
def test_quantiser(D, at, dtype):
    x, _, _ = _inputs(6, D, DTYPES[dtype], torch.float32, seed=D + 4)
    x[1, at], x[4, at] = NAN, -INF
    q, s = pkg.ssm_quantize_rows(x)
    assert torch.isnan(s[[1, 4]]).all()
    rows = [0, 2, 3, 5]
    codes, f = ol.quantize_rows(x.float().cpu().numpy()[rows])
    assert np.array_equal(q.cpu().numpy()[rows], codes.astype(np.int8))
    close(s[rows], 1 / f.astype(np.float64), U / f.astype(np.float64))
