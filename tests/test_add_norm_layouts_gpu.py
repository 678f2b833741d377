"""Rows of the norm's tensors that lie unlike each other (each at its own offset from a boundary, strides that
change it from row to row), which go element by element, against rows that lie alike (needs a GB300)."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from oracle import layers as ol
from tests.layer_helpers import DTYPES, close, np64
from tests.test_add_norm_gpu import EPS, PAIRS, U, _inputs, _inv_error, _sum

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _inside(t, off, pad, fill):
    """`t` inside a wider tensor, `off` elements from its rows' begin; (the wide tensor, the view)."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    view = wide[:, off:off + t.shape[1]]
    view.copy_(t)
    return wide, view


def _untouched(wide, off, D, fill):
    return (wide[:, :off] == fill).all() and (wide[:, off + D:] == fill).all()


# offsets and widths beyond the row of x, residual, residual_out and the output
PLACES = {"unlike": ((1, 8), (2, 8), (3, 8), (5, 8)), "one_off": ((0, 8), (0, 8), (0, 8), (1, 8)),
          "residual_off": ((0, 8), (1, 8), (0, 8), (0, 8)), "strides": ((0, 8), (0, 9), (0, 10), (0, 11)),
          "alike": ((3, 8), (3, 8), (3, 8), (3, 8)), "alike_strides": ((3, 9), (3, 9), (3, 9), (3, 9))}


@pytest.mark.parametrize("pair", PAIRS, ids=["-".join(p) for p in PAIRS])
@pytest.mark.parametrize("D", [1, 7, 31, 256, 1000, 4096, 6145, 16384])
@pytest.mark.parametrize("where", list(PLACES))
@pytest.mark.parametrize("quant", [None, "int8"])
def test_rows_anywhere(quant, where, D, pair):
    T = 3
    x, r, w = _inputs(T, D, *(DTYPES[k] for k in pair), seed=D + 7)
    h = _sum(x, r)
    place = PLACES[where]
    wx, vx = _inside(x, *place[0], 5.0)
    wr, vr = _inside(r, *place[1], 5.0)
    wh, vh = _inside(torch.zeros_like(r), *place[2], 5.0)
    out = torch.zeros(T, D, dtype=torch.int8 if quant else x.dtype, device="cuda")
    wo, vo = _inside(out, *place[3], 3)
    got = pkg.ssm_add_norm(vx, w, vr, eps=EPS, quant=quant, residual_out=vh, out=vo)
    assert torch.equal(vh, h) and torch.equal(vx, x) and torch.equal(vr, r)
    assert _untouched(wo, place[3][0], D, 3) and _untouched(wh, place[2][0], D, 5)
    assert _untouched(wx, place[0][0], D, 5) and _untouched(wr, place[1][0], D, 5)
    inv, ref = ol.add_norm(np64(h), np64(w), EPS)
    if quant is None:
        close(vo, ref, np.abs(ref) * (_inv_error(D) + 3 * U), x.dtype)
        return
    codes, f = ol.quantize_rows(h.float().cpu().numpy() * w.cpu().numpy()[None, :])
    assert np.array_equal(vo.cpu().numpy(), codes.astype(np.int8))
    close(got[1], inv / f, inv / f * (_inv_error(D) + 2 * U))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [1, 7, 33, 1000, 6145])
@pytest.mark.parametrize("x_at,q_at", [((0, 8), (1, 8)), ((1, 8), (0, 8)), ((3, 9), (2, 11)), ((0, 9), (0, 8))])
def test_quantiser_rows_anywhere(x_at, q_at, D, dtype):
    x, _, _ = _inputs(3, D, DTYPES[dtype], torch.float32, seed=D + 8)
    _, vx = _inside(x, *x_at, 5.0)
    wq, vq = _inside(torch.zeros(3, D, dtype=torch.int8, device="cuda"), *q_at, 3)
    _, s = pkg.ssm_quantize_rows(vx, vq)
    codes, f = ol.quantize_rows(x.float().cpu().numpy())
    assert np.array_equal(vq.cpu().numpy(), codes.astype(np.int8)) and _untouched(wq, q_at[0], D, 3)
    close(s, 1 / f.astype(np.float64), U / f.astype(np.float64))


@pytest.mark.parametrize("pair", PAIRS, ids=["-".join(p) for p in PAIRS])
@pytest.mark.parametrize("D", [1, 31, 1000, 6145])
@pytest.mark.parametrize("where", list(PLACES))
def test_gradient_rows_anywhere(where, D, pair):
    """The gradient of rows that lie anywhere is that of contiguous ones within its bounds."""
    T = 5
    dt, rdt = (DTYPES[k] for k in pair)
    x, r, w = _inputs(T, D, dt, rdt, seed=D + 9)
    h = _sum(x, r)
    g = torch.Generator().manual_seed(D)
    gy, gh = torch.randn(T, D, generator=g).to(dt).cuda(), torch.randn(T, D, generator=g).to(rdt).cuda()
    place = PLACES[where]
    vg, vh, vgh = (_inside(t, *p, 5.0)[1] for t, p in zip((gy, h, gh), place))
    wi, vi = _inside(torch.zeros_like(h), *place[3], 3)
    _, gw = pkg.ssm_add_norm_backward(vg, vh, w, grad_h=vgh, eps=EPS, grad_in=vi)
    assert _untouched(wi, place[3][0], D, 3)
    H, G, W = np64(h), np64(gy), np64(w)
    ref_in, ref_w = ol.add_norm_backward(G, H, W, np64(gh), EPS)
    inv, _ = ol.add_norm(H, W, EPS)
    ei = _inv_error(D)
    n, gn = H * inv[:, None], np.abs(G * W)
    dot = np.mean(np.abs(n) * gn, axis=1, keepdims=True)
    b = inv[:, None] * (gn * (ei + 4 * U) + np.abs(n) * (dot * (2 * ei + 6 * U) + dot * (3 * ei + 6 * U))) + 2 * U * np.abs(ref_in)
    close(vi, ref_in, b, rdt)
    # T rows of at most T blocks, added in fewer than 64 + 12 sums
    close(gw, ref_w, np.sum(np.abs(G * n), axis=0) * (ei + (T + 64 + 12) * U))
