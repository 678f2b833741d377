"""Parity of the RMS norm with the residual's addition, its 8-bit output and gradient, and the row
quantiser, with the float64 oracle (needs a GB300)."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from oracle import layers as ol
from tests.layer_helpers import DTYPES, U, close, np64

pytestmark = pytest.mark.gpu
EPS = 1e-5
PAIRS = [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")]
SHAPES = [(1, 1), (1, 8), (3, 31), (5, 256), (2, 1000), (7, 2048), (4, 4096), (2, 4100), (1, 6145), (3, 16384)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _inputs(T, D, dt, rdt, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g).to(dt).cuda()
    r = (torch.randn(T, D, generator=g) * 2).to(rdt).cuda()
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    return x, r, w


def _sum(x, r):
    return (x.float() + r.float()).to(r.dtype)           # the definition of h: a fp32 sum rounded to the residual's type


def _inv_error(D):
    """inv = 1 / sqrt(sum / D + eps): a thread sums at most 64 squares, then 5 + 5 levels; all terms
    positive, so the sum is within (64 + 10 + 1) u, the quotient and eps add 2, the root halves and
    adds, with the quotient, 2 more."""
    return (min(D, 64) + 13) / 2 * U + 2 * U


@pytest.mark.parametrize("pair", PAIRS, ids=["-".join(p) for p in PAIRS])
@pytest.mark.parametrize("T,D", SHAPES)
def test_norm(T, D, pair):
    dt, rdt = (DTYPES[k] for k in pair)
    x, r, w = _inputs(T, D, dt, rdt, seed=D)
    y, h = pkg.ssm_add_norm(x, w, r, eps=EPS)
    assert y.dtype == dt and torch.equal(h, _sum(x, r))
    inv, ref = ol.add_norm(np64(h), np64(w), EPS)
    close(y, ref, np.abs(ref) * (_inv_error(D) + 3 * U), dt)


@pytest.mark.parametrize("pair", PAIRS, ids=["-".join(p) for p in PAIRS])
@pytest.mark.parametrize("T,D", SHAPES)
def test_norm_int8(T, D, pair):
    dt, rdt = (DTYPES[k] for k in pair)
    x, r, w = _inputs(T, D, dt, rdt, seed=D + 1)
    q, s, h = pkg.ssm_add_norm(x, w, r, eps=EPS, quant="int8")
    assert torch.equal(h, _sum(x, r))
    inv, _ = ol.add_norm(np64(h), np64(w), EPS)
    codes, f = ol.quantize_rows(h.float().cpu().numpy() * w.cpu().numpy()[None, :])
    assert np.array_equal(q.cpu().numpy(), codes.astype(np.int8))
    close(s, inv / f, inv / f * (_inv_error(D) + 2 * U))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,D", SHAPES + [(333, 72)])
def test_quantize_rows(T, D, dtype):
    x, _, _ = _inputs(T, D, DTYPES[dtype], torch.float32, seed=D + 2)
    q, s = pkg.ssm_quantize_rows(x)
    codes, f = ol.quantize_rows(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), codes.astype(np.int8))
    close(s, 1 / f.astype(np.float64), U / f.astype(np.float64))


def test_no_residual_and_in_place():
    x, r, w = _inputs(6, 512, torch.bfloat16, torch.bfloat16)
    y, h = pkg.ssm_add_norm(x, w, eps=EPS)
    assert h is x
    close(y, ol.add_norm(np64(x), np64(w), EPS)[1], np.abs(np64(y)) * (_inv_error(512) + 4 * U), torch.bfloat16)
    want = _sum(x, r)
    y0, _ = pkg.ssm_add_norm(x, w, r, eps=EPS)
    y1, h1 = pkg.ssm_add_norm(x, w, r, eps=EPS, residual_out=r)
    assert h1 is r and torch.equal(r, want) and torch.equal(y0, y1)


@pytest.mark.parametrize("quant", [None, "int8"])
@pytest.mark.parametrize("off", [0, 1, 4])
def test_strided_rows(quant, off):
    """Rows inside wider tensors, at aligned and odd offsets; nothing beside them is written."""
    T, D = 9, 256
    x, r, w = _inputs(T, D, torch.bfloat16, torch.bfloat16, seed=4)
    wx, wr, wh = (torch.full((T, D + 16), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    wx[:, off:off + D], wr[:, off:off + D] = x, r
    kw = dict(eps=EPS, quant=quant)
    a = pkg.ssm_add_norm(x, w, r, **kw)
    wide = torch.full((T, D + 16), 3, dtype=a[0].dtype, device="cuda")
    b = pkg.ssm_add_norm(wx[:, off:off + D], w, wr[:, off:off + D], residual_out=wh[:, off:off + D],
                         out=wide[:, off:off + D], **kw)
    for p, q in zip(a, b):
        # another split of the row over threads sums in another order: the norm may differ in the last bits
        if p.dtype in (torch.float32, torch.bfloat16):
            close(q, np64(p), np.abs(np64(p)) * 2 * _inv_error(D), p.dtype)
        else:
            assert torch.equal(p, q)
    assert (wide[:, :off] == 3).all() and (wide[:, off + D:] == 3).all()
    assert (wh[:, :off] == 5).all() and (wh[:, off + D:] == 5).all()


def test_rows_without_anything_and_with_too_much():
    """Zeros, denormals, infinities and NaN: codes and scales by rule, other rows untouched."""
    x = torch.randn(8, 64, generator=torch.Generator().manual_seed(5))
    x[1] = 0
    x[2] = 0
    x[2, 3] = 1e-40
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    x[5] = 1e-38
    x = x.cuda()
    q, s = pkg.ssm_quantize_rows(x)
    codes, f = ol.quantize_rows(x.cpu().numpy())
    fine = [0, 1, 2, 5, 6, 7]
    assert np.array_equal(q.cpu().numpy()[fine], codes[fine].astype(np.int8))
    assert torch.isnan(s[3]) and torch.isnan(s[4]) and torch.isfinite(s[fine]).all()
    w = torch.ones(64, device="cuda")
    q, s, _ = pkg.ssm_add_norm(x, w, torch.zeros_like(x), eps=EPS, quant="int8")
    assert torch.isnan(s[3]) and torch.isnan(s[4]) and torch.isfinite(s[fine]).all()
    y, _ = pkg.ssm_add_norm(x, w, torch.zeros_like(x), eps=EPS)
    assert (y[1] == 0).all() and torch.isnan(y[4]).all() and torch.isfinite(y[fine]).all()


@pytest.mark.parametrize("pair", PAIRS, ids=["-".join(p) for p in PAIRS])
@pytest.mark.parametrize("T,D", [(1, 1), (3, 31), (2, 1000), (700, 256), (5, 4096), (2, 6145), (3, 16384), (1300, 40)])
@pytest.mark.parametrize("with_h", [True, False])
def test_backward(T, D, pair, with_h):
    dt, rdt = (DTYPES[k] for k in pair)
    x, r, w = _inputs(T, D, dt, rdt, seed=D + 3)
    h = _sum(x, r)
    g = torch.Generator().manual_seed(D + 4)
    gy = torch.randn(T, D, generator=g).to(dt).cuda()
    gh = torch.randn(T, D, generator=g).to(rdt).cuda() if with_h else None
    gin, gw = pkg.ssm_add_norm_backward(gy, h, w, grad_h=gh, eps=EPS)
    H, G, W = np64(h), np64(gy), np64(w)
    ref_in, ref_w = ol.add_norm_backward(G, H, W, None if gh is None else np64(gh), EPS)
    inv, _ = ol.add_norm(H, W, EPS)
    ei = _inv_error(D)
    n, gn = H * inv[:, None], np.abs(G * W)
    dot = np.mean(np.abs(n) * gn, axis=1, keepdims=True)             # its sum: the roundings of the squares' and two a product
    e_dot = dot * (2 * ei + ei + 6 * U)
    b = inv[:, None] * (gn * (ei + 4 * U) + np.abs(n) * (dot * (2 * ei + 6 * U) + e_dot)) + 2 * U * np.abs(ref_in)
    close(gin, ref_in, b, rdt)
    # grad_w: a block adds its rows one after another (T / 148 at most), then at most 64 sums and 8
    terms = np.sum(np.abs(G * n), axis=0)
    close(gw, ref_w, terms * (ei + (T / 148 + 64 + 12) * U))


def test_backward_strided_in_place_and_fixed_order():
    T, D = 40, 512
    x, r, w = _inputs(T, D, torch.bfloat16, torch.bfloat16, seed=6)
    h = _sum(x, r)
    gy, gh = torch.randn(T, D, device="cuda").bfloat16(), torch.randn(T, D, device="cuda").bfloat16()
    a = pkg.ssm_add_norm_backward(gy, h, w, grad_h=gh, eps=EPS)
    wide = torch.zeros(T, D + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, :D] = gh
    b = pkg.ssm_add_norm_backward(gy, h, w, grad_h=wide[:, :D], grad_in=wide[:, :D], eps=EPS)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and (wide[:, D:] == 0).all()


def test_empty_rows():
    w = torch.ones(16, device="cuda")
    e = torch.empty(0, 16, device="cuda")
    assert pkg.ssm_add_norm(e, w, e)[0].shape == (0, 16)
    assert pkg.ssm_quantize_rows(e)[0].shape == (0, 16)
    gw = pkg.ssm_add_norm_backward(e, e, w)[1]
    assert (gw == 0).all()
