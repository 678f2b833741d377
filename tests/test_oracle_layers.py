"""Pins of the float64 oracle of the layer operators: closed forms and central differences (CPU)."""
import numpy as np
import pytest

from oracle import layers as ol


def _gated(C=5, lens=(4, 1, 6), seed=0):
    g = np.random.default_rng(seed)
    T = sum(lens)
    x, ga, gx = (g.standard_normal((T, C)) for _ in range(3))
    lam, slots = g.standard_normal(C), g.standard_normal((len(lens), C))
    starts = np.cumsum([0] + list(lens[:-1]))
    return x, ga, gx, lam, slots, starts, list(lens), [1, 0, 1]


def test_gated_scan_one_token_closed_form():
    x, ga, gx, lam, slots, *_ = _gated(lens=(1,))
    y, s = ol.gated_scan(slots, x, ga, gx, lam, [0], [1], [1], 8.0)
    a = np.exp(-8.0 * np.log1p(np.exp(lam)) / (1 + np.exp(-ga[0])))
    assert np.allclose(y[0], a * slots[0] + np.sqrt(1 - a * a) * x[0] / (1 + np.exp(-gx[0])), rtol=1e-12, atol=0)
    assert np.array_equal(y[0], s[0])


def test_gated_scan_split_resume_and_open_gate():
    x, ga, gx, lam, slots, *_ = _gated(lens=(9,))
    y, s = ol.gated_scan(slots, x, ga, gx, lam, [0], [9], [1], 8.0)
    y1, s1 = ol.gated_scan(slots, x[:4], ga[:4], gx[:4], lam, [0], [4], [1], 8.0)
    y2, s2 = ol.gated_scan(s1, x[4:], ga[4:], gx[4:], lam, [0], [5], [1], 8.0)
    assert np.array_equal(np.concatenate([y1, y2]), y) and np.array_equal(s2, s)
    # a recurrence gate that is shut (r = 0) keeps the state whatever x is
    y, s = ol.gated_scan(slots, x, np.full_like(ga, -np.inf), gx, lam, [0], [9], [1], 8.0)
    assert np.array_equal(s, slots)


@pytest.mark.parametrize("which", range(5))
def test_gated_scan_backward_against_differences(which):
    x, ga, gx, lam, slots, starts, lens, resume = _gated()
    g = np.random.default_rng(1)
    gy, gs = g.standard_normal(x.shape), g.standard_normal(slots.shape)
    args = [x, ga, gx, lam, slots]

    def loss(v):
        y, s = ol.gated_scan(v[4], v[0], v[1], v[2], v[3], starts, lens, resume, 3.0)
        return np.sum(y * gy) + np.sum(s * gs)

    got = ol.gated_scan_backward(gy, gs, slots, x, ga, gx, lam, starts, lens, resume, 3.0)[which]
    for at in np.ndindex(args[which].shape):
        d = 1e-5
        hi, lo = [v.copy() for v in args], [v.copy() for v in args]
        hi[which][at] += d
        lo[which][at] -= d
        # central difference: d^2 f'''/6 plus 1e-16 |f| / d, both below 1e-8 here
        assert abs((loss(hi) - loss(lo)) / (2 * d) - got[at]) <= 1e-7 * (1 + abs(got[at]))


def test_add_norm_backward_against_differences():
    g = np.random.default_rng(2)
    h, gy, gh, w = g.standard_normal((3, 7)), g.standard_normal((3, 7)), g.standard_normal((3, 7)), g.standard_normal(7)

    def loss(h, w):
        return np.sum(ol.add_norm(h, w, 1e-3)[1] * gy) + np.sum(h * gh)

    gin, gw = ol.add_norm_backward(gy, h, w, gh, 1e-3)
    d = 1e-5
    for at in np.ndindex(h.shape):
        e = np.zeros_like(h)
        e[at] = d
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * d) - gin[at]) <= 1e-7 * (1 + abs(gin[at]))
    for k in range(7):
        e = np.zeros_like(w)
        e[k] = d
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * d) - gw[k]) <= 1e-7 * (1 + abs(gw[k]))


def test_quantize_rows_values_and_edges():
    v = np.array([[1.0, -2.0, 0.5, 0.0], [0.0, 0.0, 0.0, 0.0], [1e-40, -1e-40, 0.0, 0.0], [254.0, 1.0, 3.0, -127.0]],
                 dtype=np.float32)
    q, f = ol.quantize_rows(v)
    assert np.array_equal(q[0], [64.0, -127.0, 32.0, 0.0])         # 63.5 and 31.75: half to even, nearest
    assert np.array_equal(q[1], [0, 0, 0, 0]) and f[1] == ol.FLT_MAX
    assert f[2] == ol.FLT_MAX and np.all(np.abs(q[2]) <= 127)
    assert np.array_equal(q[3], [127.0, 0.0, 2.0, -64.0])          # 0.5 -> 0, 1.5 -> 2, -63.5 -> -64


def test_int8_matmul_extremes():
    x = np.full((1, 1000), -128, dtype=np.int8)
    assert ol.int8_matmul(x, [1.0], x, [0.5], [1.0])[0, 0] == 16384.0 * 1000 * 0.5 + 1.0
