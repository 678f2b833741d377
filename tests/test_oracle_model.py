"""Checks of the float64 oracle of the selective-scan model's operators: closed forms, and gradients
against differences along random directions (central differences of a float64 function: the step's
h^2 error and 1e-16 / h cancellation are both below 1e-8 of values of order one at h = 1e-5)."""
import numpy as np
import pytest

from oracle import model as om

STARTS, LENS, RESUME = [0, 5, 5, 8], [5, 0, 3, 4], [0, 1, 1, 0]


def _scan_case(seed=0, C=4, N=3, groups=2, gate=True):
    r = np.random.default_rng(seed)
    T = 12
    c = dict(slots=r.normal(size=(4, C, N)), x=r.normal(size=(T, C)), dt=r.normal(size=(T, C)) * 0.5,
             A=-np.exp(r.normal(size=(C, N)) * 0.3), B=r.normal(size=(T, groups * N)), C=r.normal(size=(T, groups * N)),
             D=r.normal(size=C), z=r.normal(size=(T, C)) if gate else None, dt_bias=r.normal(size=C))
    return c, r


def _scan(c, groups, softplus):
    return om.selective_scan(c["slots"], c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], STARTS, LENS, RESUME, c["z"],
                             c["dt_bias"], softplus, groups)


def test_scan_of_one_state_is_a_geometric_sum():
    T, a, step = 6, -0.3, 0.7
    one = np.ones((T, 1))
    y, slots, _ = om.selective_scan(np.full((1, 1, 1), 2.0), one, one * step, np.array([[a]]), one, one, None, [0], [T], [1])
    h = 2.0
    for t in range(T):
        h = np.exp(a * step) * h + step
        assert abs(y[t, 0] - h) < 1e-14
    assert abs(slots[0, 0, 0] - h) < 1e-14


def test_softplus_threshold_and_ends():
    v, step, slope = om.step_of(np.array([[-800.0, -30.0, 0.0, 20.0, 20.5, 900.0]]), None, True)
    assert np.allclose(step[0], [0.0, np.exp(-30.0), np.log(2.0), 20.0 + np.log1p(np.exp(-20.0)), 20.5, 900.0], rtol=1e-12)
    assert np.allclose(slope[0], [0.0, np.exp(-30.0), 0.5, 1 / (1 + np.exp(-20.0)), 1.0, 1.0], rtol=1e-12)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("gate", [True, False])
def test_scan_gradients_against_differences(gate, softplus):
    c, r = _scan_case(3, gate=gate)
    gy, gs = r.normal(size=c["x"].shape), r.normal(size=c["slots"].shape)

    def value(cc):
        y, slots, _ = _scan(cc, 2, softplus)
        return (y * gy).sum() + (slots * gs).sum()

    g = om.selective_scan_backward(gy, gs, c["slots"], c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], STARTS, LENS, RESUME,
                                   c["z"], c["dt_bias"], softplus, 2)
    for name in ("x", "dt", "A", "B", "C", "D", "dt_bias", "slots") + (("z",) if gate else ()):
        d = r.normal(size=c[name].shape)
        up, down = (value({**c, name: c[name] + s * 1e-5 * d}) for s in (1, -1))
        slope = (g["initial_state" if name == "slots" else name] * d).sum()
        assert abs((up - down) / 2e-5 - slope) < 1e-6 * (1 + abs(slope)), name


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("K", [1, 2, 4, 7])
def test_conv_against_differences_and_numpy(K, silu):
    r = np.random.default_rng(K)
    c = dict(x=r.normal(size=(12, 3)), weight=r.normal(size=(3, K)), slots=r.normal(size=(4, 3, K - 1)), bias=r.normal(size=3))
    go, gs = r.normal(size=c["x"].shape), r.normal(size=c["slots"].shape)

    def value(cc):
        out, after, _ = om.causal_conv(cc["x"], cc["weight"], cc["slots"], STARTS, LENS, RESUME, cc["bias"], silu)
        return (out * go).sum() + (after * gs).sum()

    _, _, v = om.causal_conv(c["x"], c["weight"], c["slots"], STARTS, LENS, RESUME, c["bias"], silu)
    ref = np.convolve(c["x"][0:5, 1], c["weight"][1, ::-1])[:5] + c["bias"][1]      # the first sequence is fresh
    assert np.allclose(v[0:5, 1], ref, atol=1e-13)
    g = om.causal_conv_backward(go, gs, c["x"], c["weight"], c["slots"], STARTS, LENS, RESUME, c["bias"], silu)
    for name in ("x", "weight", "bias") + (("slots",) if K > 1 else ()):
        d = r.normal(size=c[name].shape)
        up, down = (value({**c, name: c[name] + s * 1e-5 * d}) for s in (1, -1))
        slope = (g["initial_state" if name == "slots" else name] * d).sum()
        assert abs((up - down) / 2e-5 - slope) < 1e-6 * (1 + abs(slope)), name


def test_loss_of_equal_logits_and_gradients_against_differences():
    r = np.random.default_rng(5)
    h, w, t = r.normal(size=(6, 4)), r.normal(size=(9, 4)), np.array([0, 8, -100, 3, 3, -100])
    loss, lse = om.linear_cross_entropy(h * 0, w, t)
    assert np.allclose(loss, np.where(t == -100, 0.0, np.log(9.0))) and np.allclose(lse, loss)
    assert np.isnan(om.linear_cross_entropy(h, w, np.array([9, 0, 0, 0, 0, -1]))[0][[0, 5]]).all()
    gl = r.normal(size=6)
    gh, gw, G = om.linear_cross_entropy_backward(gl, h, w, t)
    assert (gh[[2, 5]] == 0).all() and np.allclose(G.sum(1), 0, atol=1e-14)
    for name, a, g in (("h", h, gh), ("w", w, gw)):
        d = r.normal(size=a.shape)
        up, down = ((om.linear_cross_entropy(h + s * 1e-5 * d if name == "h" else h, w + s * 1e-5 * d if name == "w" else w, t)[0]
                     * gl).sum() for s in (1, -1))
        assert abs((up - down) / 2e-5 - (g * d).sum()) < 1e-6 * (1 + abs((g * d).sum()))
