"""A NaN in one gate of the gated linear recurrence stays in its channel and its sequence (needs a GB300)."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from oracle import layers as ol
from tests.layer_helpers import DTYPES, close, gated_bounds, np64
from tests.test_gated_scan_gpu import _backward, _case, _forward, _ref_args

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


# Sequences of whole chunks (every run of tokens is a full one), a cut one, and single tokens and
# fours (the stepping kernels).
LENS = {"whole": ([128, 192], 70), "cut": ([100, 37], 98), "steps": ([1, 4, 8, 3, 2], 10), "cluster": ([1024], 500)}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("which", ["gate_a", "gate_x"])
@pytest.mark.parametrize("channel", [4, 5, 63])
@pytest.mark.parametrize("lens", list(LENS))
def test_nan_gate_stays_in_its_channel(lens, channel, which, dtype):
    lens, at = LENS[lens]
    c = _case(64, lens, resume=[1] * len(lens), dtype=DTYPES[dtype], seed=21)
    clean = dict(c)
    c[which] = c[which].clone()
    c[which][at, channel] = float("nan")
    y, slots, ch = _forward(c, train=True)
    grads = _backward(c, ch)
    # the channel itself: NaN from that token to its sequence's end, and nowhere before or beside
    first = [s for s, n in zip(*c["host"][:2]) if s <= at < s + n][0]
    seq = c["host"][0].index(first)
    end = first + lens[seq]
    bad = torch.isnan(y)
    assert bad[at:end, channel].all() and int(bad.sum()) == end - at
    assert torch.isnan(slots[seq, channel]) and int(torch.isnan(slots).sum()) == 1
    assert torch.isnan(grads[3][channel])
    # every other channel: what it is without the NaN
    args = _ref_args(clean)
    gy, gs = np64(c["grad_y"]), np64(c["grad_state"])
    y_ref, s_ref = ol.gated_scan(*args)
    ref = ol.gated_scan_backward(gy, gs, *args)
    b = gated_bounds(*args, grad_y=gy, grad_state=gs)
    rest = np.arange(64) != channel
    sel = torch.from_numpy(rest).cuda()
    dt = c["x"].dtype
    close(y[:, sel], y_ref[:, rest], b["y"][:, rest], dt)
    close(slots[:, sel], s_ref[:, rest], b["slots"][:, rest])
    for got, want, name in zip(grads[:3], ref[:3], ("grad_x", "grad_gate_a", "grad_gate_x")):
        close(got[:, sel], want[:, rest], b[name][:, rest], dt)
    close(grads[3][sel], ref[3][rest], b["grad_lam"][rest])
    close(grads[4][:, sel], ref[4][:, rest], b["grad_slots"][:, rest])
