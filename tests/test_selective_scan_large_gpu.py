"""Parity of the selective scan at sizes that fill the device with wide tiles: prompts that are cut into segments, prompts
and decode steps that are not, for every number of states the walks tell apart (needs a GB300).

The float64 oracle walks some of the channels: none reads another's values.  Sums over channels (grad_B, grad_C) are
compared whole, with few tokens.  Wide tiles are taken from 912 units times tiles of channels on (7296 where sequences have at
most 8 tokens); a tile has 64 channels up to 16 states, then 32, 16 and 8."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from tests import test_selective_scan_gpu as base
from tests.model_helpers import DTYPES

pytestmark = pytest.mark.gpu
CHANNELS = {8: 4096, 13: 4095, 16: 4096, 32: 2048, 64: 1024, 100: 1022, 128: 512}     # 64 tiles (128 with 100 states)
SUMMED = ("grad_B", "grad_C")


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _some(first, last):
    """Channels of [first, last): the ends, both sides of tiles' and blocks' edges, and one in between."""
    n = last - first
    picks = {0, 1, 7, 8, 31, 32, 63, 64, 127, 128, 255, 256, n // 2 + 3, n - 2, n - 1}
    return torch.tensor(sorted(first + p for p in picks if 0 <= p < n))


def _check(c, y, slots, grads=None, group=0):
    """Of the channels of one group."""
    C, N = c["A"].shape
    each = C // c["groups"]
    at = _some(group * each, (group + 1) * each).cuda()
    rows = slice(group * N, (group + 1) * N)
    s = dict(c, groups=1, B=c["B"][:, rows], C=c["C"][:, rows], slots=c["slots"][:, at], A=c["A"][at],
             grad_state=c["grad_state"][:, at])
    for name in ("x", "dt", "z", "grad_y"):
        s[name] = None if c[name] is None else c[name][:, at]
    for name in ("D", "dt_bias"):
        s[name] = None if c[name] is None else c[name][at]
    if grads is not None:
        grads = {k: v[at] if k in ("grad_A", "grad_D", "grad_dt_bias") else v[:, at] for k, v in grads.items() if k not in SUMMED}
    base._check(s, y[:, at], slots[:, at], grads)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("N", list(CHANNELS))
def test_a_prompt_in_segments(N, dtype):
    """Segments of 64 tokens (80 with 100 states, whose blocks are twice as many), and a sequence that is left whole."""
    C = CHANNELS[N]
    assert pkg.selective_scan_workspace_bytes(2, 1024, C, N) > (2 + 1024 // (80 if N == 100 else 64)) * C * N * 4
    c = base._case(C, N, [1000, 24], resume=[1, 0], dtype=DTYPES[dtype], seed=20 + N)
    y, slots, ch = base._forward(c, train=True)
    _check(c, y, slots, base._backward(c, ch))


@pytest.mark.parametrize("N", [16, 32])
def test_segments_of_another_length(N):
    """One sequence, in segments that are just short enough for one round of blocks (96 tokens)."""
    c = base._case(CHANNELS[N], N, [2500], resume=[1], dtype=torch.bfloat16, seed=21)
    y, slots, ch = base._forward(c, train=True)
    _check(c, y, slots, base._backward(c, ch))


def test_groups():
    c = base._case(4096, 16, [1000, 24], resume=[0, 1], dtype=torch.bfloat16, seed=22, groups=2)
    y, slots, ch = base._forward(c, train=True)
    grads = base._backward(c, ch)
    for group in (0, 1):
        _check(c, y, slots, grads, group)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [8, 16, 32, 64, 128])
def test_many_prompts_none_of_them_cut(N, dtype):
    c = base._case(CHANNELS[N] // 2, N, [60, 17, 33, 41] * 10, dtype=DTYPES[dtype], seed=23)
    y, slots, ch = base._forward(c, train=True)
    _check(c, y, slots, base._backward(c, ch))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens", [[1] * 256, [3, 1, 0, 2] * 64])
@pytest.mark.parametrize("N", [8, 16, 32, 64, 128])
def test_decode_steps(N, lens, dtype):
    c = base._case(CHANNELS[N] // 2, N, lens, resume=[1] * 256, dtype=DTYPES[dtype], seed=24)
    y, slots, _ = base._forward(c)
    _check(c, y, slots)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("C,N,lens", [(300, 16, [40, 9]), (261, 13, [40, 9]), (150, 32, [40, 9]), (75, 64, [40, 9]), (37, 128, [40, 9]),
                                      (40, 100, [40, 9]), (150, 32, [300]), (512, 128, [20])])
def test_sums_over_blocks_of_channels(C, N, lens, dtype):
    """Three blocks of channels and more, whose shares of grad_B and grad_C another kernel adds."""
    c = base._case(C, N, lens, dtype=DTYPES[dtype], seed=25)
    y, slots, ch = base._forward(c, train=True)
    base._check(c, y, slots, base._backward(c, ch), blocks=32)


@pytest.mark.parametrize("N", [13, 16])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["x", "grad_y"])
def test_what_is_no_number_stays_where_it_belongs(which, value, N):
    """One value of a sequence that resumes and is cut.  x reaches later states and the steps' gradients, grad_y the
    gradients of earlier inputs and of the slot; nothing else."""
    c = base._case(70, N, [100, 300], resume=[1, 1], seed=26)
    c[which][120, 5] = value
    y, slots, ch = base._forward(c, train=True)
    g = base._backward(c, ch)

    def exactly(t, where):
        want = torch.zeros(t.shape, dtype=torch.bool, device="cuda")
        want[where] = True
        assert torch.equal(~torch.isfinite(t), want)

    none = (slice(0, 0),)
    exactly(y, (slice(120, 400), 5) if which == "x" else none)
    exactly(slots, (1, 5) if which == "x" else none)
    exactly(g["grad_slots"], (1, 5) if which == "grad_y" else none)
    exactly(g["grad_x"], (slice(100, 121), 5) if which == "grad_y" else none)
    exactly(g["grad_dt"], (slice(120, 400), 5) if which == "x" else (slice(100, 121), 5))
    exactly(g["grad_z"], (slice(120, 400), 5) if which == "x" else (120, 5))
    exactly(g["grad_A"], 5)
    if value == float("inf"):
        assert torch.isinf(slots[1, 5] if which == "x" else g["grad_slots"][1, 5]).all()
