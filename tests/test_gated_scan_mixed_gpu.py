"""Decoding sequences beside long ones in one call of the gated linear recurrence: short sequences are
stepped, longer ones walked, by their own lengths (needs a GB300)."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from tests.layer_helpers import DTYPES
from tests.test_gated_scan_gpu import C0, _backward, _case, _check_backward, _check_forward, _forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _run(c):
    y, slots, ch = _forward(c, train=True)
    _check_forward(c, y, slots)
    grads = _backward(c, ch)
    _check_backward(c, grads)
    return y, slots, grads


def _short(lens):
    assert sum(lens) <= 16 * len(lens) and sum(lens) != len(lens)
    return lens


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("C", [1, 33, 64, 130])
def test_lengths_on_both_sides_of_the_limit(C, dtype):
    lens = _short([1] * 30 + [31, 32, 33, 34, 63, 0, 64, 65, 1, 66, 127, 128, 129, 500] + [1, 2, 3] * 40)
    _run(_case(C, lens, dtype=DTYPES[dtype], seed=C, fused=C == 64))


@pytest.mark.parametrize("where", ["first", "last"])
def test_one_prompt_beside_decodes(where):
    lens = [1] * 255
    lens = _short([3800] + lens if where == "first" else lens + [3800])
    _run(_case(64, lens, resume=[1] * 256, dtype=torch.bfloat16, seed=31))


def test_blocks_take_several_long_sequences():
    """40 of them on 20 blocks of channels: more than blocks that are resident at once; rows that TMA
    can describe and rows that it cannot."""
    rng = np.random.default_rng(5)
    lens = [1] * 400
    for k in range(40):
        lens.insert(int(rng.integers(len(lens))), int(rng.integers(65, 140)))
    lens = _short(lens)
    _run(_case(1280, lens, dtype=torch.bfloat16, seed=32))
    _run(_case(1279, lens, dtype=torch.float32, seed=33))


def test_thousands_of_sequences():
    """Long ones at the borders of what a block reads of the table at a time."""
    lens = [1] * 4200
    for k, n in ((0, 70), (31, 65), (32, 200), (1023, 90), (1024, 91), (2047, 92), (2048, 93), (3500, 64), (4199, 300)):
        lens[k] = n
    _run(_case(64, _short(lens), seed=34))


def test_only_short_ones_and_only_empty_ones_beside_one():
    _run(_case(96, _short([3] * 50 + [0] * 20), seed=35))
    _run(_case(96, _short([0] * 60 + [700] + [0] * 10), resume=[1] * 71, seed=36))
    # as many tokens as sequences counts as a decode step: every length is right all the same
    lens = [0] * 199 + [200]
    _run(_case(96, lens, resume=[1] * 200, seed=37))


def test_invalid_range_beside_a_long_one():
    c = _case(64, _short([1] * 20 + [200, 100] + [1] * 30), resume=[1] * 52, seed=38)
    c["starts"][21] = 340                                  # 340 + 100 is past the end: counts as empty
    y, slots, _ = _forward(c)
    assert torch.isnan(y[220:320]).all() and torch.equal(slots[21], c["slots"][21])
    assert not torch.isnan(y[:220]).any() and not torch.isnan(y[320:]).any()


def test_same_bits_and_graph():
    c = _case(192, _short([1] * 50 + [300, 5, 70] + [1] * 10), resume=[1] * 63, dtype=torch.bfloat16, seed=39)
    y, slots, grads = _run(c)
    again = _run(c)
    assert torch.equal(y, again[0]) and torch.equal(slots, again[1])
    assert all(torch.equal(a, b) for a, b in zip(grads, again[2]))
    s = c["slots"].clone()
    ch = pkg.gated_scan_chunk_states(len(s), *c["x"].shape)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pkg.ssm_gated_scan(s, c["x"], c["gate_a"], c["gate_x"], c["lam"], c["starts"], c["lens"], c["resume"],
                                 decay_scale=C0, chunk_states=ch)
        gr = _backward(c, ch)
    for _ in range(2):
        s.copy_(c["slots"])
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, y) and torch.equal(s, slots) and all(torch.equal(a, b) for a, b in zip(gr, grads))


def test_a_prompt_beside_decodes_is_not_stepped():
    """The call's time is of the order of the prompt's alone (it was 65 and 54 times that where one
    thread a channel pair stepped the prompt; the limit of 10 leaves room for a noisy machine)."""
    def best(lens):
        T, n, C = sum(lens), len(lens), 2048
        x, ga, gx, gy = (torch.randn(T, C, device="cuda").bfloat16() for _ in range(4))
        lam, slots = torch.zeros(C, device="cuda"), torch.zeros(n, C, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        meta = (torch.tensor(np.cumsum([0] + lens[:-1]), **i32), torch.tensor(lens, **i32), torch.ones(n, **i32))
        ch = pkg.gated_scan_chunk_states(n, T, C)
        out = [1e9, 1e9]
        for _ in range(8):
            ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
            ev[0].record()
            pkg.ssm_gated_scan(slots, x, ga, gx, lam, *meta, chunk_states=ch)
            ev[1].record()
            pkg.ssm_gated_scan_backward(gy, x, ga, gx, lam, ch, *meta)
            ev[2].record()
            torch.cuda.synchronize()
            out = [min(out[k], ev[k].elapsed_time(ev[k + 1])) for k in range(2)]
        return out
    alone, mixed = best([3800]), best(_short([1] * 255 + [3800]))
    assert mixed[0] < 10 * alone[0] and mixed[1] < 10 * alone[1], (alone, mixed)
