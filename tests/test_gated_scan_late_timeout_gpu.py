"""One warp of one block of a gated scan's cluster gives up its wait after the first round, while the
others go on (needs a GB300).

A child process runs with SSM_SCAN_TEST_FAIL_WAITS=2: the wait's limit is zero for that warp and short
for its peers.  The call must end, with NaN from there on in y, the slot and the gradients (a block that
stops may write NaN over its last two rounds too); what is not NaN, and sequences of one round, must be
right.  Nothing here faults the GPU."""
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent("""
    import torch
    import state_space_model_ssm_gb300 as pkg
    from oracle import layers as ol
    from tests.layer_helpers import close, gated_bounds, np64
    from tests.test_gated_scan_gpu import _backward, _case, _forward, _ref_args

    # 4 blocks share the first sequence (rounds of 256 tokens), 2 the second (one round)
    for rounds in (3, 4, 5, 6):
        long = 256 * rounds - 40
        for dt in (torch.float32, torch.bfloat16):
            for C in (96, 95):                             # TMA, and rows it cannot describe
                c = _case(C, [long, 100], resume=[1, 1], dtype=dt, seed=rounds)
                y, slots, ch = _forward(c, train=True)
                ch.nan_to_num_(0.0)
                grads = _backward(c, ch)
                torch.cuda.synchronize()
                args = _ref_args(c)
                y_ref, s_ref = ol.gated_scan(*args)
                gy, gs = np64(c["grad_y"]), np64(c["grad_state"])
                ref = ol.gated_scan_backward(gy, gs, *args)
                b = gated_bounds(*args, grad_y=gy, grad_state=gs)
                assert torch.isnan(slots[0]).all()
                assert torch.isnan(y[256 * (rounds - 1):long]).any(0).all()
                lost = torch.isnan(y).cpu().numpy()
                assert lost[:long].any() and not lost[long:].any()
                close(torch.where(torch.isnan(y), torch.from_numpy(y_ref).to(y), y), y_ref, b["y"], dt)
                close(slots[1], s_ref[1], b["slots"][1])
                assert torch.isnan(grads[3]).all() and torch.isnan(grads[4][0]).all()
                assert all(torch.isnan(g[:long]).any(0).all() for g in grads[:3])
                for g, r, name in zip(grads[:3], ref, ("grad_x", "grad_gate_a", "grad_gate_x")):
                    close(g[long:], r[long:], b[name][long:], dt)
    print("ok")
""")


def test_one_warp_gives_up_late():
    env = dict(os.environ, SSM_SCAN_TEST_FAIL_WAITS="2", PYTHONPATH=ROOT)
    from state_space_model_ssm_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr


CHILD_MIXED = textwrap.dedent("""
    import torch
    import state_space_model_ssm_gb300 as pkg
    from oracle import layers as ol
    from tests.layer_helpers import close, gated_bounds, np64
    from tests.test_gated_scan_gpu import _backward, _case, _forward, _ref_args

    # long sequences among short ones: 40 of them on 20 blocks of channels, so that blocks take several
    lens = ([1] * 9 + [70]) * 40 + [1] * 200
    long = torch.tensor([n > 32 for n in lens])
    rows = torch.cat([torch.full((n,), n > 32) for n in lens])
    for C in (1280, 96):
        c = _case(C, lens, resume=[1] * len(lens), seed=C)
        y, slots, ch = _forward(c, train=True)
        ch.nan_to_num_(0.0)
        grads = _backward(c, ch)
        torch.cuda.synchronize()
        args = _ref_args(c)
        y_ref, s_ref = ol.gated_scan(*args)
        b = gated_bounds(*args)
        assert torch.isnan(y[rows]).all() and torch.isnan(slots[long]).all()
        close(y[~rows], y_ref[~rows.numpy()], b["y"][~rows.numpy()])
        close(slots[~long], s_ref[~long.numpy()], b["slots"][~long.numpy()])
        assert all(torch.isnan(g[rows]).all() and not torch.isnan(g[~rows]).any() for g in grads[:3])
        assert torch.isnan(grads[3]).all() and torch.isnan(grads[4][long]).all() and not torch.isnan(grads[4][~long]).any()
    print("ok")
""")


def test_long_sequences_among_short_ones_give_up():
    """With SSM_SCAN_TEST_FAIL_WAITS=1 every wait of the walk gives up at once: NaN in the long sequences, one
    after another on the same block, and the stepped ones as they should be."""
    env = dict(os.environ, SSM_SCAN_TEST_FAIL_WAITS="1", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD_MIXED], cwd=ROOT, env=env, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
