"""The bounded waits of the gated scan's clusters and of the 8-bit product give up cleanly (needs a GB300).

A child process runs with SSM_SCAN_TEST_FAIL_WAITS=1, so every such wait gives up at once: outputs
(and slots, gradients) must be NaN, nothing may stall, and the same context must then run kernels
without such waits correctly.  Nothing here faults the GPU: the failure is a flag nothing sets."""
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

    T, C = 1500, 96
    x, ga, gx, gy = (torch.randn(T, C, device="cuda") for _ in range(4))
    lam, slots = torch.zeros(C, device="cuda"), torch.zeros(2, C, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    meta = (torch.tensor([0, 1400], **i32), torch.tensor([1400, 100], **i32), torch.tensor([1, 0], **i32))
    ch = pkg.gated_scan_chunk_states(2, T, C)
    ch.zero_()
    for dt in (torch.float32, torch.bfloat16):
        for off in (0, 1):                                 # TMA, and rows it cannot describe
            parts = []
            for v in (x, ga, gx, gy):
                wide = torch.zeros(T, C + 8, dtype=dt, device="cuda")
                wide[:, off:off + C] = v.to(dt)
                parts.append(wide[:, off:off + C])
            y = pkg.ssm_gated_scan(slots, *parts[:3], lam, *meta, chunk_states=ch)
            grads = pkg.ssm_gated_scan_backward(parts[3], *parts[:3], lam, ch, *meta)
            torch.cuda.synchronize()
            if off == 0:
                assert torch.isnan(y).all() and torch.isnan(slots).all()
                assert all(torch.isnan(g).all() for g in grads[:4]) and torch.isnan(grads[4][0]).all()
            else:                                          # the first sequence's cluster waits for its peers
                assert torch.isnan(y[:1400]).all() and torch.isnan(slots[0]).all()
                assert all(torch.isnan(g[:1400]).all() for g in grads[:3]) and torch.isnan(grads[3]).all()
    for M in (100, 600):
        xq, xs = pkg.ssm_quantize_rows(torch.randn(M, 512, device="cuda"))
        wq, ws = pkg.ssm_quantize_rows(torch.randn(300, 512, device="cuda"))
        out = pkg.ssm_int8_matmul(xq, xs, wq, ws)
        torch.cuda.synchronize()
        assert torch.isnan(out).all(), M
    # kernels without pipeline waits on the same context
    h = torch.randn(50, 96, device="cuda")
    y, _ = pkg.ssm_add_norm(h, torch.ones(96, device="cuda"))
    ref = h.double() / torch.sqrt((h.double() ** 2).mean(1, keepdim=True) + 1e-6)
    assert ((y.double() - ref).abs() <= 1e-5).all()
    print("ok")
""")


def test_waits_that_give_up_write_nan():
    env = dict(os.environ, SSM_SCAN_TEST_FAIL_WAITS="1", PYTHONPATH=ROOT)
    from state_space_model_ssm_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
