"""The example around the selective scan runs, and its gradients agree with differences (needs a GB300)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "selective_lm.py"), "--channels", "128", "--vocab", "500",
                        "--tokens", "96", "--steps", "3"], capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "serving:" in r.stdout and "training:" in r.stdout
    err = float(r.stdout.split("relative difference")[1].split()[0])
    # decoded rows against one pass: bf16 activations through two projections, each rounding of 2^-9 met a few times
    assert err < 16 * 2.0 ** -9
    for line in r.stdout.splitlines():
        if line.startswith("  gradient of"):
            slope, diff = (float(v) for v in line.split(":")[1].replace("difference", "").split(","))
            # bf16 roundings of every activation and gradient: about ten of 2^-9 each side of the slope's own size, and
            # the difference's loss, of order 6, is a sum of fp32 means (6e-8 relative), over a step of 2e-2 or more
            assert abs(slope - diff) <= 0.05 * max(abs(slope), abs(diff)) + 2e-3, line
