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
            # fp16: the gradients carry about ten roundings of 2^-11 (0.5 %).  The difference is of two losses of 72
            # tokens whose logits, of order one, are off by 2^-11 each at random: 2^-11 / 72^0.5 = 6e-5 a loss, 1.2 % of
            # the 1e-2 between them.  The step moves no exponent or activation by more than 0.3: its third-order term
            # is at most 0.3^2 / 6 = 1.5 %.  Together below 5 % with three times the losses' error.
            assert abs(slope - diff) <= 0.05 * max(abs(slope), abs(diff)), line
