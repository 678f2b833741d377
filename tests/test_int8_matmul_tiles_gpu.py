"""Either tile width of the 8-bit integer matrix product with sizes that its tests of few tiles do not
reach: several folds of the accumulator, remainders in all three sizes, all output types, scales, bias and
extreme codes at 256 tokens a tile, and many tiles repeated at 128 (needs a GB300).

A tile is 256 tokens wide where that gives at least 152 of them, else 128."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from tests.layer_helpers import DTYPES, U, close

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _wide(M, N):
    return -(-N // 128) * -(-M // 256) >= 152


def _codes(rows, K, g, kind):
    if kind == "any":
        return torch.randint(-128, 128, (rows, K), generator=g).to(torch.int8).cuda()
    v = {"lowest": -128, "highest": 127}[kind]
    return torch.full((rows, K), v, dtype=torch.int8, device="cuda")


def _exact(x, w):
    return x.double() @ w.double().t()                       # below 2^53


# 256 tokens: one to eight folds, remainders in the tokens, channels and terms
WIDE = [(2500, 2050, 4096), (2500, 2050, 4100), (2561, 1921, 1025), (2500, 2050, 8190), (20000, 130, 2049),
        (300, 9700, 3000), (256, 19456, 1024), (2305, 2177, 129)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,N,K", WIDE)
def test_wide_tiles(M, N, K, dtype):
    assert _wide(M, N)
    g = torch.Generator().manual_seed(M + N + K)
    x, w = _codes(M, K, g, "any"), _codes(N, K, g, "any")
    xs, ws = ((torch.rand(r, generator=g) * 0.1 + 1e-3).cuda() for r in (M, N))
    bias = torch.randn(N, generator=g).cuda()
    plain = _exact(x, w) * xs.double()[:, None] * ws.double()
    for b in (None, bias):
        ref = plain if b is None else plain + b.double()
        out = torch.full((M, N + 9), 3.0, dtype=DTYPES[dtype], device="cuda")
        pkg.ssm_int8_matmul(x, xs, w, ws, bias=b, out=out[:, 4:4 + N])
        # the integer rounded to fp32, two products, the bias
        close(out[:, 4:4 + N], ref.cpu().numpy(), (3.01 * U * plain.abs() + U * ref.abs()).cpu().numpy(), out.dtype)
        assert (out[:, :4] == 3).all() and (out[:, 4 + N:] == 3).all()


@pytest.mark.parametrize("M,N,K", [(2500, 2050, 4100), (300, 260, 4100), (70, 40, 9001), (12, 40, 9001)])
@pytest.mark.parametrize("kinds", [("lowest", "lowest"), ("highest", "highest"), ("lowest", "highest"),
                                   ("any", "lowest"), ("highest", "any")])
def test_extreme_codes(M, N, K, kinds):
    """Sums at the edge of what a fold holds, odd ones among them."""
    g = torch.Generator().manual_seed(K)
    x, w = _codes(M, K, g, kinds[0]), _codes(N, K, g, kinds[1])
    x[::2, 5], w[1::2, -1] = 127, 1                          # (so that not all sums are even)
    one = [torch.ones(r, device="cuda") for r in (M, N)]
    ref = _exact(x, w)
    out = pkg.ssm_int8_matmul(x, one[0], w, one[1], out_dtype=torch.float32)
    assert torch.equal(out, ref.float())                     # the exact integer, rounded once


@pytest.mark.parametrize("M,N,K", [(2048, 2304, 4096), (2300, 2000, 4100), (128, 16384, 4096), (640, 6400, 2050)])
def test_many_narrow_tiles_are_exact_every_time(M, N, K):
    assert not _wide(M, N)
    g = torch.Generator().manual_seed(M)
    x, w = _codes(M, K, g, "any"), _codes(N, K, g, "any")
    ref = _exact(x, w).float()
    one = [torch.ones(r, device="cuda") for r in (M, N)]
    for _ in range(30):
        assert torch.equal(pkg.ssm_int8_matmul(x, one[0], w, one[1], out_dtype=torch.float32), ref)


@pytest.mark.parametrize("M,N,K", [(2500, 2050, 4100), (4096, 3000, 8192)])
def test_many_wide_tiles_with_several_folds_are_exact_every_time(M, N, K):
    assert _wide(M, N)
    g = torch.Generator().manual_seed(M)
    x, w = _codes(M, K, g, "any"), _codes(N, K, g, "any")
    ref = _exact(x, w).float()
    one = [torch.ones(r, device="cuda") for r in (M, N)]
    for _ in range(30):
        assert torch.equal(pkg.ssm_int8_matmul(x, one[0], w, one[1], out_dtype=torch.float32), ref)


CHILD = textwrap.dedent("""
    import torch
    import state_space_model_ssm_gb300 as pkg

    for M, N, K in ((2500, 2050, 300), (2500, 2050, 4100), (300, 260, 4100)):
        x, w = (torch.ones(r, K, dtype=torch.int8, device="cuda") for r in (M, N))
        out = pkg.ssm_int8_matmul(x, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"))
        torch.cuda.synchronize()
        assert torch.isnan(out).all(), (M, N, K)
    # a product without pipeline waits on the same context
    x, w = torch.ones(5, 64, dtype=torch.int8, device="cuda"), torch.ones(40, 64, dtype=torch.int8, device="cuda")
    out = pkg.ssm_int8_matmul(x, torch.ones(5, device="cuda"), w, torch.ones(40, device="cuda"))
    assert (out == 64).all()
    print("ok")
""")


def test_wide_tiles_that_give_up_write_nan():
    """Every bounded wait gives up at once (SSM_SCAN_TEST_FAIL_WAITS=1): the call ends, with NaN."""
    env = dict(os.environ, SSM_SCAN_TEST_FAIL_WAITS="1", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
