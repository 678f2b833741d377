"""Parity of the 8-bit integer matrix product at every remainder of the inner size (needs a GB300).

The kernels take four terms to a word and put them in an order of their own, so a size that ends
inside a word has its own cases: for few tokens, and for tiles of 128 and of 256 tokens."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from tests.layer_helpers import DTYPES, U, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _inputs(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    x, w = (torch.randint(-128, 128, (r, K), generator=g).to(torch.int8) for r in (M, N))
    x[:, -1], w[:, -1] = 127, -128                          # a last term that no sum can lose
    scales = ((torch.rand(r, generator=g) * 0.1 + 1e-3).cuda() for r in (M, N))
    return (x.cuda(), next(scales), w.cuda(), next(scales), torch.randn(N, generator=g).cuda())


def _check(x, xs, w, ws, bias, out):
    plain = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()      # sums below 2^53: exact
    ref = plain + bias.double()
    # the integer rounded to fp32, two products, the bias
    plain, ref = plain.cpu().numpy(), ref.cpu().numpy()
    close(out, ref, 3.01 * U * np.abs(plain) + U * np.abs(ref), out.dtype)


# few tokens; tiles of 128 tokens (fewer than 152 of 256); tiles of 256
@pytest.mark.parametrize("M,N", [(5, 40), (64, 72), (70, 40), (300, 130), (2500, 2050)])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 6, 18, 34, 62, 63, 64, 65, 66, 67, 126, 130, 1000, 1001, 1002, 1003])
def test_every_remainder(M, N, K):
    x, xs, w, ws, bias = _inputs(M, N, K, seed=M + K)
    for dtype in DTYPES.values() if M <= 300 else (torch.float32,):
        _check(x, xs, w, ws, bias, pkg.ssm_int8_matmul(x, xs, w, ws, bias=bias, out_dtype=dtype))


@pytest.mark.parametrize("M,N", [(70, 40), (2500, 2050)])
@pytest.mark.parametrize("off", [0, 1, 3])
def test_a_word_cut_by_the_rows_end(M, N, off):
    """Rows inside wider tensors: what lies beside the last term is not a term."""
    K = 98
    x, xs, w, ws, bias = _inputs(M, N, K, seed=off)
    wx, ww = (torch.full((r, K + 14), 99, dtype=torch.int8, device="cuda") for r in (M, N))
    wx[:, off:off + K], ww[:, off:off + K] = x, w
    _check(x, xs, w, ws, bias,
           pkg.ssm_int8_matmul(wx[:, off:off + K], xs, ww[:, off:off + K], ws, bias=bias, out_dtype=torch.float32))
