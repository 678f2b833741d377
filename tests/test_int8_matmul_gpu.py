"""Parity of the 8-bit integer matrix product with the exact integers (needs a GB300)."""
import numpy as np
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from oracle import layers as ol
from tests.layer_helpers import DTYPES, U, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _inputs(M, N, K, seed=0, full=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-128, 128, (M, K), generator=g).to(torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g).to(torch.int8)
    if full:
        x.fill_(-128)
        w.fill_(-128)
    return (x.cuda(), (torch.rand(M, generator=g) * 0.1 + 1e-3).cuda(), w.cuda(),
            (torch.rand(N, generator=g) * 0.1 + 1e-3).cuda(), torch.randn(N, generator=g).cuda())


def _check(x, xs, w, ws, bias, out):
    ref = ol.int8_matmul(x.cpu().numpy(), xs.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy(),
                         None if bias is None else bias.cpu().numpy())
    plain = ref if bias is None else ref - bias.double().cpu().numpy()[None, :]
    # the integer rounded to fp32, two products, the bias
    close(out, ref, 3.01 * U * np.abs(plain) + U * np.abs(ref), out.dtype)


SIZES = [(1, 1, 1), (1, 8, 16), (3, 5, 7), (1, 300, 64), (2, 257, 1000), (16, 128, 128), (17, 130, 129), (33, 64, 4096),
         (64, 192, 513), (65, 127, 2048), (128, 128, 64), (129, 300, 96), (200, 1000, 1003), (256, 256, 256),
         (300, 520, 1536), (777, 401, 80), (40, 8200, 160), (64, 8191, 1040)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(M, N, K, dtype):
    x, xs, w, ws, bias = _inputs(M, N, K, seed=M + N + K)
    for b in (None, bias):
        _check(x, xs, w, ws, b, pkg.ssm_int8_matmul(x, xs, w, ws, bias=b, out_dtype=DTYPES[dtype]))


@pytest.mark.parametrize("M,N,K", [(4, 40, 9000), (130, 140, 5000), (260, 270, 16384)])
def test_largest_codes(M, N, K):
    """Every code -128: sums far past 2^24 are still the integers (rounded once)."""
    x, xs, w, ws, _ = _inputs(M, N, K, full=True)
    _check(x, xs, w, ws, None, pkg.ssm_int8_matmul(x, xs, w, ws, out_dtype=torch.float32))
    x[:, ::3] = 127
    w[:, 1::2] = 127
    _check(x, xs, w, ws, None, pkg.ssm_int8_matmul(x, xs, w, ws, out_dtype=torch.float32))


@pytest.mark.parametrize("M,N,K", [(5, 64, 256), (150, 140, 256), (300, 256, 1040)])
@pytest.mark.parametrize("off", [0, 1, 16])
def test_strided_rows(M, N, K, off):
    """Operands and output inside wider tensors; nothing beside the output is written."""
    x, xs, w, ws, bias = _inputs(M, N, K, seed=7)
    wx, ww = (torch.full((r, K + 32), 99, dtype=torch.int8, device="cuda") for r in (M, N))
    wx[:, off:off + K], ww[:, off:off + K] = x, w
    out = torch.full((M, N + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    pkg.ssm_int8_matmul(wx[:, off:off + K], xs, ww[:, off:off + K], ws, bias=bias, out=out[:, off:off + N][:, :N])
    _check(x, xs, w, ws, bias, out[:, off:off + N])
    assert (out[:, :off] == 3).all() and (out[:, off + N:] == 3).all()


def test_zero_rows_and_same_bits():
    x, xs, w, ws, bias = _inputs(70, 90, 500)
    assert pkg.ssm_int8_matmul(x[:0], xs[:0], w, ws).shape == (0, 90)
    a, b = (pkg.ssm_int8_matmul(x, xs, w, ws, bias=bias) for _ in range(2))
    assert torch.equal(a, b)


def test_chain_norm_projection():
    """add + norm in 8 bits into the product: the float product of the dequantised codes."""
    g = torch.Generator().manual_seed(1)
    T, D, N = 50, 256, 96
    x, r = (torch.randn(T, D, generator=g).cuda().bfloat16() for _ in range(2))
    wt = torch.randn(N, D, generator=g).cuda()
    q, s, h = pkg.ssm_add_norm(x, torch.ones(D, device="cuda"), r, quant="int8")
    wq, ws = pkg.ssm_quantize_rows(wt)
    out = pkg.ssm_int8_matmul(q, s, wq, ws, out_dtype=torch.float32)
    ref = (q.double() * s.double()[:, None]) @ (wq.double() * ws.double()[:, None]).t()
    close(out, ref.cpu().numpy(), 4 * U * np.abs(ref.cpu().numpy()))


@pytest.mark.parametrize("M,N,K", [(8192, 2048, 1024), (1024, 16384, 1024), (2500, 8192, 2048)])
def test_many_tiles_are_exact_every_time(M, N, K):
    """Many waves of tiles of either width, repeated: every sum is the integer (small enough for an exact fp32 product)."""
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randint(-60, 61, (r, K), generator=g).to(torch.int8).cuda() for r in (M, N))
    ref = x.float() @ w.float().t()                        # below 2^24: exact in any order
    xs, ws = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    for _ in range(30):
        assert torch.equal(pkg.ssm_int8_matmul(x, xs, w, ws, out_dtype=torch.float32), ref)
