"""As many rows as the interface's 32-bit count holds, 4 to a block, and rows far past 2^32 elements apart
(needs a GB300; about 20 GB)."""
import pytest
import torch

import state_space_model_ssm_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def test_most_rows():
    rows, part = 2**31 - 1, 2**27
    x = torch.empty(rows, 1, dtype=torch.float16, device="cuda")
    period = (torch.arange(part, device="cuda") % 7 - 3).to(torch.float16)[:, None]
    for at in range(0, rows, part):
        x[at:at + part] = period[:rows - at]
    q, s = pkg.ssm_quantize_rows(x)
    # one value a row: its code is 127 with its sign (0 for zero), its scale |x| / 127
    code = (torch.sign(period) * 127).to(torch.int8)
    top = period.double().abs()[:, 0]
    f = torch.full_like(top, 127).div(top).clamp(max=torch.finfo(torch.float32).max).float()
    scale = torch.ones_like(top).div(f.double()).float()     # each quotient in 64 bits, rounded to 32
    for at in range(0, rows, part):
        n = min(part, rows - at)
        assert torch.equal(q[at:at + n], code[:n]) and torch.equal(s[at:at + n], scale[:n])


def test_rows_far_apart():
    """Row 3 begins 6.4e9 elements past row 0."""
    T, D, stride = 4, 256, (1 << 31) + 8
    flat = torch.zeros(3 * stride + D, dtype=torch.float16, device="cuda")
    x = torch.as_strided(flat, (T, D), (stride, 1))
    x.copy_(torch.randn(T, D, generator=torch.Generator().manual_seed(1)).to(torch.float16))
    w = torch.ones(D, device="cuda")
    dense = x.contiguous()
    for a, b in zip(pkg.ssm_quantize_rows(x), pkg.ssm_quantize_rows(dense)):
        assert torch.equal(a, b)
    assert torch.equal(pkg.ssm_add_norm(x, w)[0], pkg.ssm_add_norm(dense, w)[0])
    gin, gw = pkg.ssm_add_norm_backward(x, x, w)
    want = pkg.ssm_add_norm_backward(dense, dense, w)
    assert torch.equal(gin, want[0]) and torch.equal(gw, want[1])
