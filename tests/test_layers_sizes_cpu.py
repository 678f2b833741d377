"""Sizes near 2^31 are refused before any launch, where the kernels' 32-bit token counts would not hold
them (no GPU: the pointers are never read)."""
import pytest

from state_space_model_ssm_gb300 import binding as bd
from tests.test_layers_cpu import BACK, MM, SCAN, _call

UNS = bd.SSM_ERR_UNSUPPORTED
TOP = 2**31 - 1


@pytest.fixture(scope="module")
def lib():
    from state_space_model_ssm_gb300 import build
    build.build()
    return bd.load()


@pytest.mark.parametrize("T", [TOP, TOP - 511])
def test_gated_scan_tokens(lib, T):
    one = dict(n=1, T=T, C=1, sx=1, sga=1, sgx=1)
    assert _call(lib.ssm_gated_scan, SCAN, sy=1, **one) == UNS
    assert _call(lib.ssm_gated_scan_backward, BACK, sgy=1, tx=1, ta=1, tg=1, **one) == UNS
    assert lib.ssm_gated_scan_chunks(1, T, 1) == 0
    assert lib.ssm_gated_scan_backward_workspace_bytes(1, T, 1) == 0
    assert lib.ssm_gated_scan_chunks(1, TOP - 512, 1) == 1 + (TOP - 512) // 64 + 1


@pytest.mark.parametrize("over", [dict(M=TOP), dict(M=TOP - 255), dict(N=TOP, so=TOP), dict(N=TOP - 255, so=TOP)])
def test_int8_matmul_rows(lib, over):
    assert _call(lib.ssm_int8_matmul, MM, **over) == UNS
    rows, out = over.get("M", 4), over.get("N", 16)
    assert lib.ssm_int8_matmul_workspace_bytes(0, 0, rows, out, 32, 32, 32) == 0
