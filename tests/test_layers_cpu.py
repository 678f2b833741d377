"""Refusals of the layer operators without a GPU: every call below fails a host check (or has no
work), so the aligned fake pointers are never dereferenced."""
import ctypes

import pytest
import torch

from state_space_model_ssm_gb300 import binding as bd
from state_space_model_ssm_gb300 import layers

P = 0x10000
INV, UNS = bd.SSM_ERR_INVALID_ARG, bd.SSM_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from state_space_model_ssm_gb300 import build
    build.build()
    return bd.load()


def _call(fn, defaults, **over):
    a = dict(defaults)
    a.update(over)
    return fn(*[None if v == 0 and k.startswith("p_") else v for k, v in a.items()])


SCAN = dict(p_state=P, p_x=P, p_ga=P, p_gx=P, p_lam=P, scale=8.0, p_y=P, p_starts=P, p_lens=P, p_resume=P, n=2, T=8,
            C=16, dtype=1, sx=16, sga=16, sgx=16, sy=16, p_chunks=0, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(n=-1), INV), (dict(T=-1), INV), (dict(C=0), INV), (dict(dtype=3), INV), (dict(dtype=-1), INV),
    (dict(scale=0.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(sx=15), INV), (dict(sga=15), INV), (dict(sgx=0), INV), (dict(sy=-16), INV),
    (dict(p_state=0), INV), (dict(p_x=0), INV), (dict(p_ga=0), INV), (dict(p_gx=0), INV), (dict(p_lam=0), INV),
    (dict(p_y=0), INV), (dict(p_starts=0), INV), (dict(p_lens=0), INV), (dict(p_resume=0), INV),
    (dict(p_state=P + 2), INV), (dict(p_x=P + 1), INV), (dict(p_y=P + 1), INV), (dict(dtype=0, p_ga=P + 2), INV),
    (dict(p_chunks=P + 1), INV), (dict(n=2**31 - 1, C=64, sx=64, sga=64, sgx=64, sy=64), UNS),
])
def test_gated_scan_refuses(lib, over, expect):
    assert _call(lib.ssm_gated_scan, SCAN, **over) == expect


def test_gated_scan_nothing_to_do(lib):
    assert _call(lib.ssm_gated_scan, SCAN, n=0, p_state=0, p_x=0) == 0
    assert lib.ssm_gated_scan_chunks(2, 100, 8) >= 2 + 100 // 4096
    assert lib.ssm_gated_scan_chunks(-1, 100, 8) == 0 and lib.ssm_gated_scan_chunks(1, 1, 0) == 0
    assert lib.ssm_gated_scan_backward_workspace_bytes(16, 16, 64) > 0
    assert lib.ssm_gated_scan_backward_workspace_bytes(0, 16, 64) == 0


BACK = dict(p_gy=P, p_gs=P, p_x=P, p_ga=P, p_gx=P, p_lam=P, scale=8.0, p_chunks=P, p_starts=P, p_lens=P, p_resume=P,
            n=2, T=8, C=16, dtype=1, sx=16, sga=16, sgx=16, sgy=16, p_dx=P, p_da=P, p_dg=P, tx=16, ta=16, tg=16,
            p_dlam=P, p_d0=P, p_ws=P, ws=1 << 20, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(n=-1), INV), (dict(C=-4), INV), (dict(dtype=7), INV), (dict(scale=-1.0), INV), (dict(sgy=3), INV),
    (dict(tx=3), INV), (dict(ta=3), INV), (dict(tg=3), INV), (dict(p_gy=0), INV), (dict(p_x=0), INV),
    (dict(p_chunks=0), INV), (dict(p_dx=0), INV), (dict(p_da=0), INV), (dict(p_dg=0), INV), (dict(p_dlam=0), INV),
    (dict(p_lam=0), INV), (dict(p_ws=0), INV), (dict(ws=100), INV), (dict(p_ws=P + 4), INV), (dict(p_dx=P + 1), INV),
    (dict(p_d0=P + 2), INV), (dict(p_gs=P + 1), INV), (dict(p_resume=0), INV),
])
def test_gated_scan_backward_refuses(lib, over, expect):
    assert _call(lib.ssm_gated_scan_backward, BACK, **over) == expect


NORM = dict(p_x=P, p_r=P, p_w=P, eps=1e-6, p_h=P, p_y=P, p_q=0, p_s=0, rows=4, D=16, dtype=1, rdtype=1, sx=16, sr=16,
            sh=16, sy=16, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(rows=-1), INV), (dict(D=0), INV), (dict(D=20000, sx=20000, sr=20000, sh=20000, sy=20000), UNS),
    (dict(dtype=4), INV), (dict(rdtype=2), INV), (dict(dtype=0, rdtype=1), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(sx=8), INV), (dict(sr=8), INV), (dict(sh=8), INV), (dict(sy=8), INV),
    (dict(p_x=0), INV), (dict(p_w=0), INV), (dict(p_y=0), INV), (dict(p_q=P), INV), (dict(p_y=0, p_q=P), INV),
    (dict(p_s=P), INV), (dict(p_r=0), INV), (dict(p_x=P + 1), INV), (dict(rdtype=0, p_r=P + 2), INV),
    (dict(p_w=P + 2), INV),
])
def test_add_norm_refuses(lib, over, expect):
    assert _call(lib.ssm_add_norm, NORM, **over) == expect


def test_add_norm_no_rows(lib):
    assert _call(lib.ssm_add_norm, NORM, rows=0) == 0


NBACK = dict(p_gy=P, p_h=P, p_w=P, eps=1e-6, p_gh=P, p_gin=P, p_gw=P, rows=4, D=16, dtype=1, rdtype=1, sgy=16, sh=16,
             sgh=16, sgi=16, p_ws=P, ws=1 << 20, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(rows=-1), INV), (dict(D=0), INV), (dict(D=20000, sgy=20000, sh=20000, sgh=20000, sgi=20000), UNS),
    (dict(dtype=5), INV), (dict(rdtype=2), INV), (dict(sgy=1), INV), (dict(sh=1), INV), (dict(sgh=1), INV),
    (dict(sgi=1), INV), (dict(p_gy=0), INV), (dict(p_h=0), INV), (dict(p_gin=0), INV), (dict(p_gw=0), INV),
    (dict(p_w=0), INV), (dict(p_ws=0), INV), (dict(ws=10), INV), (dict(p_gh=P + 1), INV), (dict(eps=float("inf")), INV),
])
def test_add_norm_backward_refuses(lib, over, expect):
    assert _call(lib.ssm_add_norm_backward, NBACK, **over) == expect


QUANT = dict(p_x=P, p_q=P, p_s=P, rows=4, D=16, dtype=1, sx=16, sq=16, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(rows=-2), INV), (dict(D=0), INV), (dict(D=16385, sx=16385, sq=16385), UNS), (dict(dtype=9), INV),
    (dict(sx=2), INV), (dict(sq=2), INV), (dict(p_x=0), INV), (dict(p_q=0), INV), (dict(p_s=0), INV),
    (dict(p_s=P + 2), INV), (dict(p_x=P + 1), INV),
])
def test_quantize_rows_refuses(lib, over, expect):
    assert _call(lib.ssm_quantize_rows, QUANT, **over) == expect


MM = dict(p_x=P, p_xs=P, p_w=P, p_ws=P, p_b=0, p_out=P, M=4, N=16, K=32, dtype=1, sx=32, sw=32, so=16, p_work=P,
          work=1 << 30, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(dtype=3), INV), (dict(sx=31), INV), (dict(sw=31), INV),
    (dict(so=15), INV), (dict(K=131072, sx=131072, sw=131072), UNS), (dict(p_x=0), INV), (dict(p_xs=0), INV),
    (dict(p_w=0), INV), (dict(p_ws=0), INV), (dict(p_out=0), INV), (dict(p_out=P + 1), INV), (dict(p_b=P + 2), INV),
    (dict(p_xs=P + 1), INV),
])
def test_int8_matmul_refuses(lib, over, expect):
    assert _call(lib.ssm_int8_matmul, MM, **over) == expect


def test_int8_matmul_no_rows(lib):
    assert _call(lib.ssm_int8_matmul, MM, M=0) == 0


def test_binding_refuses_cpu_tensors_and_wrong_types():
    z = torch.zeros(2, 4)
    i = torch.zeros(1, dtype=torch.int32)
    for f in (lambda: layers.ssm_gated_scan(z, z, z, z, z[0], i, i, i), lambda: layers.ssm_add_norm(z, z[0]),
              lambda: layers.ssm_add_norm_backward(z, z, z[0]), lambda: layers.ssm_quantize_rows(z)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        layers.ssm_int8_matmul(z.to(torch.int8), z[:, 0], z.to(torch.int8), z[:, 0])
    with pytest.raises(TypeError):
        layers.ssm_int8_matmul(z[0], z[0], z, z[0])
    with pytest.raises(TypeError):
        layers.ssm_quantize_rows([1.0])


def test_row_checks_of_the_binding():
    cpu = torch.device("cpu")
    t = torch.zeros(4, 12)
    f32 = torch.float32
    assert layers._rows(t[:, 2:8], "t", f32, cpu, (4, 6)) == (t.data_ptr() + 8, 12)
    assert layers._rows(t[:1, :3], "t", f32, cpu, (1, 3))[1] >= 3
    for bad, err in ((t.double(), TypeError), (t[:, ::2], ValueError), (t.t(), ValueError),
                     (t[:1].expand(4, 12), ValueError), (t[:3], ValueError), ("t", TypeError)):
        with pytest.raises(err):
            layers._rows(bad, "t", f32, cpu, (4, 6) if bad is not t and not isinstance(bad, str) and
                         tuple(bad.shape) == (4, 6) else (4, 12))
    assert ctypes.sizeof(ctypes.c_void_p) == 8
