"""Refusals and sizes of the selective-scan model's operators without a GPU: every call below fails a host check (or
has no work), so the aligned fake pointers are never dereferenced."""
import pytest
import torch

import state_space_model_ssm_gb300 as pkg
from state_space_model_ssm_gb300 import binding as bd

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


SCAN = dict(p_state=P, p_x=P, p_dt=P, p_A=P, p_B=P, p_C=P, p_D=P, p_z=P, p_bias=P, softplus=1, p_y=P, p_starts=P, p_lens=P,
            p_resume=P, n=2, T=8, C=16, N=16, G=1, dtype=1, sx=16, sdt=16, sB=16, sC=16, sz=16, sy=16, p_chunks=0, p_ws=0,
            ws=0, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(n=-1), INV), (dict(T=-1), INV), (dict(C=0), INV), (dict(N=0), INV), (dict(G=0), INV), (dict(G=3), INV),
    (dict(N=129, sB=129, sC=129), UNS), (dict(dtype=3), INV), (dict(dtype=-1), INV), (dict(sx=15), INV), (dict(sdt=15), INV),
    (dict(sB=15), INV), (dict(sC=15), INV), (dict(G=2, sB=16), INV), (dict(sz=15), INV), (dict(sy=15), INV),
    (dict(p_state=0), INV), (dict(p_x=0), INV), (dict(p_dt=0), INV), (dict(p_A=0), INV), (dict(p_B=0), INV),
    (dict(p_C=0), INV), (dict(p_y=0), INV), (dict(p_starts=0), INV), (dict(p_lens=0), INV), (dict(p_resume=0), INV),
    (dict(p_state=P + 2), INV), (dict(p_A=P + 2), INV), (dict(p_D=P + 2), INV), (dict(p_bias=P + 1), INV),
    (dict(p_x=P + 1), INV), (dict(p_z=P + 1), INV), (dict(dtype=0, p_B=P + 2), INV), (dict(p_chunks=P + 2), INV),
    (dict(T=4096, C=1024, sx=1024, sdt=1024, sz=1024, sy=1024), INV),       # a workspace is needed
    (dict(T=4096, C=1024, sx=1024, sdt=1024, sz=1024, sy=1024, p_ws=P + 4, ws=1 << 30), INV),
    (dict(T=4096, C=1024, sx=1024, sdt=1024, sz=1024, sy=1024, p_ws=P, ws=1000), INV),
    (dict(n=2**31 - 1, C=64, sx=64, sdt=64, sz=64, sy=64), UNS), (dict(T=2**31 - 1), UNS),
    (dict(n=1 << 20, C=1 << 20, sx=1 << 20, sdt=1 << 20, sz=1 << 20, sy=1 << 20), UNS),
])
def test_scan_refuses(lib, over, expect):
    assert _call(lib.ssm_selective_scan, SCAN, **over) == expect


BACK = dict(p_gy=P, p_gs=P, p_x=P, p_dt=P, p_A=P, p_B=P, p_C=P, p_D=P, p_z=P, p_bias=P, softplus=1, p_chunks=P, p_starts=P,
            p_lens=P, p_resume=P, n=2, T=8, C=16, N=16, G=1, dtype=1, sgy=16, sx=16, sdt=16, sB=16, sC=16, sz=16, p_gx=P,
            p_gdt=P, p_gA=P, p_gB=P, p_gC=P, p_gD=P, p_gz=P, p_gbias=P, p_g0=P, tx=16, tdt=16, tB=16, tC=16, tz=16, p_ws=P,
            ws=1 << 24, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(n=-1), INV), (dict(N=200, sB=200, sC=200, tB=200, tC=200), UNS), (dict(dtype=5), INV), (dict(sgy=1), INV),
    (dict(tx=1), INV), (dict(tdt=1), INV), (dict(tB=1), INV), (dict(tC=1), INV), (dict(tz=1), INV), (dict(p_gy=0), INV),
    (dict(p_x=0), INV), (dict(p_chunks=0), INV), (dict(p_gx=0), INV), (dict(p_gdt=0), INV), (dict(p_gA=0), INV),
    (dict(p_gB=0), INV), (dict(p_gC=0), INV), (dict(p_D=0), INV), (dict(p_gD=0), INV), (dict(p_z=0), INV), (dict(p_gz=0), INV),
    (dict(p_bias=0), INV), (dict(p_gbias=0), INV), (dict(p_ws=0), INV), (dict(ws=100), INV), (dict(p_ws=P + 8), INV),
    (dict(p_gA=P + 2), INV), (dict(p_g0=P + 1), INV), (dict(p_gs=P + 2), INV), (dict(p_gB=P + 1), INV),
])
def test_scan_backward_refuses(lib, over, expect):
    assert _call(lib.ssm_selective_scan_backward, BACK, **over) == expect


CONV = dict(p_x=P, p_w=P, p_b=P, p_state=P, p_out=P, p_starts=P, p_lens=P, p_resume=P, n=2, T=8, C=16, K=4, silu=1, dtype=1,
            sx=16, so=16, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(n=-1), INV), (dict(T=-1), INV), (dict(C=0), INV), (dict(K=0), INV), (dict(K=9), UNS), (dict(dtype=9), INV),
    (dict(sx=8), INV), (dict(so=8), INV), (dict(p_x=0), INV), (dict(p_w=0), INV), (dict(p_state=0), INV), (dict(p_out=0), INV),
    (dict(p_starts=0), INV), (dict(p_lens=0), INV), (dict(p_resume=0), INV), (dict(p_x=P + 1), INV), (dict(p_w=P + 2), INV),
    (dict(p_b=P + 2), INV), (dict(p_state=P + 2), INV), (dict(dtype=0, p_out=P + 2), INV), (dict(T=2**31 - 1), UNS),
])
def test_conv_refuses(lib, over, expect):
    assert _call(lib.ssm_causal_conv, CONV, **over) == expect


CONVB = dict(p_go=P, p_gs=P, p_x=P, p_w=P, p_b=P, p_s0=P, p_starts=P, p_lens=P, p_resume=P, n=2, T=8, C=16, K=4, silu=1, dtype=1,
             sgo=16, sx=16, p_gx=P, p_gw=P, p_gb=P, p_g0=P, tx=16, p_ws=P, ws=1 << 24, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(K=9), UNS), (dict(K=-1), INV), (dict(sgo=8), INV), (dict(tx=8), INV), (dict(p_go=0), INV), (dict(p_gx=0), INV),
    (dict(p_gw=0), INV), (dict(p_b=0), INV), (dict(p_gb=0), INV), (dict(p_s0=0, p_g0=0), INV), (dict(p_resume=0), INV),
    (dict(p_s0=0, p_resume=0), INV), (dict(p_ws=0), INV), (dict(ws=64), INV), (dict(p_ws=P + 16), INV), (dict(p_gw=P + 2), INV),
    (dict(p_g0=P + 2), INV), (dict(p_gx=P + 1), INV),
])
def test_conv_backward_refuses(lib, over, expect):
    assert _call(lib.ssm_causal_conv_backward, CONVB, **over) == expect


LOSS = dict(p_h=P, p_w=P, p_t=P, wide=1, ignore=-100, p_loss=P, p_lse=P, T=4, V=100, D=64, dtype=1, sh=64, sw=64, p_ws=P,
            ws=1 << 30, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(T=-1), INV), (dict(V=0), INV), (dict(D=0), INV), (dict(dtype=0), UNS), (dict(dtype=4), INV), (dict(sh=63), INV),
    (dict(sw=63), INV), (dict(D=65537, sh=65537, sw=65537), UNS), (dict(V=2**31 - 1), UNS), (dict(T=2**31 - 1), UNS),
    (dict(p_h=0), INV), (dict(p_w=0), INV), (dict(p_t=0), INV), (dict(p_loss=0), INV), (dict(p_lse=0), INV),
    (dict(p_h=P + 1), INV), (dict(p_w=P + 1), INV), (dict(p_t=P + 4), INV), (dict(p_lse=P + 2), INV), (dict(p_ws=0), INV),
    (dict(p_ws=P + 128), INV), (dict(ws=256), INV),
])
def test_loss_refuses(lib, over, expect):
    assert _call(lib.ssm_linear_cross_entropy, LOSS, **over) == expect


LOSSB = dict(p_gl=P, p_h=P, p_w=P, p_t=P, wide=0, ignore=-100, p_lse=P, p_gh=P, p_gw=P, T=4, V=100, D=64, dtype=2, sh=64, sw=64,
             th=64, tw=64, p_ws=P, ws=1 << 30, p_stream=0)


@pytest.mark.parametrize("over,expect", [
    (dict(T=-1), INV), (dict(dtype=0), UNS), (dict(th=63), INV), (dict(tw=63), INV), (dict(p_gl=0), INV), (dict(p_lse=0), INV),
    (dict(p_gh=0), INV), (dict(p_gh=P + 1), INV), (dict(p_gw=P + 1), INV), (dict(p_t=P + 2), INV), (dict(ws=1000), INV),
])
def test_loss_backward_refuses(lib, over, expect):
    assert _call(lib.ssm_linear_cross_entropy_backward, LOSSB, **over) == expect


def test_nothing_to_do(lib):
    assert _call(lib.ssm_selective_scan, SCAN, n=0, p_state=0, p_x=0) == 0
    assert _call(lib.ssm_causal_conv, CONV, n=0, p_state=0, p_x=0) == 0
    assert _call(lib.ssm_linear_cross_entropy, LOSS, T=0, p_h=0) == 0
    assert _call(lib.ssm_linear_cross_entropy_backward, LOSSB, T=0, p_h=0, p_gw=0) == 0


def test_workspaces(lib):
    assert pkg.selective_scan_workspace_bytes(0, 100, 64, 16) == 0 and pkg.selective_scan_workspace_bytes(64, 64, 64, 16) == 0
    assert pkg.selective_scan_workspace_bytes(1, 8192, 64, 16) > 0
    assert pkg.selective_scan_workspace_bytes(1, 8192, 64, 129) == 0
    assert pkg.selective_scan_backward_workspace_bytes(2, 64, 64, 16) >= 2 * 64 * 18 * 4 + 2 * 64 * 16 * 4
    assert lib.ssm_selective_scan_chunks(3, 100) == 3 + 100 // 16 + 1 and lib.ssm_selective_scan_chunks(-1, 4) == 0
    assert pkg.selective_scan_chunk_states(2, 40, 8, 4, device="cpu").shape == (5, 8, 4)
    assert pkg.causal_conv_backward_workspace_bytes(3, 100, 64, 4) >= 3 * 5 * 64 * 4
    assert pkg.causal_conv_backward_workspace_bytes(0, 100, 64, 4) == 0
    h = torch.zeros(10, 64, dtype=torch.bfloat16)
    flat = torch.zeros(100 * 72 + 64, dtype=torch.bfloat16)
    start = -flat.data_ptr() % 16 // 2
    even, odd = (flat[start + o:start + o + 100 * 72].view(100, 72)[:, :64] for o in (0, 1))
    need = pkg.linear_cross_entropy_workspace_bytes
    assert need(h, odd) - need(h, even) == 100 * 64 * 2 // 256 * 256 + (256 if 100 * 64 * 2 % 256 else 0)
    assert need(h, even, backward=True) > 256 * 256 * 2 and need(h[:0], even) == 0
    with pytest.raises(TypeError):
        need(h, None)
    with pytest.raises(TypeError):
        need(h, even.float())


def test_binding_refuses_what_is_no_cuda_tensor():
    x, i = torch.zeros(4, 8), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.ssm_selective_scan(torch.zeros(1, 8, 4), x, x, torch.zeros(8, 4), x[:, :4], x[:, :4], None, i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.ssm_selective_scan_backward(x, x, x, torch.zeros(8, 4), x[:, :4], x[:, :4], None, x, i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.ssm_causal_conv(x, torch.zeros(8, 4), torch.zeros(1, 8, 3), i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.ssm_causal_conv_backward(x, x, torch.zeros(8, 4), i, i)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.ssm_linear_cross_entropy(x.bfloat16(), x.bfloat16(), i)
    with pytest.raises(TypeError):
        pkg.ssm_linear_cross_entropy(None, x, i)
