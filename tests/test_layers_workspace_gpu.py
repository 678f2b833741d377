"""Given workspaces of the size that is asked for, and too small ones (needs a GB300)."""
import pytest
import torch

import state_space_model_ssm_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _refused(call, need):
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"),
               torch.empty(need + 256, dtype=torch.uint8, device="cuda")[1:]):
        with pytest.raises(pkg.SsmScanError) as e:
            call(workspace=ws)
        assert e.value.status == -1


@pytest.mark.parametrize("M,N,K", [(5, 40, 63), (200, 130, 63), (200, 130, 64)])
def test_product(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    w, ws = torch.randint(-128, 128, (N, K), generator=g, device="cuda").to(torch.int8), torch.ones(N, device="cuda")
    need, shared = None, None
    for _ in range(6):                                      # other tokens through the same workspace: none are left over
        x = torch.randint(-128, 128, (M, K), generator=g, device="cuda").to(torch.int8)
        xs = torch.ones(M, device="cuda")

        def call(**kw):
            return pkg.ssm_int8_matmul(x, xs, w, ws, out_dtype=torch.float32, **kw)

        if need is None:
            need = pkg.int8_matmul_workspace_bytes(x, w)
            assert need > 0
            shared = torch.empty(need, dtype=torch.uint8, device="cuda")
            _refused(call, need)
        assert torch.equal(call(workspace=shared).double(), x.double() @ w.double().t())


@pytest.mark.parametrize("M,N,K", [(5, 400, 1003), (16, 2000, 500), (64, 130, 999), (200, 400, 1003)])
def test_product_packs_before_it_reads(M, N, K):
    """Calls without a pause, each with operands of its own through one workspace."""
    g = torch.Generator(device="cuda").manual_seed(K)
    ops = [[torch.randint(-128, 128, (r, K), generator=g, device="cuda").to(torch.int8) for r in (M, N)] for _ in range(12)]
    one = [torch.ones(r, device="cuda") for r in (M, N)]
    ws = torch.empty(pkg.int8_matmul_workspace_bytes(*ops[0]), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(M, N, device="cuda") for _ in ops]
    torch.cuda.synchronize()
    for _ in range(20):
        for (x, w), out in zip(ops, outs):
            pkg.ssm_int8_matmul(x, one[0], w, one[1], out=out, workspace=ws)
    for (x, w), out in zip(ops, outs):
        assert torch.equal(out.double(), x.double() @ w.double().t())


def test_norm_gradient():
    T, D = 40, 100
    g, h, w = torch.randn(T, D, device="cuda"), torch.randn(T, D, device="cuda"), torch.ones(D, device="cuda")
    need = pkg.add_norm_backward_workspace_bytes(T, D)

    def call(**kw):
        return pkg.ssm_add_norm_backward(g, h, w, **kw)

    _refused(call, need)
    want = call()
    got = call(workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
