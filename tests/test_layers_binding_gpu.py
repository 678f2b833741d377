"""The layer operators called with every argument by name, on the current and on another stream (needs a GB300)."""
import pytest
import torch

import state_space_model_ssm_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _calls():
    g = torch.Generator(device="cuda").manual_seed(3)
    T, C = 70, 64
    x, ga, gx, gy = (torch.randn(T, C, generator=g, device="cuda") for _ in range(4))
    i32 = dict(dtype=torch.int32, device="cuda")
    meta = dict(seq_starts=torch.tensor([0], **i32), seq_lens=torch.tensor([T], **i32),
                resume_flags=torch.tensor([1], **i32))
    lam, w = torch.zeros(C, device="cuda"), torch.ones(C, device="cuda")
    chunks = pkg.gated_scan_chunk_states(1, T, C)
    pkg.ssm_gated_scan(torch.ones(1, C, device="cuda"), x, ga, gx, lam, *meta.values(), chunk_states=chunks)
    q, s = pkg.ssm_quantize_rows(x)
    torch.cuda.synchronize()
    return {
        "ssm_gated_scan": lambda: dict(state_slots=torch.ones(1, C, device="cuda"), x=x, gate_a=ga, gate_x=gx, lam=lam, **meta),
        "ssm_gated_scan_backward": lambda: dict(grad_y=gy, x=x, gate_a=ga, gate_x=gx, lam=lam, chunk_states=chunks, **meta),
        "ssm_add_norm": lambda: dict(x=x, weight=w, residual=gx),
        "ssm_add_norm_backward": lambda: dict(grad_y=gy, h=x, weight=w),
        "ssm_quantize_rows": lambda: dict(x=x),
        "ssm_int8_matmul": lambda: dict(x=q, x_scales=s, w=q, w_scales=s),
    }


@pytest.mark.parametrize("name", ["ssm_gated_scan", "ssm_gated_scan_backward", "ssm_add_norm", "ssm_add_norm_backward",
                                  "ssm_quantize_rows", "ssm_int8_matmul"])
def test_by_name_is_by_place(name):
    fn, args = getattr(pkg, name), _calls()[name]

    def flat(v):
        return list(v) if isinstance(v, tuple) else [v]

    want = flat(fn(*args().values()))
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        a = args()
        torch.cuda.synchronize()
        got = flat(fn(**a, stream=stream))
        torch.cuda.synchronize()
        assert len(got) == len(want) and all(torch.equal(p, q) for p, q in zip(got, want))
