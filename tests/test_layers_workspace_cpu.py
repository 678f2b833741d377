"""Sizes of the layer operators' workspaces as a user asks for them (no GPU)."""
import pytest
import torch

import state_space_model_ssm_gb300 as pkg


@pytest.fixture(scope="module", autouse=True)
def built():
    from state_space_model_ssm_gb300 import build
    build.build()
    pkg.load()


def _rows(rows, width, stride=None, off=0):
    """An int8 [rows, width] tensor whose rows begin `off` bytes past 16-byte boundaries when the stride allows."""
    stride = stride or width
    flat = torch.zeros(rows * stride + 64, dtype=torch.int8)
    start = -flat.data_ptr() % 16 + off
    return flat[start:start + rows * stride].view(rows, stride)[:, :width]


def test_gradient_workspaces():
    assert pkg.gated_scan_backward_workspace_bytes(3, 30, 64) >= 3 * 64 * 4
    assert pkg.gated_scan_backward_workspace_bytes(0, 30, 64) == 0
    assert pkg.add_norm_backward_workspace_bytes(5, 100) == 5 * 100 * 4
    assert pkg.add_norm_backward_workspace_bytes(1 << 20, 100) < 1 << 20
    assert pkg.add_norm_backward_workspace_bytes(5, 1 << 20) == 0           # (refused by the call)


def test_product_workspace():
    up = lambda v: (v + 255) // 256 * 256                                  # noqa: E731
    need = pkg.int8_matmul_workspace_bytes
    assert need(_rows(5, 64), _rows(40, 64)) == 0                           # few tokens, whole words
    assert need(_rows(5, 64, 80, 1), _rows(40, 64)) == up(5 * 64)           # the tokens' rows off the boundary
    assert need(_rows(5, 64), _rows(40, 64, 72)) == up(40 * 64)             # the weights' rows at every other one
    assert need(_rows(5, 63, 64), _rows(40, 63, 64)) == up(5 * 64) + up(40 * 64)
    assert need(_rows(200, 64), _rows(40, 64)) == up(200 * 64 * 2)          # tokens as fp16
    assert need(_rows(200, 63, 64), _rows(40, 63, 64)) == up(200 * 64 * 2)
    assert need(_rows(200, 63), _rows(40, 63)) == up(200 * 64 * 2) + up(40 * 64)
    assert need(_rows(0, 64), _rows(40, 64)) == 0
    with pytest.raises(ValueError):
        need(_rows(5, 64), _rows(40, 48))
    with pytest.raises(TypeError):
        need(_rows(5, 64).float(), _rows(40, 64))
    with pytest.raises(TypeError):
        need(_rows(5, 64), None)
