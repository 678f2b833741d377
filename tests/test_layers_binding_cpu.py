"""The binding of the layer operators without a GPU: every documented argument can be given by name."""
import inspect

import pytest
import torch

from state_space_model_ssm_gb300 import layers

OPERATORS = ["ssm_gated_scan", "ssm_gated_scan_backward", "ssm_add_norm", "ssm_add_norm_backward",
             "ssm_quantize_rows", "ssm_int8_matmul"]


@pytest.mark.parametrize("name", OPERATORS)
def test_every_argument_by_name(name):
    """On CPU tensors the call is refused for its device (after its arguments are bound)."""
    fn = getattr(layers, name)
    z, i = torch.zeros(2, 4), torch.zeros(1, dtype=torch.int32)
    needed = [p.name for p in inspect.signature(fn).parameters.values() if p.default is p.empty]
    ints = ("seq_starts", "seq_lens", "resume_flags")
    args = {k: i if k in ints else z[0] if k in ("lam", "weight") else z.to(torch.int8) if k in ("w", "x") and
            name == "ssm_int8_matmul" else z[:, 0] if k.endswith("scales") else z for k in needed}
    with pytest.raises(ValueError, match="CUDA"):
        fn(**args)
    with pytest.raises(ValueError, match="CUDA"):
        fn(*args.values())
    with pytest.raises(ValueError, match="CUDA"):
        fn(**args, stream=0)


@pytest.mark.parametrize("name", OPERATORS)
def test_a_missing_argument_is_named(name):
    fn = getattr(layers, name)
    first = next(iter(inspect.signature(fn).parameters))
    with pytest.raises(TypeError, match=f"{name}.*{first}"):
        fn()
