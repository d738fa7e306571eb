"""Arguments of the wrong kind are ValueErrors that name them, also those that no
table can be asked for (CPU only)."""
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe

x = torch.zeros(2, 8, dtype=torch.bfloat16)


@pytest.mark.parametrize("name,call", [
    ("eps", lambda v: moe.rms_norm(x, out=x.clone(), eps=v)),
    ("eps", lambda v: moe.rms_norm_backward(x, x, out=x.clone(), eps=v)),
    ("element", lambda v: moe.quantize_mx(x, v)),
    ("quantize", lambda v: moe.rms_norm(x, quantize=v)),
])
@pytest.mark.parametrize("value", [[1e-6], {"fp8": 1}, torch.ones(3), torch.tensor(1e-6)], ids=["list", "dict", "tensor", "scalar"])
def test_named_in_a_value_error(name, call, value):
    with pytest.raises(ValueError, match=name):
        call(value)


@pytest.mark.parametrize("value", [pytest.param(10 ** 400, id="large"), 1e300, 2.0 ** -151, -0.0, float("-inf"), float("nan"), -1])
def test_eps_of_any_size(value):
    with pytest.raises(ValueError, match="eps"):
        moe.rms_norm(x, out=x.clone(), eps=value)
