"""The plain Fp8Linear refuses what its kernels would read by a wrong address or as a wrong type. No launch is made, so
no GPU is needed."""

import pytest
import torch

from fp8_delayed_scaling_quantize_b200.linear import Fp8Linear


def test_an_input_on_the_host():
    with pytest.raises(ValueError, match="GPU"):
        Fp8Linear(32, 32)(torch.zeros(4, 32, dtype=torch.bfloat16))


def test_a_bias_or_weight_of_another_type():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    for name in ("bias", "weight"):
        layer = Fp8Linear(32, 32)
        p = getattr(layer, name)
        p.data = p.data.float()
        with pytest.raises(TypeError, match="bf16"):
            layer(x)


@pytest.mark.gpu
def test_parameters_on_the_host():
    x = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="device"):
        Fp8Linear(32, 32)(x)
    layer = Fp8Linear(32, 32, device="cuda")
    layer.bias.data = layer.bias.data.cpu()
    with pytest.raises(ValueError, match="device"):
        layer(x)
    with pytest.raises(TypeError, match="bf16"):
        Fp8Linear(32, 32, device="cuda")(x.float())
