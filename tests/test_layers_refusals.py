"""Layers refuse what their kernels could not read: parameters of another type or place than the input's GPU. No
launch is made, so no GPU is needed."""

import pytest
import torch

from fp8_delayed_scaling_quantize_b200.experts import Fp8Experts
from fp8_delayed_scaling_quantize_b200.linear import Fp8Linear, Fp8MLP


def _layers():
    return [(Fp8Linear(32, 32, activation="silu"), ()), (Fp8MLP(32, 64), ()),
            (Fp8Experts(2, 32, 32), (torch.tensor([0, 2, 4], dtype=torch.int32),))]


@pytest.mark.parametrize("i", range(3))
def test_an_input_on_the_host_is_refused(i):
    layer, more = _layers()[i]
    with pytest.raises(ValueError, match="GPU"):
        layer(torch.zeros(4, 32, dtype=torch.bfloat16), *more)


@pytest.mark.parametrize("i", range(3))
def test_parameters_of_another_type_are_refused(i):
    layer, more = _layers()[i]
    with pytest.raises(TypeError, match="bf16"):
        layer.float()(torch.zeros(4, 32, dtype=torch.bfloat16), *more)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(3))
def test_parameters_on_the_host_are_refused(i):
    layer, more = _layers()[i]
    with pytest.raises(ValueError, match="device"):
        layer(torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"), *(t.cuda() for t in more))
