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


def test_extents_past_32_bit_tiles_are_refused():
    """A tile may reach 256 rows or columns past the last one, which has to be counted in 32 bits too."""
    import fp8_delayed_scaling_quantize_b200 as fp8
    A, S, big = 0x7F0000000000, 0x7F0000100000, (1 << 31) - 16

    def act(M=64, N=64, K=64):
        return fp8.raw_status("fp8_mm_act", A, 0, A, 0, S, S, fp8.FP8_NT, M, N, K, 1, 0, 0, 0, None, None, 0, 4, None, 0,
                              None, A + (1 << 40), None)

    def experts(layout, M=64, N=64, K=64):
        return fp8.raw_status("fp8_mm_experts", A, 0, A, 0, S, S, 0, layout, M, N, K, 4, S + 64, None, 0, None,
                              A + (1 << 40), None)

    for kw in (dict(M=big), dict(N=big), dict(K=big)):
        assert act(**kw) == fp8.FP8_ERR_UNSUPPORTED, kw
        for layout in (fp8.FP8_NT, fp8.FP8_NN, fp8.FP8_TN):
            assert experts(layout, **kw) == fp8.FP8_ERR_UNSUPPORTED, (layout, kw)
