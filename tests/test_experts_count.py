"""Fp8Experts refuses a number of experts that its products do not take before any of its rings has moved."""

import pytest

import fp8_delayed_scaling_quantize_b200 as fp8
from fp8_delayed_scaling_quantize_b200.experts import Fp8Experts


@pytest.mark.parametrize("experts", [-1, 0, fp8.FP8_MM_MAX_EXPERTS + 1])
def test_refused(experts):
    with pytest.raises(ValueError, match="experts"):
        Fp8Experts(experts, 16, 16)


@pytest.mark.parametrize("experts", [1, fp8.FP8_MM_MAX_EXPERTS])
def test_taken(experts):
    assert Fp8Experts(experts, 16, 16).weight.shape == (experts, 16, 16)
