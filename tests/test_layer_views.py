"""The layers on tensors that start anywhere in their storage: inputs, residuals, gradients and parameters that are
views at any element give, bit for bit, what copies of them give."""

import copy

import pytest
import torch

from fp8_delayed_scaling_quantize_b200.experts import Fp8Experts
from fp8_delayed_scaling_quantize_b200.linear import Fp8Linear, Fp8MLP

pytestmark = pytest.mark.gpu

T, D = 24, 64
KINDS = {
    "linear": (lambda: Fp8Linear(D, D, device="cuda"), False),
    "linear with activation": (lambda: Fp8Linear(D, D, device="cuda", activation="gelu"), True),
    "linear with residual": (lambda: Fp8Linear(D, D, device="cuda"), True),
    "mlp": (lambda: Fp8MLP(D, 2 * D, device="cuda"), True),
    "experts": (lambda: Fp8Experts(3, D, D, device="cuda", activation="silu"), False),
}


def _at(t, first):
    """t's values as a contiguous view that starts `first` elements into its storage."""
    flat = torch.empty(t.numel() + first, dtype=t.dtype, device=t.device)
    flat[first:].copy_(t.reshape(-1))
    return flat[first:].view(t.shape)


def _step(layer, x, r, off, g):
    """Output and gradients of one step whose incoming gradient is g as it is."""
    x = x.detach().requires_grad_(True)
    y = layer(x, off) if off is not None else layer(x) if r is None else layer(x, r)
    return [y.detach(), *torch.autograd.grad(y, [x, *layer.parameters()], g)]


@pytest.mark.parametrize("first", [0, 1, 4, 7])
@pytest.mark.parametrize("kind", list(KINDS))
def test_views_at_any_element(kind, first):
    make, residual = KINDS[kind]
    gen = torch.Generator("cuda").manual_seed(first)
    rand = lambda: torch.randn(T, D, device="cuda", generator=gen).bfloat16()  # noqa: E731
    a = make()
    b = make()
    b.load_state_dict(copy.deepcopy(a.state_dict()))
    off = torch.tensor([0, 5, 5, T], dtype=torch.int32, device="cuda") if kind == "experts" else None
    for moved in ("x", "residual", "g", "parameters"):
        if moved == "parameters":
            for p in b.parameters():
                p.data = _at(p.data, first)
        x, g, r = rand(), rand(), rand() if residual else None
        put = lambda t, name: _at(t, first) if moved == name and t is not None else t  # noqa: E731
        want = _step(a, x, r, off, g)
        got = _step(b, put(x, "x"), put(r, "residual"), off, put(g, "g"))
        for p, q in zip(want, got):
            assert torch.equal(p, q), moved
        assert torch.equal(a.fp8_rings, b.fp8_rings)


@pytest.mark.parametrize("kind", list(KINDS))
def test_an_output_joined_to_others(kind):
    """The gradient of torch.cat arrives as a view at the element where the output starts."""
    layer, _ = KINDS[kind][0](), None
    x = torch.randn(T, D, device="cuda").bfloat16()
    y = layer(x, torch.tensor([0, 5, 5, T], dtype=torch.int32, device="cuda")) if kind == "experts" else layer(x)
    head = torch.zeros(3, dtype=torch.bfloat16, device="cuda")
    torch.cat([head, y.flatten()]).mul(2).sum().backward()
    assert all(torch.isfinite(p.grad).all() for p in layer.parameters())
