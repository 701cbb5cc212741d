"""The layers keep an activation's input for the backward pass where its gradient is asked for, and nowhere else."""

import pytest
import torch

from fp8_delayed_scaling_quantize_b200 import experts, linear

pytestmark = pytest.mark.gpu


def _spy(monkeypatch, module, name, at):
    """Calls of module.name, each with whether its argument `at` (the kept input) was given."""
    kept, call = [], getattr(module, name)

    def spied(*args, **kwargs):
        kept.append(args[at] is not None)
        return call(*args, **kwargs)

    monkeypatch.setattr(module, name, spied)
    return kept


LEARN = {"all": ("x", "weight1", "bias1", "weight2", "bias2"), "the input": ("x",), "weight1": ("weight1",),
         "bias1": ("bias1",), "the second product": ("weight2", "bias2"), "nothing": ()}


@pytest.mark.parametrize("activation", [None, "relu", "silu"])
@pytest.mark.parametrize("learn", list(LEARN))
def test_mlp(monkeypatch, activation, learn):
    mlp, whole = (linear.Fp8MLP(64, 128, device="cuda", activation=activation) for _ in range(2))
    whole.load_state_dict(mlp.state_dict())
    gen = torch.Generator("cuda").manual_seed(2)
    x, g = (torch.randn(20, 64, device="cuda", generator=gen).bfloat16() for _ in range(2))
    for name, p in mlp.named_parameters():
        p.requires_grad_(name in LEARN[learn])
    kept = _spy(monkeypatch, linear, "fp8_mm_act_out8", 18)
    xs = x.clone().requires_grad_("x" in LEARN[learn])
    y = mlp(xs)
    first = learn not in ("the second product", "nothing")
    assert kept == [activation is not None and first]
    xw = x.clone().requires_grad_(True)
    yw = whole(xw)
    assert torch.equal(y, yw)
    yw.backward(g)
    if learn == "nothing":
        assert y.grad_fn is None
        return
    y.backward(g)
    for name, p, q in [("x", xs, xw), *((n, p, dict(whole.named_parameters())[n]) for n, p in mlp.named_parameters())]:
        assert (p.grad is not None) == (name in LEARN[learn])
        assert p.grad is None or torch.equal(p.grad, q.grad), name


def test_without_gradients_nothing_is_kept(monkeypatch):
    x = torch.randn(20, 64, device="cuda").bfloat16().requires_grad_(True)
    off = torch.tensor([0, 9, 20], dtype=torch.int32, device="cuda")
    kept = [_spy(monkeypatch, linear, "fp8_mm_act_out8", 18), _spy(monkeypatch, linear, "fp8_mm_act", 20),
            _spy(monkeypatch, experts, "fp8_mm_experts", 15)]
    layers = [(linear.Fp8MLP(64, 128, device="cuda"), ()), (linear.Fp8Linear(64, 64, device="cuda", activation="gelu"), ()),
              (experts.Fp8Experts(2, 64, 64, device="cuda", activation="gelu"), (off,))]
    for layer, more in layers:
        with torch.no_grad():
            y = layer(x, *more)
        assert y.grad_fn is None
    assert kept == [[False], [False, False], [False]]
    for layer, more in layers:
        layer(x, *more)
    assert kept == [[False, True], [False, False, False, True], [False, True]]
