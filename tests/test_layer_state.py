"""The layers' rings as their state is made, saved and loaded: every ring has a scale before the first forward,
whatever a checkpoint holds."""

import copy

import pytest
import torch

import fp8_delayed_scaling_quantize_b200 as fp8
from fp8_delayed_scaling_quantize_b200.experts import Fp8Experts
from fp8_delayed_scaling_quantize_b200.linear import Fp8Linear, Fp8MLP

SCALE = fp8.FP8_RING_HISTORY  # the scale's word of a ring
KINDS = ("linear", "linear with activation", "mlp", "experts")


def _layer(kind, device="cpu"):
    if kind == "mlp":
        return Fp8MLP(64, 64, device=device)
    if kind == "experts":
        return Fp8Experts(2, 64, 64, device=device)
    return Fp8Linear(64, 64, device=device, activation="silu" if kind != "linear" else None)


def _is_fresh(rings):
    want = torch.zeros_like(rings)
    want[:, SCALE] = torch.tensor([1.0]).view(torch.int32).item()
    return torch.equal(rings, want)


def _in_use(rings):
    """Rings with a history: scale 2 + i, index 5."""
    rings = torch.zeros_like(rings)
    rings[:, SCALE] = (2.0 + torch.arange(len(rings), device=rings.device)).view(torch.int32)
    rings[:, SCALE + 1] = 5
    return rings


@pytest.mark.parametrize("kind", KINDS)
def test_rings_have_a_scale_from_the_start(kind):
    assert _is_fresh(_layer(kind).fp8_rings)


@pytest.mark.parametrize("assign", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_state_of_a_layer_that_never_ran(kind, assign):
    state = _layer(kind).state_dict()
    old = dict(state, fp8_rings=torch.zeros_like(state["fp8_rings"]))  # rings without a scale
    for s in (state, old):
        layer = _layer(kind)
        layer.load_state_dict(copy.deepcopy(s), assign=assign)
        assert _is_fresh(layer.fp8_rings)


@pytest.mark.parametrize("kind", KINDS)
def test_weights_alone_leave_the_rings(kind):
    layer = _layer(kind)
    weights = {k: v for k, v in layer.state_dict().items() if k != "fp8_rings"}
    layer.load_state_dict(weights, strict=False)
    assert _is_fresh(layer.fp8_rings)
    used = _in_use(layer.fp8_rings)
    layer.fp8_rings.copy_(used)
    layer.load_state_dict(weights, strict=False)
    assert torch.equal(layer.fp8_rings, used)


@pytest.mark.parametrize("kind", KINDS)
def test_rings_in_use_are_restored_and_lost_ones_are_not(kind):
    layer = _layer(kind)
    used = _in_use(layer.fp8_rings)
    layer.load_state_dict(dict(layer.state_dict(), fp8_rings=used))
    assert torch.equal(layer.fp8_rings, used)
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        state = used.clone()
        state[1, SCALE] = torch.tensor([bad]).view(torch.int32).item()
        layer.load_state_dict(dict(layer.state_dict(), fp8_rings=state))
        assert _is_fresh(layer.fp8_rings[1:2])
        assert torch.equal(layer.fp8_rings[0], used[0]) and torch.equal(layer.fp8_rings[2:], used[2:])


@pytest.mark.parametrize("kind", KINDS)
def test_a_layer_inside_a_module_and_one_without_memory(kind):
    net = torch.nn.Sequential(torch.nn.Identity(), _layer(kind))
    net.load_state_dict({k: torch.zeros_like(v) for k, v in net.state_dict().items()})
    assert _is_fresh(net[1].fp8_rings)
    layer = _layer(kind, "meta")
    assert not layer._rings_ready  # its first forward resets them
    layer.load_state_dict(_layer(kind).state_dict(), assign=True)
    assert layer._rings_ready and _is_fresh(layer.fp8_rings)


def _run(layer, kind, x, off):
    return layer(x, off) if kind == "experts" else layer(x)


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["never ran", "weights alone", "without a scale", "without memory"])
@pytest.mark.parametrize("kind", KINDS)
def test_first_step_after_loading(kind, how):
    """Outputs and gradients of the first step are those of the layer that the weights came from."""
    a = _layer(kind, "cuda")
    state = copy.deepcopy(a.state_dict())
    b = _layer(kind, "meta").to_empty(device="cuda") if how == "without memory" else _layer(kind, "cuda")
    if how in ("weights alone", "without memory"):
        del state["fp8_rings"]
    if how == "without a scale":
        state["fp8_rings"].zero_()
    b.load_state_dict(state, strict=how in ("never ran", "without a scale"))
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    x = torch.randn(8, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    g = torch.ones_like(x)
    ya, yb = _run(a, kind, x, off), _run(b, kind, x, off)
    assert torch.isfinite(yb).all() and torch.equal(ya, yb)
    for p, q in zip(torch.autograd.grad(ya, list(a.parameters()), g), torch.autograd.grad(yb, list(b.parameters()), g)):
        assert torch.isfinite(q).all() and torch.equal(p, q)
    assert torch.equal(a.fp8_rings, b.fp8_rings)
    a.reset_scaling()
    assert _is_fresh(a.fp8_rings)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_a_first_forward_in_a_graph_keeps_its_history(kind):
    """Replays of a layer's first forward fold one amax each: the graph holds no reset of the rings."""
    a, b = _layer(kind, "cuda"), _layer(kind, "cuda")
    b.load_state_dict(a.state_dict())
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    with torch.no_grad():
        _run(_layer(kind, "cuda"), kind, x, off)  # the kernels are loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(graph):
        y = _run(a, kind, x, off)
    for step in range(3):
        x.copy_(torch.randn(8, 64, device="cuda") * 2.0 ** step)
        graph.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            assert torch.equal(y, _run(b, kind, x, off))
        assert torch.equal(a.fp8_rings, b.fp8_rings) and fp8.fp8_ring_get(a.fp8_rings[0]).idx == step + 1
