"""The layers on the activation epilogue and the expert products: Fp8Linear with activation and residual, Fp8MLP,
Fp8Experts, and a mixture-of-experts block of them.

Every kernel below them has its own test against 64 bits; here a layer must give, bit for bit, what its documented
sequence of calls gives (same rings), and its gradients must point where fp32's do."""

import pytest
import torch

import fp8_delayed_scaling_quantize_b200 as fp8
import ref64 as R

pytestmark = pytest.mark.gpu

E4, E5 = 0, 1
NT, NN, TN = 0, 1, 2
CODE = {None: 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
FUN = {None: lambda z: z, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
       "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}


def _rings(n):
    r = torch.empty(n, 20, dtype=torch.int32, device="cuda")
    for i in range(n):
        fp8.fp8_ring_init(r[i], 1.0)
    return r


def _q(t, fmt, ring):
    q, f = torch.empty(t.numel(), dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
    fp8.fp8_quantize(t, t.numel(), fmt, ring, q, f[0:1], f[1:2])
    return q, f[1:2]


def _grad(g, z, act, ring, off=None):
    T, N = g.shape
    q, f = torch.empty(T * N, dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
    if off is None:
        db = torch.empty(N, dtype=torch.bfloat16, device="cuda")
        fp8.fp8_act_grad(g, z, T, N, act, E5, ring, 0, q, f[0:1], f[1:2], db)
    else:
        db = torch.empty(len(off) - 1, N, dtype=torch.bfloat16, device="cuda")
        fp8.fp8_act_grad_experts(g, z, T, N, len(off) - 1, off, act, E5, ring, 0, q, f[0:1], f[1:2], db)
    return q, f[1:2], db


def _mm(a, fa, sa, b, fb, sb, layout, M, N, K):
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_mm(a, fa, b, fb, sa, sb, layout, M, N, K, 1, 0, 0, 0, None, None, 0, out)
    return out


def _same(a, b, what=""):
    assert a.shape == b.shape and torch.equal(a.view(torch.int16), b.contiguous().view(torch.int16)), what


def _cos(a, b):
    a, b = a.detach().double().reshape(-1), b.detach().double().reshape(-1)
    return float(a @ b / a.norm() / b.norm())


@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T,K,N,bias,residual", [(1, 64, 32, True, False), (24, 128, 256, False, True),
                                                 (200, 256, 192, True, True), (513, 144, 272, True, False)])
def test_linear_with_activation_and_residual(act, T, K, N, bias, residual):
    from fp8_delayed_scaling_quantize_b200.linear import Fp8Linear
    if act is None and not residual:
        residual = True  # without either it is the plain layer, tested elsewhere
    layer = Fp8Linear(K, N, bias=bias, device="cuda", activation=act)
    gen = R.gen(T + N)
    with torch.no_grad():
        layer.weight.copy_(R.bf16(gen, (N, K), 0.5))
        if bias:
            layer.bias.copy_(R.bf16(gen, (N,), 0.3))
    rings, a = _rings(3), CODE[act]
    for step, f in enumerate((1.0, 4.0)):  # the second step under the scales that the first published
        x = R.bf16(gen, (T, K), f).requires_grad_(True)
        r = R.bf16(gen, (T, N), 1.0).requires_grad_(True) if residual else None
        g = R.bf16(gen, (T, N), 0.1 * f)
        for p in (layer.weight, layer.bias):
            if p is not None:
                p.grad = None
        y = layer(x, r)
        y.backward(g)
        with torch.no_grad():
            x8, sx = _q(x.detach(), E4, rings[0])
            w8, sw = _q(layer.weight.detach(), E4, rings[1])
            z, want = (torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            fp8.fp8_mm_act(x8, E4, w8, E4, sx, sw, NT, T, N, K, 1, 0, 0, 0, layer.bias, None, 0, a, r, 0, z, want)
            _same(y.detach(), want)
            inv = 1.0 / (sx.double() * sw.double())
            z64, ez = R.z_and_bound(R.dec(x8, E4).view(T, K), R.dec(w8, E4).view(N, K), NT, inv,
                                    layer.bias.double() if bias else None)
            R.check_bf16(y, *R.y_and_bound(z64, ez, a, r.double() if residual else None), f"step {step}")
            g8, sg, db = _grad(g, z if a else None, a, rings[2])
            _same(x.grad, _mm(g8, E5, sg, w8, E4, sw, NN, T, K, N), "dX")
            _same(layer.weight.grad, _mm(g8, E5, sg, x8, E4, sx, TN, N, K, T), "dW")
            if bias:
                _same(layer.bias.grad, db, "db")
            if residual:
                _same(r.grad, g, "residual")
        assert torch.equal(layer.fp8_rings, rings)


@pytest.mark.parametrize("act,shape,D,H,bias,residual", [("gelu_tanh", (300,), 128, 512, True, True),
                                                         ("silu", (2, 17), 64, 80, False, True),
                                                         ("relu", (1,), 256, 1024, True, False)])
def test_mlp_is_its_calls(act, shape, D, H, bias, residual):
    from fp8_delayed_scaling_quantize_b200.linear import Fp8MLP
    mlp = Fp8MLP(D, H, bias=bias, device="cuda", activation=act)
    gen = R.gen(D)
    if bias:
        with torch.no_grad():
            mlp.bias1.copy_(R.bf16(gen, (H,), 0.2))
            mlp.bias2.copy_(R.bf16(gen, (D,), 0.2))
    rings, a = _rings(6), CODE[act]
    T = int(torch.tensor(shape).prod())
    for f in (1.0, 0.3, 2.0):
        x = R.bf16(gen, (*shape, D), f).requires_grad_(True)
        g = R.bf16(gen, (*shape, D), 1e-2 * f)
        for p in mlp.parameters():
            p.grad = None
        y = mlp(x, x if residual else None)
        y.backward(g)
        with torch.no_grad():
            x2, g2 = x.detach().view(T, D), g.view(T, D)
            x8, sx = _q(x2, E4, rings[0])
            w1, s1 = _q(mlp.weight1.detach(), E4, rings[1])
            w2, s2 = _q(mlp.weight2.detach(), E4, rings[3])
            z, h8 = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T * H, dtype=torch.uint8, device="cuda")
            st, want = torch.empty(2, device="cuda"), torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
            fp8.fp8_mm_act_out8(x8, E4, w1, E4, sx, s1, NT, T, H, D, 1, 0, 0, 0, mlp.bias1, None, 0, a, z, E4, rings[2], h8,
                                st[0:1], st[1:2])
            fp8.fp8_mm_act(h8, E4, w2, E4, st[1:2], s2, NT, T, D, H, 1, 0, 0, 0, mlp.bias2, None, 0, 0,
                           x2 if residual else None, 0, None, want)
            _same(y.detach().view(T, D), want)
            g8, sg, db2 = _grad(g2, None, 0, rings[4])
            dh = _mm(g8, E5, sg, w2, E4, s2, NN, T, H, D)
            _same(mlp.weight2.grad, _mm(g8, E5, sg, h8, E4, st[1:2], TN, D, H, T), "dW2")
            z8, sz, db1 = _grad(dh, z, a, rings[5])
            _same(mlp.weight1.grad, _mm(z8, E5, sz, x8, E4, sx, TN, H, D, T), "dW1")
            dx = _mm(z8, E5, sz, w1, E4, s1, NN, T, D, H)
            if residual:  # autograd's sum of the two uses of x
                dx = dx + g2
            _same(x.grad.view(T, D), dx, "dX")
            if bias:
                _same(mlp.bias2.grad, db2, "db2")
                _same(mlp.bias1.grad, db1, "db1")
        assert torch.equal(mlp.fp8_rings, rings)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_mlp_gradients_point_with_fp32(act):
    """Relative rms errors: E4M3 operands 0.026 each, E5M2 0.053. The first weight's gradient takes g, W2, dz and x:
    sqrt(2 * 0.053^2 + 2 * 0.026^2) = 0.084, a cosine of 1 / sqrt(1 + 0.084^2) = 0.9965; 0.99 leaves room for the slope's
    change. ReLU's slope jumps: z is off by sqrt(2) * 0.026 = 0.037 of its deviation, so a share of 0.037 / pi = 0.0118
    of the values changes sign and is wrong by all of itself, which adds 0.0118 / 0.5 to the squared error:
    1 / sqrt(1 + 0.0071 + 0.0236) = 0.985. Hence 0.98 for ReLU."""
    least = 0.98 if act == "relu" else 0.99
    from fp8_delayed_scaling_quantize_b200.linear import Fp8MLP
    D, H, T = 256, 1024, 400
    mlp = Fp8MLP(D, H, device="cuda", activation=act)
    gen = R.gen(3)
    x, g = R.bf16(gen, (T, D)).requires_grad_(True), R.bf16(gen, (T, D))
    for _ in range(2):  # the second step uses published scales
        x.grad = None
        for p in mlp.parameters():
            p.grad = None
        y = mlp(x, x)
        y.backward(g)
    ref = [p.detach().float().requires_grad_(True) for p in (x, mlp.weight1, mlp.bias1, mlp.weight2, mlp.bias2)]
    yr = FUN[act](ref[0] @ ref[1].t() + ref[2]) @ ref[3].t() + ref[4] + ref[0]
    yr.backward(g.float())
    assert _cos(y, yr) > 0.995
    for p, q in zip((x, mlp.weight1, mlp.bias1, mlp.weight2, mlp.bias2), ref):
        assert _cos(p.grad, q.grad) > least


def test_mlp_parts_frozen_empty_batch_and_state_dict():
    from fp8_delayed_scaling_quantize_b200.linear import Fp8Linear, Fp8MLP
    mlp = Fp8MLP(64, 128, device="cuda")
    x = R.bf16(R.gen(1), (40, 64))
    with torch.no_grad():
        y0 = mlp(x)
    assert y0.grad_fn is None
    mlp.weight1.requires_grad_(False)
    mlp.bias1.requires_grad_(False)
    mlp(x).sum().backward()  # only the second linear learns
    assert mlp.weight1.grad is None and mlp.bias1.grad is None and mlp.weight2.grad is not None
    other = Fp8MLP(64, 128, device="cuda")
    other.load_state_dict(mlp.state_dict())
    assert torch.equal(other.fp8_rings, mlp.fp8_rings)
    _same(other(x).detach(), mlp(x).detach())
    lin = Fp8Linear(64, 32, device="cuda", activation="silu")
    for layer, width in ((other, 64), (lin, 32)):
        e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
        out = layer(e)
        assert out.shape == (0, width)
        out.sum().backward()
        assert e.grad.shape == (0, 64) and all((p.grad == 0).all() for p in layer.parameters())


@pytest.mark.parametrize("act,counts,K,N,bias", [("silu", [40, 0, 300, 7], 128, 192, True), (None, [3, 1, 0, 2], 64, 256, True),
                                                 ("gelu", [0, 0, 500], 80, 144, False)])
def test_experts_are_their_calls(act, counts, K, N, bias):
    from fp8_delayed_scaling_quantize_b200.experts import Fp8Experts
    E, behind = len(counts), 5
    layer = Fp8Experts(E, K, N, bias=bias, device="cuda", activation=act)
    gen = R.gen(K)
    if bias:
        with torch.no_grad():
            layer.bias.copy_(R.bf16(gen, (E, N), 0.3))
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    T, n = int(off[-1]) + behind, int(off[-1])
    rings, a = _rings(3), CODE[act]
    for f in (1.0, 3.0):
        x = R.bf16(gen, (T, K), f).requires_grad_(True)
        g = R.bf16(gen, (T, N), 1e-2 * f)
        layer.weight.grad = None
        if bias:
            layer.bias.grad = None
        y = layer(x, off)
        y.backward(g)
        with torch.no_grad():
            x8, sx = _q(x.detach(), E4, rings[0])
            w8, sw = _q(layer.weight.detach(), E4, rings[1])
            z, want = (torch.zeros(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            fp8.fp8_mm_experts(x8, E4, w8, E4, sx, sw, 0, NT, T, N, K, E, off, layer.bias, a, z, want)
            _same(y.detach(), want)
            assert (y[n:] == 0).all()
            g8, sg, db = _grad(g, z, a, rings[2], off)
            dx, dw = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda"), torch.empty_like(layer.weight)
            fp8.fp8_mm_experts(g8, E5, w8, E4, sg, sw, 0, NN, T, K, N, E, off, None, 0, None, dx)
            fp8.fp8_mm_experts(g8, E5, x8, E4, sg, sx, 0, TN, N, K, T, E, off, None, 0, None, dw)
            _same(x.grad, dx, "dX")
            _same(layer.weight.grad, dw, "dW")
            if bias:
                _same(layer.bias.grad, db, "db")
            assert (x.grad[n:] == 0).all()
        assert torch.equal(layer.fp8_rings, rings)


def test_experts_empty_batch_no_grad_and_state_dict():
    from fp8_delayed_scaling_quantize_b200.experts import Fp8Experts
    a = Fp8Experts(3, 64, 32, device="cuda", activation="relu")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    a(e, off).sum().backward()
    assert e.grad.shape == (0, 64) and all((p.grad == 0).all() for p in a.parameters())
    x = R.bf16(R.gen(2), (30, 64))
    off.copy_(torch.tensor([0, 10, 10, 30], dtype=torch.int32))
    with torch.no_grad():
        y = a(x, off)
    assert y.grad_fn is None
    b = Fp8Experts(3, 64, 32, device="cuda", activation="relu")
    b.load_state_dict(a.state_dict())
    _same(a(x, off).detach(), b(x, off).detach())


def test_a_second_derivative_is_refused():
    from fp8_delayed_scaling_quantize_b200.linear import Fp8MLP
    mlp = Fp8MLP(64, 64, device="cuda")
    x = R.bf16(R.gen(2), (8, 64)).requires_grad_(True)
    (dx,) = torch.autograd.grad(mlp(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


def _route(x, router, top):
    """Token-sorted copies for the top experts of each token: (rows, offsets, source token, gate)."""
    p, e = torch.softmax(x.float() @ router, -1).topk(top, -1)
    order = torch.argsort(e.reshape(-1), stable=True)
    counts = torch.bincount(e.reshape(-1), minlength=router.shape[1])
    off = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
    token = order // top
    return x[token], off, token, p.reshape(-1)[order]


def test_mixture_of_experts_block_trains_with_fp32():
    """Router, two expert products with SiLU between, gates and the sum over a token's experts: two optimiser steps;
    in the second, outputs and every gradient against the same block in fp32."""
    from fp8_delayed_scaling_quantize_b200.experts import Fp8Experts
    D, H, E, T, top = 128, 256, 8, 300, 2
    gen = R.gen(5)
    up, down = Fp8Experts(E, D, H, device="cuda", activation="silu"), Fp8Experts(E, H, D, device="cuda")
    router = torch.randn(D, E, generator=gen, device="cuda") * 0.3
    x, g = R.bf16(gen, (T, D)), R.bf16(gen, (T, D))
    opt = torch.optim.SGD([*up.parameters(), *down.parameters()], lr=1e-3)
    rows, off, token, gate = _route(x, router, top)
    for _ in range(2):
        opt.step()  # the first without gradients: nothing changes
        opt.zero_grad()
        xr = rows.clone().requires_grad_(True)
        h = down(up(xr, off), off)
        y = torch.zeros(T, D, device="cuda").index_add(0, token, h.float() * gate[:, None])
        y.backward(g.float())
    params = [up.weight, up.bias, down.weight, down.bias]
    ref = [p.detach().float().requires_grad_(True) for p in params]
    xf = rows.float().requires_grad_(True)
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), (off[1:] - off[:-1]).long())
    hf = FUN["silu"](torch.einsum("tk,tnk->tn", xf, ref[0][e]) + ref[1][e])
    hf = torch.einsum("tk,tnk->tn", hf, ref[2][e]) + ref[3][e]
    yf = torch.zeros(T, D, device="cuda").index_add(0, token, hf * gate[:, None])
    yf.backward(g.float())
    assert _cos(y, yf) > 0.995 and _cos(xr.grad, xf.grad) > 0.99
    for p, q in zip(params, ref):
        assert _cos(p.grad, q.grad) > 0.99


def test_an_expert_step_is_captured_and_follows_its_routing():
    """Forward and backward in one CUDA graph, replayed with other offsets and inputs: what an eager layer with the
    same rings gives. No eager autograd graph of the captured layer lives at capture."""
    from fp8_delayed_scaling_quantize_b200.experts import Fp8Experts
    E, K, N, T = 4, 64, 128, 96
    a, b = (Fp8Experts(E, K, N, device="cuda", activation="silu") for _ in range(2))
    gen = R.gen(6)
    x, g = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    a.reset_scaling()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(a(x, off), [a.weight, a.bias], g)
    torch.cuda.current_stream().wait_stream(side)
    b.load_state_dict(a.state_dict())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = a(x, off)
        grads = torch.autograd.grad(y, [a.weight, a.bias], g)
    for counts in ([10, 20, 30, 36], [0, 96, 0, 0], [1, 2, 3, 4]):
        x.copy_(R.bf16(gen, (T, K)))
        g.copy_(R.bf16(gen, (T, N)))
        off.copy_(torch.tensor([0] + counts).cumsum(0).to(torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = b(x, off)
        dw, db = torch.autograd.grad(want, [b.weight, b.bias], g)
        _same(y.detach(), want.detach())
        _same(grads[0], dw)
        _same(grads[1], db)
        assert torch.equal(a.fp8_rings, b.fp8_rings)


def test_refusals():
    from fp8_delayed_scaling_quantize_b200.experts import Fp8Experts
    from fp8_delayed_scaling_quantize_b200.linear import Fp8Linear, Fp8MLP
    for make in (lambda: Fp8Linear(64, 32, device="cuda", activation="tanh"), lambda: Fp8MLP(64, 40, device="cuda"),
                 lambda: Fp8Experts(4, 20, 32, device="cuda"), lambda: Fp8MLP(64, 64, device="cuda", activation="swiglu")):
        with pytest.raises(ValueError):
            make()
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    lin, ex = Fp8Linear(64, 32, device="cuda", activation="relu"), Fp8Experts(4, 64, 32, device="cuda")
    for call in (lambda: lin(x[:, :32]), lambda: lin(x, x), lambda: ex(x, off[:4]), lambda: ex(x, off.long()),
                 lambda: ex(x, off.cpu()), lambda: ex(x.view(2, 4, 64), off)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lin(x.float()), lambda: lin(x, torch.zeros(8, 32, device="cuda")), lambda: ex(x.float(), off)):
        with pytest.raises(TypeError):
            call()
