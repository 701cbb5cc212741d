"""FP8 training linear layer on the fp8lite C ABI (torch.autograd).

After the AstrAI commit logs (``astrai/extension/fp8.py`` @4dc5e923 and
@f4c44ebf):

* a linear layer owns three delayed-scaling rings, for x, W and the output
  gradient g (bullet on the three _ScaleRing objects per linear);
* forward quantizes x and W to E4M3 and computes y = x W^T (+ bias fused in
  the GEMM epilogue); backward quantizes g to E5M2 and computes dX = g W and
  dW = g^T x with the scales the forward used (bullets on carrying the
  forward's scale to backward and on the scale snapshot);
* backward reads only what forward saved, so it runs in FP8 wherever it is
  called (bullet on the autograd Function owning the forward/backward pair);
* gradients are bf16; the bias gradient is the column sum of the bf16 g over
  the flattened leading dimensions, computed only when the bias needs a
  gradient (bullets on the conditional column sum and the 3-D backward).

Every computation runs in the library's CUDA kernels; torch provides the
buffers and the stream. The forward saves the FP8 codes of x and W (one byte
per element) rather than the bf16 tensors. The rings are a registered buffer
(`fp8_rings`, three 80-byte rings), so they travel with the module's
state_dict for checkpoint and resume.

With an activation or a residual the same layer runs through the GEMM's
activation epilogue, y = act(x W^T + b) + residual in one launch, and its
backward pass quantizes the gradient through the activation, with the bias
gradient, in one pass (`Fp8LinearActFunction`). `Fp8MLP` is two such linears
whose hidden activation leaves the first product as FP8 codes: no bf16 hidden
tensor and no quantize pass of it in the forward.

The layers can be captured into a CUDA graph, forward and backward. As for any
torch module, no eager autograd graph of the same parameters may live at that
time (an output that was kept, say): its leaves are bound to the eager stream,
and torch would make that stream wait for the capture.
"""

import contextlib

import torch
from torch.autograd.function import once_differentiable

from . import (FP8_ACT_GELU, FP8_ACT_GELU_TANH, FP8_ACT_NONE, FP8_ACT_RELU, FP8_ACT_SILU, FP8_E4M3, FP8_E5M2, FP8_NN,
               FP8_NT, FP8_RING_BYTES, FP8_RING_HISTORY, FP8_TN, fp8_act_grad, fp8_bias_grad, fp8_mm, fp8_mm_act,
               fp8_mm_act_out8, fp8_mm_grouped, fp8_quantize, fp8_quantize_many, fp8_ring_init)

_RING_WORDS = FP8_RING_BYTES // 4
_SCALE_ONE = 0x3F800000  # the bits of 1.0f

ACTIVATIONS = {None: FP8_ACT_NONE, "relu": FP8_ACT_RELU, "gelu": FP8_ACT_GELU, "gelu_tanh": FP8_ACT_GELU_TANH,
               "silu": FP8_ACT_SILU}


def _act_code(activation):
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is none of {sorted(a for a in ACTIVATIONS if a)}")
    return ACTIVATIONS[activation]


def _dense(t):
    """t contiguous and from a 16-byte boundary on, as the kernels load it: a view that starts elsewhere is copied."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _rows_of(x, features, what):
    """x as dense rows [T, features]."""
    if x.shape[-1] != features:
        raise ValueError(f"{what} features {x.shape[-1]} != {features}")
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{what} must be bf16")
    return _dense(x.reshape(-1, features))


_HERE = contextlib.nullcontext()
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on_input(x, rings, *params):
    """What the kernels take by address: bf16 parameters and the rings on the input's GPU. Returns a context in which
    that GPU is current: the launches go to the current device's stream."""
    for t in params:
        if t is not None and t.dtype is not torch.bfloat16:
            raise TypeError("parameters and residual must be bf16")
    dev = x.get_device()
    if dev < 0:
        raise ValueError("the input must be on a GPU")
    for t in (rings, *params):
        if t is not None and t.get_device() != dev:
            raise ValueError(f"parameters and rings must be on the input's device {x.device}")
    # a device context costs 3 us, asking for the current device a tenth of that
    return _HERE if dev == _current_device() else torch.cuda.device(dev)


def _quantize(t, n, fmt, ring):
    q = torch.empty(n, dtype=torch.uint8, device=t.device)
    amax = torch.empty(1, dtype=torch.float32, device=t.device)
    scale = torch.empty(1, dtype=torch.float32, device=t.device)
    fp8_quantize(t, n, fmt, ring, q, amax, scale)
    return q, scale


class Fp8LinearFunction(torch.autograd.Function):
    """y = x W^T + b with FP8 operands and delayed scaling (three rings)."""

    @staticmethod
    def forward(ctx, x, weight, bias, rings):
        N, K = weight.shape
        if x.shape[-1] != K:
            raise ValueError(f"input features {x.shape[-1]} != weight's {K}")
        if x.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
            raise TypeError("Fp8Linear takes bf16 inputs and weights")
        x2 = _dense(x.reshape(-1, K))
        w = _dense(weight)
        T = x2.shape[0]
        # x and W in one quantize launch (each with its own ring)
        dev = x.device
        x8 = torch.empty(T * K, dtype=torch.uint8, device=dev)
        w8 = torch.empty(N * K, dtype=torch.uint8, device=dev)
        stats = torch.empty(4, dtype=torch.float32, device=dev)  # amax x, amax W, scale x, scale W
        amax_x, amax_w, sx, sw = stats[0:1], stats[1:2], stats[2:3], stats[3:4]
        fp8_quantize_many([(x2, T * K, FP8_E4M3, rings[0], x8, amax_x, sx),
                           (w, N * K, FP8_E4M3, rings[1], w8, amax_w, sw)])
        y = torch.empty(T, N, dtype=torch.bfloat16, device=x.device)
        b = bias.contiguous() if bias is not None else None
        fp8_mm(x8, FP8_E4M3, w8, FP8_E4M3, sx, sw, FP8_NT, T, N, K, 1, 0, 0, 0, b, None, 0, y)
        ctx.save_for_backward(x8, w8, sx, sw, rings)
        ctx.dims = (T, N, K)
        ctx.x_shape = x.shape
        ctx.has_bias = bias is not None
        return y.reshape(*x.shape[:-1], N)

    @staticmethod
    def backward(ctx, gy):
        x8, w8, sx, sw, rings = ctx.saved_tensors
        T, N, K = ctx.dims
        need_x, need_w, need_b = ctx.needs_input_grad[0], ctx.needs_input_grad[1], ctx.needs_input_grad[2]
        g2 = _dense(gy.reshape(-1, N).to(torch.bfloat16))
        dx = dw = db = None
        if need_x or need_w:
            g8, sg = _quantize(g2, T * N, FP8_E5M2, rings[2])
            # dX = g W: A = g [T, N], B = W [N, K] (K-major rows of B are W's rows)
            # dW = g^T x: A = g [T, N] read MN-major, B = x [T, K]
            probs = []
            if need_x:
                dx = torch.empty(T, K, dtype=torch.bfloat16, device=gy.device)
                probs.append((g8, FP8_E5M2, w8, FP8_E4M3, sg, sw, FP8_NN, T, K, N, None, None, 0, dx))
            if need_w:
                dw = torch.empty(N, K, dtype=torch.bfloat16, device=gy.device)
                probs.append((g8, FP8_E5M2, x8, FP8_E4M3, sg, sx, FP8_TN, N, K, T, None, None, 0, dw))
            if len(probs) == 2:  # both read only g8: one launch shares the grid
                fp8_mm_grouped(probs)
            else:
                a8, fa, b8, fb, sa, sb, layout, M, Nn, Kk, _, _, _, out = probs[0]
                fp8_mm(a8, fa, b8, fb, sa, sb, layout, M, Nn, Kk, 1, 0, 0, 0, None, None, 0, out)
            if need_x:
                dx = dx.reshape(ctx.x_shape)
        if ctx.has_bias and need_b:
            db = torch.empty(N, dtype=torch.bfloat16, device=gy.device)
            fp8_bias_grad(g2, T, N, db)
        return dx, dw, db, None


def _quantize_many(jobs, device):
    """Delayed quantizes in one launch: jobs (tensor, fmt, ring) -> [(codes, scale)]."""
    stats = torch.empty(2 * len(jobs), dtype=torch.float32, device=device)
    out = [torch.empty(t.numel(), dtype=torch.uint8, device=device) for t, _, _ in jobs]
    fp8_quantize_many([(t if t.numel() else None, t.numel(), fmt, ring, q if t.numel() else None, stats[i:i + 1],
                        stats[len(jobs) + i:len(jobs) + i + 1])
                       for i, ((t, fmt, ring), q) in enumerate(zip(jobs, out))])
    return [(q, stats[len(jobs) + i:len(jobs) + i + 1]) for i, q in enumerate(out)]


def _grad_codes(g2, z, act, ring, need_bias):
    """E5M2 codes of g act'(z), their scale and the bias gradient, in one pass."""
    T, N = g2.shape
    g8 = torch.empty(T * N, dtype=torch.uint8, device=g2.device)
    stats = torch.empty(2, dtype=torch.float32, device=g2.device)
    db = torch.empty(N, dtype=torch.bfloat16, device=g2.device) if need_bias else None
    fp8_act_grad(g2, z, T, N, act, FP8_E5M2, ring, 0, g8, stats[0:1], stats[1:2], db)
    return g8, stats[1:2], db


def _dx_dw(g8, sg, w8, sw, x8, sx, T, N, K, need_x, need_w):
    """dX = g W and dW = g^T x from the codes; both in one grouped launch."""
    dx = torch.empty(T, K, dtype=torch.bfloat16, device=g8.device) if need_x else None
    dw = torch.empty(N, K, dtype=torch.bfloat16, device=g8.device) if need_w else None
    probs = []
    if need_x:
        probs.append((g8, FP8_E5M2, w8, FP8_E4M3, sg, sw, FP8_NN, T, K, N, None, None, 0, dx))
    if need_w:
        probs.append((g8, FP8_E5M2, x8, FP8_E4M3, sg, sx, FP8_TN, N, K, T, None, None, 0, dw))
    if probs:
        fp8_mm_grouped(probs)
    return dx, dw


class Fp8LinearActFunction(torch.autograd.Function):
    """y = act(x W^T + b) + residual with FP8 operands and delayed scaling.
    learn: whether gradients are recorded, which a Function cannot see for
    itself (under no_grad its needs_input_grad are those of the leaves); without
    them the activation's input is not kept."""

    @staticmethod
    def forward(ctx, x, weight, bias, rings, act, residual, learn=True):
        N, K = weight.shape
        x2 = _rows_of(x, K, "input")
        T = x2.shape[0]
        if weight.dtype != torch.bfloat16:
            raise TypeError("Fp8Linear takes bf16 inputs and weights")
        r2 = None
        if residual is not None:
            if residual.shape != (*x.shape[:-1], N):
                raise ValueError(f"residual shape {tuple(residual.shape)} != {(*x.shape[:-1], N)}")
            r2 = _rows_of(residual, N, "residual")
        dev = x.device
        (x8, sx), (w8, sw) = _quantize_many([(x2, FP8_E4M3, rings[0]), (_dense(weight), FP8_E4M3, rings[1])], dev)
        y = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
        z = None
        if act != FP8_ACT_NONE and learn and any(ctx.needs_input_grad[:3]):
            z = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
        b = bias.contiguous() if bias is not None else None
        if T:
            fp8_mm_act(x8, FP8_E4M3, w8, FP8_E4M3, sx, sw, FP8_NT, T, N, K, 1, 0, 0, 0, b, None, 0, act, r2, 0, z, y)
        ctx.save_for_backward(x8, w8, sx, sw, rings, z)
        ctx.dims, ctx.act, ctx.x_shape, ctx.has_bias = (T, N, K), act, x.shape, bias is not None
        return y.reshape(*x.shape[:-1], N)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        x8, w8, sx, sw, rings, z = ctx.saved_tensors
        T, N, K = ctx.dims
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        need_b = need_b and ctx.has_bias
        dx = dw = db = None
        if need_x or need_w or need_b:
            g2 = _dense(gy.reshape(-1, N).to(torch.bfloat16))
            g8, sg, db = _grad_codes(g2, z, ctx.act, rings[2], need_b)
            if T:
                dx, dw = _dx_dw(g8, sg, w8, sw, x8, sx, T, N, K, need_x, need_w)
            else:
                dx = torch.empty(T, K, dtype=torch.bfloat16, device=gy.device) if need_x else None
                dw = torch.zeros(N, K, dtype=torch.bfloat16, device=gy.device) if need_w else None
            if need_x:
                dx = dx.reshape(ctx.x_shape)
        return dx, dw, db, None, None, gy if ctx.needs_input_grad[5] else None, None


def _fresh_rings(count, device):
    """`count` rings as fp8_ring_init(ring, 1.0) leaves them."""
    rings = torch.zeros(count, _RING_WORDS, dtype=torch.int32, device=device)
    rings[:, FP8_RING_HISTORY] = _SCALE_ONE
    return rings


class Fp8Layer(torch.nn.Module):
    """A layer with delayed-scaling rings, which are ready for use from the start: the first forward launches no reset,
    so a graph may capture it."""

    RINGS = 3

    def _make_rings(self, device):
        self.register_buffer("fp8_rings", _fresh_rings(self.RINGS, device))
        self._rings_ready = not self.fp8_rings.is_meta  # a layer made without memory resets them in its first forward

    def reset_scaling(self):
        """Reset the rings (scale 1, empty history)."""
        for i in range(self.RINGS):
            fp8_ring_init(self.fp8_rings[i], 1.0)
        self._rings_ready = True

    def _load_from_state_dict(self, state_dict, prefix, *args, **kwargs):
        super()._load_from_state_dict(state_dict, prefix, *args, **kwargs)
        if prefix + "fp8_rings" not in state_dict:
            return  # weights alone: the rings stay as they are
        # Restored rings are used as they are, but for those without a scale (a scale of 0 makes every output NaN)
        with torch.no_grad():
            scale = self.fp8_rings[:, FP8_RING_HISTORY].contiguous().view(torch.float32)
            good = (scale > 0) & torch.isfinite(scale)
            self.fp8_rings.copy_(torch.where(good[:, None], self.fp8_rings,
                                             _fresh_rings(self.RINGS, self.fp8_rings.device)))
        self._rings_ready = not self.fp8_rings.is_meta


class Fp8Linear(Fp8Layer):
    """Drop-in training linear layer (bf16 parameters, FP8 compute).

    in_features and out_features must be multiples of 16 (the GEMMs read
    every operand through 16-byte-aligned rows). activation: None, "relu",
    "gelu", "gelu_tanh" or "silu", applied to the output in the GEMM's
    epilogue; forward(x, residual) adds a bf16 residual after it.
    """

    def __init__(self, in_features, out_features, bias=True, device=None, activation=None):
        super().__init__()
        self.activation = activation
        self._act = _act_code(activation)
        if in_features % 16 or out_features % 16:
            raise ValueError("Fp8Linear needs in_features and out_features divisible by 16")
        self.in_features, self.out_features = in_features, out_features
        kw = {"device": device, "dtype": torch.bfloat16}
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features, **kw))
        self.bias = torch.nn.Parameter(torch.zeros(out_features, **kw)) if bias else None
        self._make_rings(device)
        torch.nn.init.normal_(self.weight, std=in_features ** -0.5)

    def forward(self, x, residual=None):
        rings, weight, bias = self.fp8_rings, self.weight, self.bias
        with _on_input(x, rings, weight, bias, residual):
            if not self._rings_ready:
                self.reset_scaling()
            if self._act == FP8_ACT_NONE and residual is None:
                return Fp8LinearFunction.apply(x, weight, bias, rings)
            return Fp8LinearActFunction.apply(x, weight, bias, rings, self._act, residual, torch.is_grad_enabled())


class Fp8MLPFunction(torch.autograd.Function):
    """y = act(x W1^T + b1) W2^T + b2 + residual. The hidden activation goes
    from the first product to the second as E4M3 codes under its own ring; for
    the backward pass its input z is kept in bf16, where the activation's
    gradient is asked for. Rings: x, W1, hidden, W2, the
    gradients of the output and of z."""

    @staticmethod
    def forward(ctx, x, w1, b1, w2, b2, rings, act, residual, learn=True):
        H, D = w1.shape
        N = w2.shape[0]
        x2 = _rows_of(x, D, "input")
        T, dev = x2.shape[0], x.device
        r2 = None
        if residual is not None:
            if residual.shape != (*x.shape[:-1], N):
                raise ValueError(f"residual shape {tuple(residual.shape)} != {(*x.shape[:-1], N)}")
            r2 = _rows_of(residual, N, "residual")
        b1, b2 = (b.contiguous() if b is not None else None for b in (b1, b2))
        (x8, sx), (w18, sw1), (w28, sw2) = _quantize_many(
            [(x2, FP8_E4M3, rings[0]), (_dense(w1), FP8_E4M3, rings[1]), (_dense(w2), FP8_E4M3, rings[3])], dev)
        z = None
        if act != FP8_ACT_NONE and learn and any(ctx.needs_input_grad[:3]):  # what the first product's gradients read
            z = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        h8 = torch.empty(T * H, dtype=torch.uint8, device=dev)
        stats = torch.empty(2, dtype=torch.float32, device=dev)
        sh = stats[1:2]
        y = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
        if T:
            fp8_mm_act_out8(x8, FP8_E4M3, w18, FP8_E4M3, sx, sw1, FP8_NT, T, H, D, 1, 0, 0, 0, b1, None, 0, act, z,
                            FP8_E4M3, rings[2], h8, stats[0:1], sh)
            fp8_mm_act(h8, FP8_E4M3, w28, FP8_E4M3, sh, sw2, FP8_NT, T, N, H, 1, 0, 0, 0, b2, None, 0, FP8_ACT_NONE, r2,
                       0, None, y)
        ctx.save_for_backward(x8, w18, h8, w28, sx, sw1, sh, sw2, rings, z)
        ctx.dims, ctx.act, ctx.x_shape = (T, D, H, N), act, x.shape
        return y.reshape(*x.shape[:-1], N)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        x8, w18, h8, w28, sx, sw1, sh, sw2, rings, z = ctx.saved_tensors
        T, D, H, N = ctx.dims
        need_x, need_w1, need_b1, need_w2, need_b2 = ctx.needs_input_grad[:5]
        dx = dw1 = db1 = dw2 = db2 = None
        inner = need_x or need_w1 or need_b1
        if T and (inner or need_w2 or need_b2):
            g2 = _dense(gy.reshape(-1, N).to(torch.bfloat16))
            g8, sg, db2 = _grad_codes(g2, None, FP8_ACT_NONE, rings[4], need_b2)
            dh, dw2 = _dx_dw(g8, sg, w28, sw2, h8, sh, T, N, H, inner, need_w2)
            if inner:
                z8, sz, db1 = _grad_codes(dh, z, ctx.act, rings[5], need_b1)
                dx, dw1 = _dx_dw(z8, sz, w18, sw1, x8, sx, T, H, D, need_x, need_w1)
            if need_x:
                dx = dx.reshape(ctx.x_shape)
        elif not T:
            zero = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=gy.device)  # noqa: E731
            dx = zero(*ctx.x_shape) if need_x else None
            dw1, db1 = zero(H, D) if need_w1 else None, zero(H) if need_b1 else None
            dw2, db2 = zero(N, H) if need_w2 else None, zero(N) if need_b2 else None
        return dx, dw1, db1, dw2, db2, None, None, gy if ctx.needs_input_grad[7] else None, None


class Fp8MLP(Fp8Layer):
    """Two FP8 linears with an activation between (bf16 parameters).

    features and hidden must be multiples of 16. forward(x, residual) adds a
    bf16 residual (often x itself) in the second product's epilogue.
    """

    RINGS = 6

    def __init__(self, features, hidden, bias=True, device=None, activation="gelu_tanh"):
        super().__init__()
        if features % 16 or hidden % 16:
            raise ValueError("Fp8MLP needs features and hidden divisible by 16")
        self.features, self.hidden, self.activation = features, hidden, activation
        self._act = _act_code(activation)
        kw = {"device": device, "dtype": torch.bfloat16}
        self.weight1 = torch.nn.Parameter(torch.empty(hidden, features, **kw))
        self.weight2 = torch.nn.Parameter(torch.empty(features, hidden, **kw))
        self.bias1 = torch.nn.Parameter(torch.zeros(hidden, **kw)) if bias else None
        self.bias2 = torch.nn.Parameter(torch.zeros(features, **kw)) if bias else None
        self._make_rings(device)
        torch.nn.init.normal_(self.weight1, std=features ** -0.5)
        torch.nn.init.normal_(self.weight2, std=hidden ** -0.5)

    def forward(self, x, residual=None):
        rings, params = self.fp8_rings, (self.weight1, self.bias1, self.weight2, self.bias2)
        with _on_input(x, rings, *params, residual):
            if not self._rings_ready:
                self.reset_scaling()
            return Fp8MLPFunction.apply(x, *params, rings, self._act, residual, torch.is_grad_enabled())
