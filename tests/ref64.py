"""Plain 64-bit forms of the epilogue, activation-gradient and expert products, and their error bounds.

The bounds, per output, from the number of roundings (half-steps: bf16 2^-8, E4M3 2^-4, E5M2 2^-3 of the value):
* z: the tensor core adds 32 products a step into fp32; K / 32 truncating additions of partial sums no larger than
  the absolute sum S err by at most K / 32 * 2^-23 S, which is 2^-16 S up to K = 4096, and the scale and bias add two
  fp32 roundings (2^-23 of |z| + |bias|);
* activation: slope at most 1.13; its own formula errs by at most 2^-20 max(1, |z|): ex2.approx and rcp.approx are
  good to 2^-22, the erf form to 2^-22.7 (1.5e-7), each multiplied by |z|, and what is cut off at |z| > 100 is below
  2^-100;
* the last rounding: half a step of the result.
"""

import math

import torch

F8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}
FMAX = {0: 448.0, 1: 57344.0}
HALF = {0: 2.0 ** -4, 1: 2.0 ** -3}      # half a step, relative
HALF_MIN = {0: 2.0 ** -10, 1: 2.0 ** -17}  # half the smallest subnormal
NONE, RELU, GELU, GELU_TANH, SILU = range(5)
C = math.sqrt(2 / math.pi)


def dec(codes, fmt):
    return codes.view(F8[fmt]).double()


def act(z, a):
    if a == RELU:
        return torch.where(z < 0, torch.zeros_like(z), z)
    if a == GELU:
        return z * torch.special.ndtr(z)
    if a == GELU_TANH:
        return z * torch.sigmoid(2 * C * (z + 0.044715 * z ** 3))
    if a == SILU:
        return z * torch.sigmoid(z)
    return z


def slope(z, a):
    """act'(z), written from the formulas."""
    if a == RELU:
        return (z > 0).double()
    if a == GELU:
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if a == GELU_TANH:
        t = torch.tanh(C * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * C * (1 + 3 * 0.044715 * z * z)
    if a == SILU:
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def op(a, b, layout):
    """[.., M, K] x [.., K, N] of the operands as stored."""
    if layout == 2:
        a = a.transpose(-1, -2)
    return a @ (b.transpose(-1, -2) if layout == 0 else b)


def z_and_bound(a, b, layout, inv, bias=None):
    """z in 64 bits and how far the kernel's fp32 z may be from it."""
    z = op(a, b, layout) * inv
    s = op(a.abs(), b.abs(), layout) * inv
    if bias is not None:
        z = z + bias
        s = s + bias.abs()
    return z, 2.0 ** -16 * s + 2.0 ** -22 * z.abs() + 2.0 ** -140


def y_and_bound(z, ez, a, residual=None):
    y = act(z, a)
    e = ez if a == NONE else 1.13 * ez + 2.0 ** -20 * z.abs().clamp(min=1.0)
    if residual is not None:
        y = y + residual
        e = e + 2.0 ** -23 * y.abs()
    return y, e


def check_bf16(got, want, err, what=""):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tol = err + 2.0 ** -8 * (want.abs() + err)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN in other places"
    assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), what + ": infinities"
    d = torch.where(fin, (got - want).abs(), torch.zeros_like(want))
    bad = d > torch.where(fin, tol, torch.zeros_like(tol) + 1.0)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((d / tol).nan_to_num().max()):.3g} x"


def check_codes(got, fmt, y, err, scale, what=""):
    """Codes against clamp(y * scale): half a step, and the error of y scaled."""
    t = (y * scale).clamp(-FMAX[fmt], FMAX[fmt])
    e = err * scale + 2.0 ** -23 * t.abs()
    tol = (HALF[fmt] * (t.abs() + e)).clamp(min=HALF_MIN[fmt]) + e
    d = (dec(got, fmt) - t).abs()
    assert d.shape == t.shape
    assert not (d > tol).any(), f"{what}: {int((d > tol).sum())} of {d.numel()} outside, worst {float((d / tol).max()):.3g} x"


def codes(gen, shape, fmt, std=None):
    std = FMAX[fmt] / 5.0 if std is None else std
    v = torch.randn(shape, generator=gen, device="cuda") * std
    return v.clamp_(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8)


def bf16(gen, shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)
