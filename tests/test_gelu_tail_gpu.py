"""GELU (erf) and its slope over every bf16 input, to the precision of their bf16 rounding far into the tail.

Bounds, x = |z|. Forward: Phi(-x) errs by at most E = min(2^-21, 2^-13 Phi(-x)): the fit by the smaller of 6e-8 and
1e-4 of it, a sum of seven terms below 1.2, rcp.approx and the last products by less than 2^-22 altogether, and
ex2.approx(-0.72 x^2) by a relative 2^-22 + 3 x^2 2^-25 (three roundings of its argument), which is 2^-16 at x = 13.
Slope: 7.1.26 errs by 7.5e-8 absolutely and, up to x = 13.3, where the exponential ends, by 0.04 Phi(-x) relatively:
E = min(2^-21, 2^-4 Phi(-x)). It adds z phi(z), whose exponential has a relative error of 2^-20 + x^2 2^-23 with its
products. The stored value adds half a step, 2^-8 of it. An exponential below 2^-126 is flushed, which it is from
x = 13.22 on (x^2 / 2 = 126 ln 2). In Phi a factor of P(t) = 0.03 stands on it and |z| = 13.22 in the product:
0.4 * 2^-126, below 2^-125. In the slope z / sqrt(2 pi) = 5.28 does: 5.28 * 2^-126, below 2^-123, and falling with x."""

import math

import pytest
import torch

import fp8_delayed_scaling_quantize_b200 as fp8
import ref64 as R

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


def _inputs():
    bits = torch.arange(0, 65536, dtype=torch.int32).to(torch.int16).cuda().view(torch.bfloat16)
    z = bits[torch.isfinite(bits)]
    return z[: z.numel() // 16 * 16].contiguous()


def _lower(x):
    """Phi(-x) in 64 bits without cancellation."""
    return 0.5 * torch.special.erfc(x / math.sqrt(2))


def _phi(z, tail):
    """Phi(z) and the kernel's error bound of it, `tail` of Phi(-|z|) at most."""
    x = z.abs()
    low = _lower(x)
    return torch.where(z < 0, low, 1 - low), torch.minimum(torch.full_like(x, 2.0 ** -21), tail * low)


def _check(got, want, err, flushed, z):
    tol = err + HALF * (want.abs() + err) + flushed
    d = (got.double() - want).abs() / tol
    assert torch.isfinite(got).all()
    assert float(d.max()) <= 1.0, f"{float(d.max()):.3g} x at z = {float(z[d.argmax()])}"


@pytest.mark.parametrize("M", [1, 64])
def test_forward(M):
    """z enters as the bias of a product of zeros: few rows run swapped, more by tiles."""
    z = _inputs()
    N = z.numel()
    a, b = torch.zeros(M, 16, dtype=torch.uint8, device="cuda"), torch.zeros(N, 16, dtype=torch.uint8, device="cuda")
    one, out = torch.ones(1, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_mm_act(a, 0, b, 0, one, one, 0, M, N, 16, 1, 0, 0, 0, z, None, 0, R.GELU, None, 0, None, out)
    z64 = z.double()
    phi, e = _phi(z64, 2.0 ** -13)
    for row in (0, M - 1):
        # past 1e38 the product z Phi(z) is z itself
        _check(out[row], z64 * phi, z64.abs() * (e + torch.where(z64 > 0, 2.0 ** -23, 0.0)), 2.0 ** -125, z)


def test_slope():
    """One row with g = 1: the bias gradient is the slope in bf16."""
    z = _inputs()
    n = z.numel()
    g, ring, stats = torch.ones_like(z), torch.empty(20, dtype=torch.int32, device="cuda"), torch.empty(2, device="cuda")
    fp8.fp8_ring_init(ring, 1.0)
    out, db = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(n, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_act_grad(g, z, 1, n, R.GELU, 0, ring, 0, out, stats[0:1], stats[1:2], db)
    z64 = z.double().clamp(-1e4, 1e4)
    phi, e = _phi(z64, 2.0 ** -4)
    d = z64 * torch.exp(-z64 * z64 / 2) / math.sqrt(2 * math.pi)
    x2 = torch.minimum(z64 * z64, torch.full_like(z64, 200.0))
    _check(db, phi + d, e + d.abs() * (2.0 ** -20 + x2 * 2.0 ** -23) + 2.0 ** -23 * phi, 2.0 ** -123, z)
