"""A NaN in an activation's input is seen in every output that it reaches, and in no other."""

import pytest
import torch

import fp8_delayed_scaling_quantize_b200 as fp8
import ref64 as R

pytestmark = pytest.mark.gpu

ACTS = [R.RELU, R.GELU, R.GELU_TANH, R.SILU]


def _grad(g, z, act, fmt, offsets=None):
    rows, cols = z.shape
    ring, stats = torch.empty(20, dtype=torch.int32, device="cuda"), torch.empty(2, device="cuda")
    fp8.fp8_ring_init(ring, 16.0)
    out = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    if offsets is None:
        db = torch.empty(1, cols, dtype=torch.bfloat16, device="cuda")
        fp8.fp8_act_grad(g, z, rows, cols, act, fmt, ring, 0, out, stats[0:1], stats[1:2], db)
    else:
        db = torch.empty(len(offsets) - 1, cols, dtype=torch.bfloat16, device="cuda")
        fp8.fp8_act_grad_experts(g, z, rows, cols, len(offsets) - 1, offsets, act, fmt, ring, 0, out, stats[0:1],
                                 stats[1:2], db)
    return R.dec(out, fmt), stats[0], db, fp8.fp8_ring_get(ring)


@pytest.mark.parametrize("bits", [0x7FC0, -0x40, 0x7F81, -1], ids=["quiet", "-quiet", "signalling", "all ones"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("act", ACTS)
def test_gradient(act, fmt, bits):
    """Codes and bias gradients of the NaN's place are NaN, whatever the incoming gradient; the amax passes over it."""
    gen = R.gen(act)
    g, z = R.bf16(gen, (70, 72)), R.bf16(gen, (70, 72))
    places = [(0, 0), (33, 7), (34, 8), (69, 71)]
    g[33, 7] = 0.0
    clean = _grad(g, z, act, fmt)
    nan = torch.zeros(70, 72, dtype=torch.bool, device="cuda")
    for at in places:
        z.view(torch.int16)[at] = bits
        nan[at] = True
    off = torch.tensor([0, 34, 34, 70], dtype=torch.int32, device="cuda")
    for offsets in (None, off):
        codes, amax, db, ring = _grad(g, z, act, fmt, offsets)
        assert torch.equal(torch.isnan(codes), nan)
        assert torch.equal(codes[~nan], clean[0][~nan])
        edges = [0, 70] if offsets is None else off.tolist()
        for e, (lo, hi) in enumerate(zip(edges, edges[1:])):
            assert torch.equal(torch.isnan(db[e]), nan[lo:hi].any(0))
        assert torch.isfinite(amax) and ring.hist[0] == float(amax)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [3, 130])
def test_product(act, M, residual):
    """The bias of one column is NaN: that column of the output is, of the kept input too, and no other."""
    N, K = 160, 64
    gen = R.gen(M)
    a, b, one = R.codes(gen, (M, K), 0), R.codes(gen, (N, K), 0), torch.full((1,), 90.0, device="cuda")
    bias = R.bf16(gen, (N,))
    bias[37] = float("nan")
    res = R.bf16(gen, (M, N)) if residual else None
    out, pre = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fp8.fp8_mm_act(a, 0, b, 0, one, one, 0, M, N, K, 1, 0, 0, 0, bias, None, 0, act, res, 0, pre, out)
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[:, 37] = True
    assert torch.equal(torch.isnan(out), want) and torch.equal(torch.isnan(pre), want)
