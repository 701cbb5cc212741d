"""Where the weight gradient of fp8_mm_experts reads: blocks that end among another expert's rows, and token matrices
at the ends of their memory, after graphs and buffers of earlier calls are gone (bounds: ref64.py)."""

import gc

import pytest
import torch

import fp8_delayed_scaling_quantize_b200 as fp8
import ref64 as R

TN = 2


def _off(counts):
    return torch.tensor([0] + list(counts), dtype=torch.int64).cumsum(0).to(torch.int32)


def _call(a, b, off, sa, out):
    fp8.fp8_mm_experts(a, 1, b, 0, sa, sa, 0, TN, a.shape[1], b.shape[1], a.shape[0], len(off) - 1, off, None, R.NONE,
                       None, out)


def _check(a, b, off, sa, out, experts):
    inv = 1.0 / (sa.double() * sa.double())
    for e in experts:
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            assert (out[e] == 0).all()
            continue
        z, ez = R.z_and_bound(R.dec(a[lo:hi], 1), R.dec(b[lo:hi], 0), TN, inv)
        R.check_bf16(out[e], z, ez, f"rows [{lo}, {hi})")


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["a", "b"])
@pytest.mark.parametrize("counts", [range(1, 65), range(65, 130), range(100, 300)], ids=["1-64", "65-129", "100-299"])
def test_every_tail_beside_nan(counts, where):
    """Every length of an expert's last block, with NaN codes in the rows of the experts on both sides."""
    g = R.gen(5)
    off = _off([n for c in counts for n in (c, 3)])  # an expert that is checked, then three rows of one that is NaN
    T, E = int(off[-1]), 2 * len(counts)
    a, b = R.codes(g, (T, 48), 1), R.codes(g, (T, 272), 0)
    for e in range(1, E, 2):
        (a if where == "a" else b)[int(off[e]):int(off[e + 1])] = 0x7F
    sa = torch.full((1,), 30.0, device="cuda")
    out = torch.empty(E, 48, 272, dtype=torch.bfloat16, device="cuda")
    _call(a, b, off.cuda(), sa, out)
    assert fp8.fp8_last_device_error() == fp8.FP8_OK
    _check(a, b, off, sa, out, range(0, E, 2))
    assert torch.isnan(out[1::2]).all()


@pytest.mark.gpu
def test_after_graphs_and_buffers_are_gone():
    """Calls of a few rows, captured and replayed, whose graph and memory are given back before the next ones'."""
    g = R.gen(6)
    sa = torch.full((1,), 30.0, device="cuda")
    for turn in range(6):
        states = []
        for counts, M, N in (([1] + [0] * 20, 384, 1056), ([0, 30, 0], 1152, 592), ([0] * 40 + [1], 256, 272)):
            off = _off(counts)
            T = int(off[-1]) + 3 * (turn % 2)
            states.append((R.codes(g, (T, M), 1), R.codes(g, (T, N), 0), off.cuda(), sa,
                           torch.empty(len(counts), M, N, dtype=torch.bfloat16, device="cuda")))
        for s in states:
            _call(*s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                for s in states:
                    _call(*s)
        for s in states:
            s[4].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert fp8.fp8_last_device_error() == fp8.FP8_OK
        for s in states:
            _check(*s, range(len(s[2]) - 1))
        del graph, states, s
        gc.collect()
        torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("off", [[0, 5, 40], [3, 3, 40], [0, 7, 9], [11, 20, 33], [40, 40, 40], [0, 0, 0], [-5, 3, 99],
                                 [30, 7, 12]])
@pytest.mark.parametrize("cols", [8, 2056])
def test_zeros_in_rows_of_no_expert(off, cols):
    rows, pad = 40, 64
    buf = torch.full((rows * cols + 2 * pad,), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_experts_zero_rest(buf[pad:], rows, 2 * cols, 2, torch.tensor(off, dtype=torch.int32, device="cuda"))
    lo = min(max(off[0], 0), rows)
    hi = min(max(off[2], lo), rows)
    v = buf[pad:pad + rows * cols].view(rows, cols)
    assert (v[:lo] == 0).all() and (v[lo:hi] == 7).all() and (v[hi:] == 0).all()
    assert (buf[:pad] == 7).all() and (buf[pad + rows * cols:] == 7).all()


def test_refusals_of_zeros_in_rows_of_no_expert():
    A = 0x7F0000000000

    def status(out=A, rows=4, row_bytes=32, experts=2, offsets=A + 64):
        return fp8.raw_status("fp8_experts_zero_rest", out, rows, row_bytes, experts, offsets, None)

    assert status(rows=0, out=None) == fp8.FP8_OK  # no rows: no launch
    for bad in (dict(out=None), dict(rows=-1), dict(row_bytes=0), dict(experts=0), dict(offsets=None)):
        assert status(**bad) == fp8.FP8_ERR_INVALID_ARG, bad
    for bad in (dict(experts=513), dict(rows=1 << 31), dict(row_bytes=1 << 32)):
        assert status(**bad) == fp8.FP8_ERR_UNSUPPORTED, bad
    for bad in (dict(row_bytes=24), dict(out=A + 8), dict(offsets=A + 2)):
        assert status(**bad) == fp8.FP8_ERR_ALIGNMENT, bad
