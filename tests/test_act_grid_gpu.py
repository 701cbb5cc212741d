"""fp8_act_grad where its grid changes with the device's SM count: the widths at which clusters of 16 CTAs give way to
clusters of 8, and strips of 16 columns to wider ones (bounds: test_act_grad_gpu.py)."""

import pytest
import torch

import ref64 as R
from test_act_grad_gpu import _check, _call

import fp8_delayed_scaling_quantize_b200 as fp8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", [R.NONE, R.GELU])
@pytest.mark.parametrize("rows", [700, 9000])
@pytest.mark.parametrize("per_sm", [1, 2, 4])
def test_widths_around_a_full_device(rows, per_sm, act):
    """strips of 16 columns x 8 CTAs around `per_sm` for each SM, and their neighbours."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    cols = 16 * -(-sms * per_sm // 8)
    for c in (cols - 16, cols - 8, cols, cols + 8):
        gen = R.gen(c + rows)
        g, z = R.bf16(gen, (rows, c), 1e-3), R.bf16(gen, (rows, c), 2.0)
        ring = torch.empty(20, dtype=torch.int32, device="cuda")
        s = float(torch.tensor(R.FMAX[1] / 5e-3, dtype=torch.float32))
        fp8.fp8_ring_init(ring, s)
        _check(g, z, rows, c, act, 1, _call(g, z, rows, c, act, 1, ring), s, f"{rows}x{c}")


@pytest.mark.parametrize("cols", [8, 16, 32, 128])
def test_narrow_tensors_in_a_graph(cols):
    """The widest clusters, captured and replayed on another stream than the one that captured them."""
    rows = 5000
    gen = R.gen(cols)
    g, z = R.bf16(gen, (rows, cols), 1e-3), R.bf16(gen, (rows, cols), 2.0)
    ring, other = (torch.empty(20, dtype=torch.int32, device="cuda") for _ in range(2))
    for r in (ring, other):
        fp8.fp8_ring_init(r, 1e6)
    out, stats = torch.empty(rows * cols, dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
    db = torch.empty(cols, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        fp8.fp8_act_grad(g, z, rows, cols, R.SILU, 1, ring, 0, out, stats[0:1], stats[1:2], db)
    with torch.cuda.stream(stream):
        graph.replay()
    torch.cuda.synchronize()
    want = torch.empty_like(out), torch.empty_like(db)
    fp8.fp8_act_grad(g, z, rows, cols, R.SILU, 1, other, 0, want[0], stats[0:1], stats[1:2], want[1])
    assert torch.equal(out, want[0]) and torch.equal(db, want[1]) and torch.equal(ring, other)
