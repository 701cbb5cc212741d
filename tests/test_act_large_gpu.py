"""The epilogue, gradient and expert calls past 2^31 elements, where an offset in 32 bits would wrap, and several calls
at once. Sampled rows against the 64-bit forms (bounds: ref64.py)."""

import pytest
import torch

import fp8_delayed_scaling_quantize_b200 as fp8
import ref64 as R

pytestmark = pytest.mark.gpu

M, N, K = 70000, 32768, 16  # 2.29e9 outputs
ROWS = [0, 1, 127, 128, 33333, 65535, 65536, 69887, 69888, 69998, 69999]


def _big(gen, std=1.0):
    return torch.empty(M, N, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=gen)


def test_product_with_residual_and_preact():
    g = R.gen(1)
    a, b = R.codes(g, (M, K), 0), R.codes(g, (N, K), 0)
    sa, sb = torch.tensor([90.0], device="cuda"), torch.tensor([500.0], device="cuda")
    res, out, pre = _big(g), torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_mm_act(a, 0, b, 0, sa, sb, 0, M, N, K, 1, 0, 0, 0, None, None, 0, R.SILU, res, 0, pre, out)
    assert fp8.fp8_last_device_error() == fp8.FP8_OK
    z, ez = R.z_and_bound(R.dec(a[ROWS], 0), R.dec(b, 0), 0, 1.0 / 45000.0)
    R.check_bf16(pre[ROWS], z, ez)
    R.check_bf16(out[ROWS], *R.y_and_bound(z, ez, R.SILU, res[ROWS].double()))


def test_gradient():
    gen = R.gen(2)
    g, z = _big(gen, 1e-3), _big(gen)
    ring = torch.empty(20, dtype=torch.int32, device="cuda")
    fp8.fp8_ring_init(ring, 1e7)
    out = torch.empty(M, N, dtype=torch.uint8, device="cuda")
    st, db = torch.empty(2, device="cuda"), torch.empty(N, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_act_grad(g, z, M, N, R.GELU, 1, ring, 0, out, st[0:1], st[1:2], db)
    dz = g[ROWS].double() * R.slope(z[ROWS].double(), R.GELU)
    e = g[ROWS].double().abs() * 2.0 ** -20 * z[ROWS].double().abs().clamp(min=1.0) + 2.0 ** -23 * dz.abs()
    R.check_codes(out[ROWS], 1, dz, e, 1e7)
    cols = slice(N - 64, N)
    d = g[:, cols].double() * R.slope(z[:, cols].double(), R.GELU)
    e = g[:, cols].double().abs() * 2.0 ** -20 * z[:, cols].double().abs().clamp(min=1.0) + 2.0 ** -23 * d.abs()
    R.check_bf16(db[cols], d.sum(0), e.sum(0) + M * 2.0 ** -24 * d.abs().sum(0))


def test_experts():
    g = R.gen(3)
    off = torch.tensor([0, 40000, 40000, 69990], dtype=torch.int32)
    a, b = R.codes(g, (M, K), 0), R.codes(g, (3, N, K), 0)
    sa, sb = torch.tensor([90.0], device="cuda"), torch.tensor([500.0], device="cuda")
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_mm_experts(a, 0, b, 0, sa, sb, 0, 0, M, N, K, 3, off.cuda(), None, R.NONE, None, out)
    assert fp8.fp8_last_device_error() == fp8.FP8_OK
    assert (out[69990:] == 0).all()
    for rows, e in (([r for r in ROWS if r < 40000], 0), ([r for r in ROWS if 40000 <= r < 69990], 2)):
        z, ez = R.z_and_bound(R.dec(a[rows], 0), R.dec(b[e], 0), 0, 1.0 / 45000.0)
        R.check_bf16(out[rows], z, ez)


def test_weight_gradients_of_many_experts():
    E, m, n, T = 512, 2048, 2112, 700  # 2.2e9 outputs
    g = R.gen(4)
    counts = torch.bincount(torch.randint(0, E, (T,), generator=torch.Generator().manual_seed(1)), minlength=E)
    off = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
    a, b = R.codes(g, (T, m), 1), R.codes(g, (T, n), 0)
    s = torch.tensor([100.0], device="cuda")
    out = torch.empty(E, m, n, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_mm_experts(a, 1, b, 0, s, s, 0, 2, m, n, T, E, off.cuda(), None, R.NONE, None, out)
    assert fp8.fp8_last_device_error() == fp8.FP8_OK
    for e in (0, 1, 255, 256, 480, 510, 511):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            assert (out[e] == 0).all()
        else:
            R.check_bf16(out[e], *R.z_and_bound(R.dec(a[lo:hi], 1), R.dec(b[lo:hi], 0), 2, 1e-4), f"expert {e}")


def test_calls_on_two_streams_at_once():
    """The same calls, eight of each kind in flight on two streams: what they give one after the other."""
    m, n, k, E = 512, 384, 256, 5
    g = R.gen(5)
    a, b, w = R.codes(g, (m, k), 0), R.codes(g, (n, k), 0), R.codes(g, (E, n, k), 0)
    s = torch.tensor([100.0], device="cuda")
    res, gz = R.bf16(g, (m, n)), R.bf16(g, (m, n))
    off = torch.tensor([0, 100, 101, 300, 300, 512], dtype=torch.int32, device="cuda")

    def calls(i, o):
        fp8.fp8_mm_act(a, 0, b, 0, s, s, 0, m, n, k, 1, 0, 0, 0, None, None, 0, R.GELU, res, 0, None, o["y"][i])
        fp8.fp8_mm_experts(a, 0, w, 0, s, s, 0, 0, m, n, k, E, off, None, R.SILU, None, o["e"][i])
        fp8.fp8_act_grad(gz, res, m, n, R.SILU, 1, o["ring"][i], 0, o["q"][i], None, o["st"][i], o["db"][i])
        fp8.fp8_mm_act_out8(a, 0, b, 0, s, s, 0, m, n, k, 1, 0, 0, 0, None, None, 0, R.RELU, None, 0, o["ring8"][i],
                            o["h"][i], None, o["st8"][i])

    def buffers():
        e = lambda *x, **kw: torch.zeros(8, *x, device="cuda", **kw)  # noqa: E731
        o = dict(y=e(m, n, dtype=torch.bfloat16), e=e(m, n, dtype=torch.bfloat16), q=e(m, n, dtype=torch.uint8),
                 h=e(m, n, dtype=torch.uint8), db=e(n, dtype=torch.bfloat16), st=e(1), st8=e(1),
                 ring=e(20, dtype=torch.int32), ring8=e(20, dtype=torch.int32))
        for r in (*o["ring"], *o["ring8"]):
            fp8.fp8_ring_init(r, 50.0)
        return o

    want, got = buffers(), buffers()
    for i in range(8):
        calls(i, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            calls(i, got)
    torch.cuda.synchronize()
    for key in want:
        assert torch.equal(want[key], got[key]), key
