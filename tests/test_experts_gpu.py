"""fp8_mm_experts against a 64-bit form (bounds: ref64.py)."""

import pytest
import torch

import fp8_delayed_scaling_quantize_b200 as fp8
import ref64 as R

NT, NN, TN = 0, 1, 2


def _off(counts, first=0):
    return torch.tensor([first] + list(counts), dtype=torch.int64).cumsum(0).to(torch.int32)


def _rows(layout, counts, N, K, first=0, behind=0, act=R.NONE, bias=False, preact=False, fa=0, fb=0, stride=1, move=0,
          seed=1, clean=True):
    """NT / NN: one call, every row checked, rows of no expert left as they were."""
    g = R.gen(seed)
    off = _off(counts, first)
    E, T = len(counts), int(off[-1]) + behind
    a = R.codes(g, (T, K), fa)
    b = R.codes(g, (E, N, K) if layout == NT else (E, K, N), fb)
    sa = torch.tensor([R.FMAX[fa] / 5], device="cuda")
    sb = (1 + torch.rand(E if stride else 1, generator=g, device="cuda")) * R.FMAX[fb] * 10
    bias_t = R.bf16(g, (E, N), 0.3) if bias else None
    buf = lambda: torch.full((T * N + move + 32,), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    out, pre = buf(), buf() if preact else None
    fp8.fp8_mm_experts(a, fa, b, fb, sa, sb, stride, layout, T, N, K, E, off.cuda(), bias_t, act,
                       None if pre is None else pre[move:], out[move:])
    assert fp8.fp8_last_device_error() == fp8.FP8_OK
    what = f"{layout} {list(counts)[:8]} N {N} K {K} act {act}"
    for t in (out, pre):
        if t is not None:
            v = t[move:move + T * N].view(T, N)
            assert (v[:int(off[0])] == 7).all() and (v[int(off[-1]):] == 7).all(), what
            assert (t[:move] == 7).all() and (t[move + T * N:] == 7).all(), what
    ad = R.dec(a, fa)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        inv = 1.0 / (sa.double() * sb[e * stride].double())
        z, ez = R.z_and_bound(ad[lo:hi], R.dec(b[e], fb), layout, inv, bias_t[e].double() if bias else None)
        R.check_bf16(out[move:move + T * N].view(T, N)[lo:hi], *R.y_and_bound(z, ez, act), f"{what} expert {e}")
        if preact:
            R.check_bf16(pre[move:move + T * N].view(T, N)[lo:hi], z, ez, f"{what} preact of {e}")


def _sum(counts, M, N, first=0, behind=0, fa=1, fb=0, move=0, seed=2):
    """TN: rows of no expert hold NaN codes, which no output may see."""
    g = R.gen(seed)
    off = _off(counts, first)
    E, T = len(counts), int(off[-1]) + behind
    a, b = R.codes(g, (T, M), fa), R.codes(g, (T, N), fb)
    for t, nan in ((a, 0x7F), (b, 0x7F)):
        t[:int(off[0])] = nan
        t[int(off[-1]):] = nan
    sa, sb = torch.tensor([R.FMAX[fa] * 3], device="cuda"), torch.tensor([R.FMAX[fb] / 5], device="cuda")
    out = torch.full((E * M * N + move + 32,), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_mm_experts(a, fa, b, fb, sa, sb, 0, TN, M, N, T, E, off.cuda(), None, R.NONE, None, out[move:])
    assert fp8.fp8_last_device_error() == fp8.FP8_OK
    assert (out[:move] == 7).all() and (out[move + E * M * N:] == 7).all()
    inv = 1.0 / (sa.double() * sb.double())
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        got = out[move:move + E * M * N].view(E, M, N)[e]
        if lo == hi:
            assert (got == 0).all()
            continue
        z, ez = R.z_and_bound(R.dec(a[lo:hi], fa), R.dec(b[lo:hi], fb), TN, inv)
        R.check_bf16(got, z, ez, f"TN {list(counts)[:8]} {M}x{N} expert {e}")


COUNTS = {
    "one row": [1],
    "one expert": [300],
    "empty ones": [0, 5, 0, 0, 130, 1, 0],
    "ends inside tiles": [127, 128, 129, 1, 255, 257, 64],
    "short": [1, 0, 2, 16, 17, 3, 0, 33, 1, 1],
    "uneven": [3, 900, 0, 12, 40],
    "all on the last": [0] * 30 + [77],
    "many": [(7 * i) % 23 for i in range(512)],
}


@pytest.mark.gpu
@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
@pytest.mark.parametrize("layout,N,K", [(NT, 256, 128), (NT, 130, 16), (NT, 7, 272), (NT, 1032, 400), (NN, 272, 144),
                                        (NN, 16, 48)])
def test_rows(counts, layout, N, K):
    act = (N + len(counts)) % 5
    _rows(layout, counts, N, K, act=act, bias=K % 32 == 16, preact=act != R.NONE, seed=N + K)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", COUNTS.values(), ids=COUNTS.keys())
@pytest.mark.parametrize("M,N", [(16, 16), (144, 272), (256, 512)])
def test_sums(counts, M, N):
    _sum(counts, M, N, seed=M)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[200, 0, 31], [4, 9, 0, 2]], ids=["long", "short"])
@pytest.mark.parametrize("first,behind", [(0, 0), (5, 0), (0, 40), (130, 129)])
@pytest.mark.parametrize("move", [0, 8, 1])
def test_rows_of_no_expert_and_alignment(counts, first, behind, move):
    for N in (264, 137):
        _rows(NT, counts, N, 80, first=first, behind=behind, act=R.SILU, bias=True, preact=True, move=move)
    _rows(NN, counts, 144, 80, first=first, behind=behind, move=move)
    _sum(counts, 144, 80, first=first, behind=behind, move=move)


@pytest.mark.gpu
@pytest.mark.parametrize("fa,fb", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_formats_and_scales(fa, fb):
    for counts in ([40, 300], [3, 5]):
        for stride in (0, 1):
            _rows(NT, counts, 144, 256, fa=fa, fb=fb, stride=stride)
            _rows(NN, counts, 144, 256, fa=fa, fb=fb, stride=stride)
        _sum(counts, 144, 256, fa=fa, fb=fb)


@pytest.mark.gpu
@pytest.mark.parametrize("layout,N,K", [(NT, 2048, 1024), (NN, 1024, 2064)])
def test_large(layout, N, K):
    counts = [1500, 700, 0, 1, 2100, 350, 512, 129]
    _rows(layout, counts, N, K, act=R.GELU_TANH, bias=True, preact=True, behind=7)
    _sum(counts, 1024, 528, behind=7)
    _rows(layout, [9, 0, 30, 2] * 16, N, K, act=R.SILU, bias=True)


@pytest.mark.gpu
def test_other_experts_nan_does_not_spread():
    """A tile's rows of the next expert are loaded and dropped: NaN there stays there."""
    N, K, counts = 272, 144, [40, 300, 5, 64]
    off = _off(counts)
    T = int(off[-1])
    g = R.gen(9)
    a, b = R.codes(g, (T, K), 0), R.codes(g, (4, N, K), 0)
    a[40:340] = 0x7F
    sa = torch.ones(1, device="cuda")
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    for n, o in ((T, off), (45, _off([40, 5]))):
        fp8.fp8_mm_experts(a, 0, b, 0, sa, sa, 0, NT, n, N, K, len(o) - 1, o.cuda(), None, R.NONE, None, out)
        assert torch.isfinite(out[:40]).all() and torch.isnan(out[40:min(n, 340)]).all()
    fp8.fp8_mm_experts(a, 0, b, 0, sa, sa, 0, NT, T, N, K, 4, off.cuda(), None, R.NONE, None, out)
    assert torch.isfinite(out[340:]).all()
    dw = torch.empty(4, K, K, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_mm_experts(a, 0, a, 0, sa, sa, 0, TN, K, K, T, 4, off.cuda(), None, R.NONE, None, dw)
    assert torch.isnan(dw[1]).all() and torch.isfinite(dw[[0, 2, 3]]).all()


@pytest.mark.gpu
def test_offsets_out_of_order_touch_nothing_else():
    """Offsets that break their contract are limited: values differ from nothing defined, but no buffer's edge is
    crossed and the call ends."""
    T, N, K = 200, 256, 64
    g = R.gen(3)
    a, b, sa = R.codes(g, (T, K), 0), R.codes(g, (3, N, K), 0), torch.ones(1, device="cuda")
    want = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_mm_experts(a, 0, b, 0, sa, sa, 0, NT, T, N, K, 3, torch.tensor([0, 150, 150, 200], dtype=torch.int32).cuda(),
                       None, R.NONE, None, want)
    buf = torch.full((T * N + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    bad = torch.tensor([-9, 150, 20, 1 << 30], dtype=torch.int32).cuda()  # taken as 0, 150, 150, 200
    fp8.fp8_mm_experts(a, 0, b, 0, sa, sa, 0, NT, T, N, K, 3, bad, None, R.NONE, None, buf[2048:])
    assert torch.equal(buf[2048:2048 + T * N].view(T, N), want)
    assert (buf[:2048] == 7).all() and (buf[2048 + T * N:] == 7).all()


@pytest.mark.gpu
def test_no_rows():
    sa = torch.ones(1, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    b = torch.zeros(3, 32, 16, dtype=torch.uint8, device="cuda")
    fp8.fp8_mm_experts(None, 0, b, 0, sa, sa, 0, NT, 0, 32, 16, 3, off, None, R.NONE, None, None)
    dw = torch.full((3, 32, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_mm_experts(None, 0, None, 0, sa, sa, 0, TN, 32, 16, 0, 3, off, None, R.NONE, None, dw)
    assert (dw == 0).all()
    out = torch.full((4, 32), 7.0, dtype=torch.bfloat16, device="cuda")  # rows, but none of an expert
    a = torch.zeros(4, 16, dtype=torch.uint8, device="cuda")
    fp8.fp8_mm_experts(a, 0, b, 0, sa, sa, 0, NT, 4, 32, 16, 3, off, None, R.NONE, None, out)
    assert (out == 7).all()


@pytest.mark.gpu
def test_a_captured_call_follows_its_offsets():
    T, N, K, E = 300, 256, 128, 4
    g = R.gen(11)
    a, b, sa = R.codes(g, (T, K), 0), R.codes(g, (E, N, K), 0), torch.full((1,), 50.0, device="cuda")
    off = _off([100, 100, 50, 50]).cuda()
    out, want = (torch.zeros(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    call = lambda o: fp8.fp8_mm_experts(a, 0, b, 0, sa, sa, 0, NT, T, N, K, E, off, None, R.SILU, None, o)  # noqa: E731
    call(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for counts in ([100, 100, 50, 50], [0, 300, 0, 0], [1, 2, 3, 4]):
        off.copy_(_off(counts))
        want.fill_(3.0)
        out.fill_(3.0)
        call(want)
        graph.replay()
        assert torch.equal(out, want)


A, S = 0x7F0000000000, 0x7F0000100000


def _status(layout=NT, M=64, N=128, K=128, experts=4, offsets=S + 64, a8=A, b8=A, sa=S, sb=S, stride=0, bias=None, act=0,
            preact=None, out=A, fa=0):
    return fp8.raw_status("fp8_mm_experts", a8, fa, b8, 0, sa, sb, stride, layout, M, N, K, experts, offsets, bias, act,
                          preact, out, None)


def test_refusals():
    E, AL, U = fp8.FP8_ERR_INVALID_ARG, fp8.FP8_ERR_ALIGNMENT, fp8.FP8_ERR_UNSUPPORTED
    for kw in (dict(fa=2), dict(layout=3), dict(act=5), dict(act=-1), dict(M=-1), dict(N=0), dict(K=0), dict(experts=0),
               dict(offsets=None), dict(a8=None), dict(b8=None), dict(sa=None), dict(sb=None), dict(out=None),
               dict(stride=2), dict(stride=-1), dict(layout=TN, stride=1), dict(layout=TN, bias=A),
               dict(layout=TN, act=1), dict(layout=TN, preact=A), dict(preact=A), dict(layout=TN, M=0), dict(layout=TN, K=-1)):
        assert _status(**kw) == E, kw
    for kw in (dict(K=24), dict(layout=NN, K=24), dict(layout=NN, N=24), dict(layout=TN, M=24), dict(layout=TN, N=24),
               dict(a8=A + 8), dict(b8=A + 8), dict(out=A + 1), dict(preact=A + 4097), dict(bias=A + 1), dict(sa=S + 2),
               dict(sb=S + 2), dict(offsets=S + 2)):
        assert _status(**kw) == AL, kw
    for kw in (dict(experts=513), dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31)):
        assert _status(**kw) == U, kw
