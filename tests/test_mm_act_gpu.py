"""fp8_mm_act and fp8_mm_act_out8 against a 64-bit form (bounds: ref64.py)."""

import pytest
import torch

import fp8_delayed_scaling_quantize_b200 as fp8
import ref64 as R

NT, NN, TN = 0, 1, 2
INV = 1.0 / (90.0 * 4480.0)


def _operands(seed, layout, M, N, K, batch=1, fa=0, fb=0, bcast_b=False):
    g = R.gen(seed)
    sa = (batch,) + ((M, K) if layout != TN else (K, M))
    sb = (1 if bcast_b else batch,) + ((N, K) if layout == NT else (K, N))
    a = R.codes(g, sa, fa, 90.0 if fa == 0 else 9000.0)
    b = R.codes(g, sb, fb, 90.0 if fb == 0 else 9000.0)
    return g, a, b, torch.tensor([90.0 if fa == 0 else 9000.0], device="cuda"), \
        torch.tensor([4480.0 if fb == 0 else 448000.0], device="cuda")


def _run(seed, layout, M, N, K, act, bias=0, residual="none", preact=False, batch=1, fa=0, fb=0, pad=0,
         bcast_b=False, offset=0):
    """One call, every output checked, what lies between and behind the matrices left as it was. offset: elements
    that out, residual and preact are moved from a 16-byte boundary."""
    g, a, b, sa, sb = _operands(seed, layout, M, N, K, batch, fa, fb, bcast_b)
    inv = 1.0 / (sa.double() * sb.double())
    std = float(K) ** 0.5 * 0.02
    sc = M * N + pad
    buf = lambda: torch.full((batch * sc + offset + 64,), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    out, z_out = buf(), buf() if preact else None
    cut = lambda t: t[offset:offset + batch * sc].view(batch, sc)[:, :M * N].view(batch, M, N)  # noqa: E731
    bias_t = bias_s = None
    bias64 = None
    if bias == 1:
        bias_t = R.bf16(g, (N,), std)
        bias64 = bias_t.double()
    elif bias == 2:
        bias_t, bias_s = R.codes(g, (N,), 0, 60.0), torch.tensor([100.0], device="cuda")
        bias64 = R.dec(bias_t, 0) / 100.0
    res_t, res64, stride_r = None, None, 0
    if residual == "full":
        res_t, stride_r = buf(), sc
        cut(res_t).copy_(R.bf16(g, (batch, M, N), std))
        res64 = cut(res_t).double()
    elif residual == "broadcast":
        res_t = torch.empty(M * N + offset, dtype=torch.bfloat16, device="cuda")
        res_t[offset:] = R.bf16(g, (M * N,), std)
        res64 = res_t[offset:].view(1, M, N).double()
    elif residual == "in place":
        cut(out).copy_(R.bf16(g, (batch, M, N), std))
        res_t, stride_r, res64 = out, sc, cut(out).double()
    fp8.fp8_mm_act(a, fa, b, fb, sa, sb, layout, M, N, K, batch, a[0].numel(), 0 if bcast_b else b[0].numel(), sc,
                   bias_t, bias_s, 0, act, None if res_t is None else res_t[offset:], stride_r,
                   None if z_out is None else z_out[offset:], out[offset:])
    assert fp8.fp8_last_device_error() == fp8.FP8_OK
    z, ez = R.z_and_bound(R.dec(a, fa), R.dec(b, fb), layout, inv, bias64)
    y, ey = R.y_and_bound(z, ez, act, res64)
    what = f"{layout} {M}x{N}x{K} b{batch} act {act} bias {bias} residual {residual}"
    R.check_bf16(cut(out), y, ey, what)
    if preact:
        R.check_bf16(cut(z_out), z, ez, what + " preact")
    for t in (out, z_out):
        if t is not None:
            assert (t[:offset] == 7).all() and (t[offset + batch * sc:] == 7).all(), what
            if pad:
                assert (t[offset:offset + batch * sc].view(batch, sc)[:, M * N:] == 7).all(), what


SHAPES = [
    # smallest, swapped (M <= 32) with and without a cluster split, odd N in every path
    (NT, 1, 1, 16), (NT, 1, 7, 32), (NT, 3, 130, 48), (NT, 1, 4096, 4096), (NT, 16, 1000, 2048), (NT, 32, 257, 1040),
    (NN, 1, 144, 16), (NN, 31, 1040, 2064), (NN, 17, 128, 4096),
    # unswapped: 64-, 128- and 256-wide tiles, ragged rows and columns
    (NT, 33, 64, 16), (NT, 33, 63, 144), (NT, 129, 257, 128), (NT, 300, 520, 1040), (NT, 128, 8192, 256),
    (NT, 1000, 1536, 1024), (NN, 33, 16, 48), (NN, 255, 528, 272), (NN, 1001, 1040, 2064),
    (TN, 16, 16, 1), (TN, 144, 272, 77), (TN, 1024, 1024, 2048),
]


@pytest.mark.gpu
@pytest.mark.parametrize("layout,M,N,K", SHAPES)
@pytest.mark.parametrize("act", [R.NONE, R.RELU, R.GELU, R.GELU_TANH, R.SILU])
def test_shapes_and_activations(layout, M, N, K, act):
    _run(M + N + K + act, layout, M, N, K, act, bias=(act + M) % 3, residual=("full", "none", "in place")[act % 3],
         preact=(act + N) % 2 == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("layout,M,N,K", [(NT, 4096, 4096, 2048), (NN, 3000, 4112, 2064), (TN, 4096, 3856, 2080)])
def test_pair_tiles(layout, M, N, K):
    _run(5, layout, M, N, K, R.GELU_TANH, bias=1, residual="full", preact=True)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(5, 144, 256), (40, 136, 128), (200, 264, 384)])
@pytest.mark.parametrize("residual", ["full", "broadcast", "in place"])
@pytest.mark.parametrize("offset,pad", [(0, 0), (0, 24), (0, 3), (1, 0), (4, 8)])
def test_batches_strides_and_alignment(M, N, K, residual, offset, pad):
    """Whole-tile stores, and the plain stores that unaligned bases and strides take."""
    if offset % 2:
        offset += 1  # out is 4-byte aligned
    _run(M + pad, NT, M, N, K, R.SILU, bias=1, residual=residual, preact=True, batch=3, pad=pad, offset=offset)
    if N % 16 == 0:  # NN refuses other widths
        _run(M + pad, NN, M, N, K, R.NONE, residual=residual, batch=3, pad=pad, offset=offset, bcast_b=True)


@pytest.mark.gpu
@pytest.mark.parametrize("fa,fb", [(0, 1), (1, 0), (1, 1)])
def test_formats(fa, fb):
    for layout, M, N, K in ((NT, 8, 320, 512), (NT, 130, 320, 512), (NN, 130, 320, 512), (TN, 128, 320, 512)):
        _run(3, layout, M, N, K, R.GELU, bias=2, residual="full", preact=True, fa=fa, fb=fb)


@pytest.mark.gpu
def test_residual_and_preact_may_be_unaligned_apart():
    """out aligned, residual two bytes past a boundary: plain accesses."""
    M, N, K = 70, 128, 64
    g, a, b, sa, sb = _operands(1, NT, M, N, K)
    res = R.bf16(g, (M * N + 1,))
    out, pre = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fp8.fp8_mm_act(a, 0, b, 0, sa, sb, NT, M, N, K, 1, 0, 0, 0, None, None, 0, R.SILU, res[1:], 0, pre, out)
    z, ez = R.z_and_bound(R.dec(a[0], 0), R.dec(b[0], 0), NT, INV)
    R.check_bf16(pre, z, ez)
    R.check_bf16(out, *R.y_and_bound(z, ez, R.SILU, res[1:].view(M, N).double()))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 64])
@pytest.mark.parametrize("act", [R.NONE, R.RELU, R.GELU, R.GELU_TANH, R.SILU])
def test_nan_and_infinities(M, act):
    """A NaN operand row gives NaN in its row alone; an infinite z gives the activation's limits."""
    N, K = 256, 64
    g, a, b, sa, sb = _operands(2, NT, M, N, K, fa=1)
    a[0, 1, 5] = 0x7E          # NaN (E5M2)
    b = torch.where(b == 0, torch.ones_like(b), b)
    b[0, :, 9] = 0x38          # 1.0, so that inf * b keeps its sign
    a[0, 2, 9], a[0, 3, 9] = 0x7C, 0xFC  # +inf, -inf
    out, pre = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fp8.fp8_mm_act(a, 1, b, 0, sa, sb, NT, M, N, K, 1, 0, 0, 0, None, None, 0, act, None, 0, pre, out)
    assert torch.isnan(out[1]).all() and torch.isnan(pre[1]).all()
    assert (pre[2] == float("inf")).all() and (pre[3] == -float("inf")).all()
    assert (out[2] == float("inf")).all()
    assert (out[3] == (-float("inf") if act == R.NONE else 0.0)).all()
    rest = [i for i in range(M) if i not in (1, 2, 3)]
    assert torch.isfinite(out[rest]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("layout,M,N,K,fmt", [(NT, 1, 128, 32, 0), (NT, 33, 65, 144, 0), (NT, 257, 512, 1024, 1),
                                              (NN, 300, 272, 272, 0), (TN, 144, 528, 100, 0), (NT, 4096, 4096, 2048, 0)])
@pytest.mark.parametrize("act", [R.NONE, R.RELU, R.GELU, R.GELU_TANH, R.SILU])
def test_out8(layout, M, N, K, fmt, act):
    g, a, b, sa, sb = _operands(M + act, layout, M, N, K)
    inv = 1.0 / (sa.double() * sb.double())
    bias = R.bf16(g, (N,), 0.3)
    ring = torch.empty(20, dtype=torch.int32, device="cuda")
    s0 = R.FMAX[fmt] / (1.5 * K ** 0.5 * 0.08)  # the largest values saturate
    fp8.fp8_ring_init(ring, s0)
    s0 = float(torch.tensor(s0, dtype=torch.float32))
    out = torch.full((M * N + 64,), 9, dtype=torch.uint8, device="cuda")
    pre = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    amax, scale = (torch.empty(1, device="cuda") for _ in range(2))
    for call in range(2):  # the second under the scale that the first published
        fp8.fp8_mm_act_out8(a, 0, b, 0, sa, sb, layout, M, N, K, 1, 0, 0, 0, bias, None, 0, act,
                            pre if call == 0 else None, fmt, ring, out, amax, scale)
        z, ez = R.z_and_bound(R.dec(a[0], 0), R.dec(b[0], 0), layout, inv, bias.double())
        y, ey = R.y_and_bound(z, ez, act)
        s = s0 if call == 0 else float(host.scale)  # noqa: F821
        assert float(scale) == s
        R.check_codes(out[:M * N].view(M, N), fmt, y, ey, s, f"call {call}")
        assert (out[M * N:] == 9).all()
        top = float(y.abs().max())
        e = float(ey.max())
        assert abs(float(amax) - top) <= e + 2.0 ** -23 * top
        host = fp8.fp8_ring_get(ring)
        assert host.idx == call + 1 and host.hist[call] == float(amax) and host.amax_bits == 0 and host.ticket == 0
        if call == 0:
            R.check_bf16(pre, z, ez)
            assert host.scale == float(torch.tensor(R.FMAX[fmt]) / amax.cpu())


@pytest.mark.gpu
def test_plain_epilogue_equals_fp8_mm():
    """With act NONE and no residual the outputs are fp8_mm's, bit for bit, where both run the same tiles."""
    for layout, M, N, K in ((NT, 1, 4096, 4096), (NT, 200, 520, 512), (NN, 640, 1040, 272), (TN, 256, 272, 300)):
        g, a, b, sa, sb = _operands(8, layout, M, N, K)
        bias = R.bf16(g, (N,))
        x, y = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        fp8.fp8_mm(a, 0, b, 0, sa, sb, layout, M, N, K, 1, 0, 0, 0, bias, None, 0, x)
        fp8.fp8_mm_act(a, 0, b, 0, sa, sb, layout, M, N, K, 1, 0, 0, 0, bias, None, 0, R.NONE, None, 0, None, y)
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.gpu
def test_captured_and_replayed_on_another_stream():
    M, N, K = 260, 384, 512
    g, a, b, sa, sb = _operands(4, NT, M, N, K)
    res = R.bf16(g, (M, N))
    want, out, pre = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    call = lambda o: fp8.fp8_mm_act(a, 0, b, 0, sa, sb, NT, M, N, K, 1, 0, 0, 0, None, None, 0, R.GELU, res, 0, pre, o)  # noqa: E731
    call(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
        call(out)
    side = torch.cuda.Stream()
    for _ in range(3):
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want)


# ---------------------------------------------------------------- refusals (no GPU) ---

A, S = 0x7F0000000000, 0x7F0000100000


def _act(act=1, residual=None, stride_r=0, preact=None, M=128, N=128, K=128, batch=1, stride_c=0, layout=0, out=A + 4096,
         a8=A, sa=S, bias=None, bias_scale=None):
    return fp8.raw_status("fp8_mm_act", a8, 0, A + 65536, 0, sa, S + 4, layout, M, N, K, batch, 0, 0, stride_c, bias,
                          bias_scale, 0, act, residual, stride_r, preact, out, None)


def _out8(act=1, preact=None, fmt=0, ring=S + 64, out=A + 4096, scale=S + 8, amax=None, K=128):
    return fp8.raw_status("fp8_mm_act_out8", A, 0, A + 65536, 0, S, S + 4, 0, 128, 128, K, 1, 0, 0, 0, None, None, 0, act,
                          preact, fmt, ring, out, amax, scale, None)


def test_refusals():
    E, AL, U = fp8.FP8_ERR_INVALID_ARG, fp8.FP8_ERR_ALIGNMENT, fp8.FP8_ERR_UNSUPPORTED
    assert _act(act=5) == E and _act(act=-1) == E
    assert _act(out=None) == E and _act(a8=None) == E and _act(sa=None) == E
    assert _act(M=0) == E and _act(N=0) == E and _act(K=0) == E and _act(batch=0) == E
    assert _act(layout=3) == E and _act(bias_scale=S) == E
    assert _act(residual=A, stride_r=-8) == E
    assert _act(residual=A, batch=2, stride_c=128 * 128, stride_r=128) == E
    assert _act(batch=2, stride_c=8) == E
    assert _act(preact=A + 4096) == E and _act(preact=A, residual=A) == E  # preact is out, preact is residual
    assert _act(residual=A + 4096, batch=2, stride_c=128 * 128, stride_r=0) == E  # in place under another stride
    assert _out8(preact=A + 4096) == E
    assert _act(residual=A + 1) == AL and _act(preact=A + 1) == AL and _act(out=A + 2) == AL
    assert _act(K=24) == AL and _act(a8=A + 8) == AL
    assert _act(M=1 << 31) == U
    assert _out8(act=7) == E and _out8(fmt=2) == E and _out8(ring=None) == E and _out8(scale=None) == E
    assert _out8(out=None) == E
    assert _out8(preact=A + 1) == AL and _out8(ring=S + 2) == AL and _out8(scale=S + 9) == AL and _out8(amax=S + 1) == AL
    assert _out8(K=8) == AL
