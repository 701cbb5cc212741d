"""fp8_act_grad against a 64-bit form and against differences.

Bounds: dz is g times the slope, whose own formula errs by at most 2^-20 max(1, |z|) for |z| <= 1 (ex2.approx and
rcp.approx good to 2^-22, three more fp32 roundings) and decays with the slope's tail beyond; codes add half a step; a
bias gradient of n rows in fp32 adds n 2^-24 of the absolute sum and half a bf16 step."""

import pytest
import torch

import fp8_delayed_scaling_quantize_b200 as fp8
import ref64 as R


def _call(g, z, rows, cols, act, fmt, ring, flags=0, dbias=True, out=None):
    out = torch.full((rows * cols + 64,), 9, dtype=torch.uint8, device="cuda") if out is None else out
    amax, scale = (torch.empty(1, device="cuda") for _ in range(2))
    db = torch.full((cols + 8,), 7.0, dtype=torch.bfloat16, device="cuda") if dbias else None
    fp8.fp8_act_grad(g if rows else None, z if rows else None, rows, cols, act, fmt, ring, flags, out if rows else None,
                     amax, scale, db)
    return out, amax, scale, db


def _check(g, z, rows, cols, act, fmt, got, s, what):
    out, amax, scale, db = got
    z64 = z.double() if z is not None else torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    dz = g.double() * R.slope(z64, act)
    e = g.double().abs() * (2.0 ** -20 * z64.abs().clamp(min=1.0) if act > R.RELU else 0.0) + 2.0 ** -23 * dz.abs()
    assert float(scale) == s, what
    R.check_codes(out[:rows * cols].view(rows, cols), fmt, dz, e, s, what)
    assert (out[rows * cols:] == 9).all(), what
    top = float(dz.abs().max()) if rows else 0.0
    assert abs(float(amax) - top) <= (float(e.max()) if rows else 0.0), what
    if db is not None:
        R.check_bf16(db[:cols], dz.sum(0), e.sum(0) + rows * 2.0 ** -24 * dz.abs().sum(0), what + " dbias")
        assert (db[cols:] == 7).all(), what


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 4096), (2, 72), (31, 64), (33, 1040), (64, 16), (65, 128), (129, 264),
                                       (1000, 24), (513, 1016), (2048, 4096), (20000, 48), (7, 9992)])
@pytest.mark.parametrize("act", [R.NONE, R.RELU, R.GELU, R.GELU_TANH, R.SILU])
def test_shapes(rows, cols, act):
    gen = R.gen(rows + cols + act)
    g, z = R.bf16(gen, (rows, cols), 1e-3), R.bf16(gen, (rows, cols), 2.0)
    z = None if act == R.NONE and cols % 16 else z
    for fmt in (0, 1):
        ring = torch.empty(20, dtype=torch.int32, device="cuda")
        s = float(torch.tensor(R.FMAX[fmt] / 2.5e-3, dtype=torch.float32))  # the largest values saturate
        fp8.fp8_ring_init(ring, s)
        got = _call(g, z, rows, cols, act, fmt, ring, dbias=(rows + fmt) % 3 != 0)
        _check(g, z, rows, cols, act, fmt, got, s, f"{rows}x{cols} act {act} fmt {fmt}")
        h = fp8.fp8_ring_get(ring)
        a = float(got[1])
        assert (h.idx, h.hist[0], h.amax_bits, h.ticket) == (1, a, 0, 0)
        assert h.scale == (float(torch.tensor(R.FMAX[fmt]) / torch.tensor(a)) if a > 0 else s)
        again = _call(g, z, rows, cols, act, fmt, ring)
        _check(g, z, rows, cols, act, fmt, again, float(h.scale), "under the published scale")


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(8191, 296), (8192, 296), (8201, 576), (9999, 584), (10001, 1024), (8192, 1032)])
@pytest.mark.parametrize("act", [R.NONE, R.RELU, R.GELU, R.GELU_TANH, R.SILU])
def test_tall_and_narrow(rows, cols, act):
    test_shapes(rows, cols, act)


@pytest.mark.gpu
def test_no_rows():
    ring = torch.empty(20, dtype=torch.int32, device="cuda")
    fp8.fp8_ring_init(ring, 3.0)
    out, amax, scale, db = _call(None, None, 0, 72, R.SILU, 1, ring)
    assert float(amax) == 0.0 and float(scale) == 3.0 and (db[:72] == 0).all() and (db[72:] == 7).all()
    h = fp8.fp8_ring_get(ring)
    assert h.idx == 1 and h.scale == 3.0 and h.ticket == 0


@pytest.mark.gpu
@pytest.mark.parametrize("act", [R.RELU, R.GELU, R.GELU_TANH, R.SILU])
def test_slope_over_every_bf16_value(act):
    """g = 1 over every finite z and both infinities: the slope against its formula, its limits 0 and 1."""
    bits = torch.arange(0, 65536, dtype=torch.int32).to(torch.int16).cuda().view(torch.bfloat16)
    z = bits[~torch.isnan(bits)]
    z = z[:z.numel() // 8 * 8].contiguous()
    rows, cols = z.numel() // 8, 8
    ring = torch.empty(20, dtype=torch.int32, device="cuda")
    fp8.fp8_ring_init(ring, 256.0)
    g = torch.ones_like(z).view(rows, cols)
    out, amax, _, _ = _call(g, z.view(rows, cols), rows, cols, act, 0, ring, dbias=False)
    want = R.slope(z.double().clamp(-1e4, 1e4), act).view(rows, cols)
    e = 2.0 ** -20 * torch.ones_like(want)
    R.check_codes(out[:rows * cols].view(rows, cols), 0, want, e, 256.0)
    assert abs(float(amax) - float(want.max())) <= 2.0 ** -20


@pytest.mark.gpu
@pytest.mark.parametrize("act", [R.GELU, R.GELU_TANH, R.SILU])
def test_against_differences(act):
    """The slope against (act(z + h) - act(z - h)) / 2h in 64 bits: third derivatives are below 2, so h = 1e-4 errs by
    1e-8; the code's half step is the rest."""
    z = R.bf16(R.gen(1), (64, 64), 2.0)
    ring = torch.empty(20, dtype=torch.int32, device="cuda")
    fp8.fp8_ring_init(ring, 256.0)
    out, _, _, _ = _call(torch.ones_like(z), z, 64, 64, act, 0, ring, dbias=False)
    z64 = z.double()
    want = (R.act(z64 + 1e-4, act) - R.act(z64 - 1e-4, act)) / 2e-4
    R.check_codes(out[:4096].view(64, 64), 0, want, 2.0 ** -20 + torch.zeros_like(want), 256.0)


@pytest.mark.gpu
def test_nan_stays_in_its_column():
    g, z = R.bf16(R.gen(2), (100, 64)), R.bf16(R.gen(3), (100, 64))
    g[17, 5] = float("nan")
    z[40, 9] = float("nan")
    ring = torch.empty(20, dtype=torch.int32, device="cuda")
    fp8.fp8_ring_init(ring, 100.0)
    out, amax, _, db = _call(g, z, 100, 64, R.SILU, 0, ring)
    q = R.dec(out[:6400].view(100, 64), 0)
    assert torch.isnan(q[17, 5]) and torch.isnan(q[40, 9]) and int(torch.isnan(q).sum()) == 2
    assert torch.isnan(db[5]) and torch.isnan(db[9]) and int(torch.isnan(db[:64]).sum()) == 2
    assert torch.isfinite(amax).all()


@pytest.mark.gpu
def test_none_equals_quantize_and_deferred_fold():
    rows, cols = 300, 520
    g = R.bf16(R.gen(4), (rows, cols))
    rings = torch.empty(2, 20, dtype=torch.int32, device="cuda")
    for r in rings:
        fp8.fp8_ring_init(r, 50.0)
    want = torch.empty(rows * cols, dtype=torch.uint8, device="cuda")
    am, sc = (torch.empty(1, device="cuda") for _ in range(2))
    fp8.fp8_quantize_ex(g, fp8.FP8_IN_BF16, rows * cols, 1, rings[0], fp8.FP8_QUANTIZE_DEFER_FOLD, want, am, sc)
    out, amax, scale, _ = _call(g, None, rows, cols, R.NONE, 1, rings[1], flags=fp8.FP8_QUANTIZE_DEFER_FOLD)
    assert torch.equal(out[:rows * cols], want) and torch.equal(amax, am) and torch.equal(scale, sc)
    assert torch.equal(rings[0], rings[1])
    fp8.fp8_rings_fold(rings, 2, [1, 1])
    assert torch.equal(rings[0], rings[1]) and fp8.fp8_ring_get(rings[1]).idx == 1


@pytest.mark.gpu
def test_captured_with_its_ring():
    rows, cols = 500, 256
    g, z = R.bf16(R.gen(5), (rows, cols)), R.bf16(R.gen(6), (rows, cols))
    ring, other = (torch.empty(20, dtype=torch.int32, device="cuda") for _ in range(2))
    fp8.fp8_ring_init(ring, 1.0)
    fp8.fp8_ring_init(other, 1.0)
    out, db = torch.empty(rows * cols, dtype=torch.uint8, device="cuda"), torch.empty(cols, dtype=torch.bfloat16, device="cuda")
    am, sc = (torch.empty(1, device="cuda") for _ in range(2))
    fp8.fp8_act_grad(g, z, rows, cols, R.GELU, 1, ring, 0, out, am, sc, db)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.fp8_act_grad(g, z, rows, cols, R.GELU, 1, ring, 0, out, am, sc, db)
    graph.replay()
    graph.replay()
    first = out.clone(), db.clone()
    for _ in range(3):
        fp8.fp8_act_grad(g, z, rows, cols, R.GELU, 1, other, 0, out, am, sc, db)
    assert torch.equal(out, first[0]) and torch.equal(db, first[1]) and torch.equal(ring, other)


A, S = 0x7F0000000000, 0x7F0000100000


def _status(g=A, z=A, rows=8, cols=64, act=4, fmt=1, ring=S, flags=0, out=A, amax=None, scale=S + 128, db=None):
    return fp8.raw_status("fp8_act_grad", g, z, rows, cols, act, fmt, ring, flags, out, amax, scale, db, None)


def test_refusals():
    E, AL = fp8.FP8_ERR_INVALID_ARG, fp8.FP8_ERR_ALIGNMENT
    for kw in (dict(act=5), dict(act=-1), dict(fmt=2), dict(rows=-1), dict(cols=0), dict(cols=-8), dict(rows=1 << 40),
               dict(rows=1 << 36, cols=64), dict(g=None), dict(z=None), dict(out=None), dict(ring=None),
               dict(scale=None), dict(flags=1), dict(flags=3), dict(flags=4)):
        assert _status(**kw) == E, kw
    for kw in (dict(cols=12), dict(g=A + 2), dict(z=A + 8), dict(out=A + 8), dict(ring=S + 2), dict(scale=S + 130),
               dict(amax=S + 1), dict(db=S + 1)):
        assert _status(**kw) == AL, kw


# ------------------------------------------------------------- rows of experts ---


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[5], [300], [0, 5, 0, 0, 130, 1, 0], [127, 128, 129, 1, 255, 257, 64], [0] * 30 + [77],
                                    [(7 * i) % 23 for i in range(512)], [2000, 1, 0, 3000]])
@pytest.mark.parametrize("cols", [8, 264, 1040, 4096])
@pytest.mark.parametrize("act", [R.NONE, R.SILU])
def test_rows_of_experts(counts, cols, act):
    gen = R.gen(cols + len(counts))
    first, behind = (3, 9) if len(counts) % 2 else (0, 0)
    off = torch.tensor([first] + counts).cumsum(0).to(torch.int32)
    E, T, lo, hi = len(counts), int(off[-1]) + behind, int(off[0]), int(off[-1])
    g, z = R.bf16(gen, (T, cols), 1e-3), R.bf16(gen, (T, cols), 2.0)
    g[:lo] = 1.0  # rows of no expert: neither amax nor sums may see them
    g[hi:] = float("nan")
    ring = torch.empty(20, dtype=torch.int32, device="cuda")
    s = float(torch.tensor(R.FMAX[1] / 2.5e-3, dtype=torch.float32))
    fp8.fp8_ring_init(ring, s)
    out = torch.full((T, cols), 9, dtype=torch.uint8, device="cuda")
    amax, scale = (torch.empty(1, device="cuda") for _ in range(2))
    db = torch.full((E, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_act_grad_experts(g, z, T, cols, E, off.cuda(), act, 1, ring, 0, out, amax, scale, db)
    assert (out[:lo] == 9).all() and (out[hi:] == 9).all() and float(scale) == s
    dz = g[lo:hi].double() * R.slope(z[lo:hi].double(), act)
    e = g[lo:hi].double().abs() * (2.0 ** -20 * z[lo:hi].double().abs().clamp(min=1.0) if act else 0.0) + 2.0 ** -23 * dz.abs()
    R.check_codes(out[lo:hi], 1, dz, e, s)
    assert abs(float(amax) - float(dz.abs().max())) <= float(e.max())
    for k in range(E):
        a, b = int(off[k]) - lo, int(off[k + 1]) - lo
        d = dz[a:b]
        R.check_bf16(db[k], d.sum(0), e[a:b].sum(0) + (b - a) * 2.0 ** -24 * d.abs().sum(0), f"expert {k}")
    h = fp8.fp8_ring_get(ring)
    assert (h.idx, h.hist[0], h.amax_bits, h.ticket) == (1, float(amax), 0, 0)


@pytest.mark.gpu
def test_experts_without_rows_and_offsets_out_of_order():
    ring = torch.empty(20, dtype=torch.int32, device="cuda")
    fp8.fp8_ring_init(ring, 3.0)
    g = R.bf16(R.gen(1), (50, 64))
    amax, scale = (torch.empty(1, device="cuda") for _ in range(2))
    db = torch.full((4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((50 * 64 + 256,), 9, dtype=torch.uint8, device="cuda")
    fp8.fp8_act_grad_experts(g, None, 50, 64, 4, torch.zeros(5, dtype=torch.int32, device="cuda"), 0, 1, ring, 0, out, amax,
                             scale, db)
    assert (db == 0).all() and float(amax) == 0.0 and (out == 9).all()
    bad = torch.tensor([-5, 20, 10, 10, 1 << 30], dtype=torch.int32, device="cuda")  # rows 0..20, none, none, 10..50
    fp8.fp8_act_grad_experts(g, None, 50, 64, 4, bad, 0, 1, ring, 0, out, amax, scale, db)
    assert (out[50 * 64:] == 9).all() and float(amax) == float(g.float().abs().max())
    assert (db[1:3] == 0).all()


def test_refusals_of_experts():
    E, AL, U = fp8.FP8_ERR_INVALID_ARG, fp8.FP8_ERR_ALIGNMENT, fp8.FP8_ERR_UNSUPPORTED

    def status(experts=4, offsets=S + 256, rows=8, cols=64, z=A, ring=S):
        return fp8.raw_status("fp8_act_grad_experts", A, z, rows, cols, experts, offsets, 4, 1, ring, 0, A, None, S + 128,
                              None, None)

    assert status(experts=0) == E and status(offsets=None) == E and status(z=None) == E and status(ring=None) == E
    assert status(rows=-1) == E and status(rows=1 << 31) == E
    assert status(offsets=S + 2) == AL and status(cols=12) == AL
    assert status(experts=513) == U
