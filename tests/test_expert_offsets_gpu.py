"""Offsets that are out of range or decrease mean the same rows to every entry point that takes them: each is limited
to [0, rows] and to no less than the one before. Every value here is a small whole number, so sums are exact."""

import pytest
import torch

import fp8_delayed_scaling_quantize_b200 as fp8

pytestmark = pytest.mark.gpu

ROWS, COLS = 200, 64
ONE = {0: 0x38, 1: 0x3C}  # 1.0 in E4M3 and E5M2


def _random(seed, experts):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-40, ROWS + 60, (experts + 1,), generator=g).tolist()


OFFSETS = {
    "in order": [0, 20, 20, 90, ROWS], "rows of none": [7, 20, 20, 90, 150], "one back": [0, 20, 10, 10, 150],
    "past the ends": [-5, 20, 10, 10, 1 << 30], "all back": [150, 90, 20, 7, 0], "the last back": [0, 50, 180, 60],
    "negative": [-9, -3, -1, -7], "one expert, back": [120, 30], "least and largest": [-(1 << 31), (1 << 31) - 1, 0],
    **{f"random {n}": _random(n, n) for n in (3, 31, 32, 33, 70, 512)},
    "up and down": [v for i in range(60) for v in (3 * i, 3 * i - 2)],
}


def _ranges(off):
    """First and last row of each expert, the rows that have one, and each row's expert (-1: none)."""
    lim, top = [], 0
    for v in off:
        top = max(top, min(max(v, 0), ROWS))
        lim.append(top)
    owner = torch.full((ROWS,), -1, dtype=torch.long)
    for e, (lo, hi) in enumerate(zip(lim, lim[1:])):
        owner[lo:hi] = e
    return list(zip(lim, lim[1:])), owner.cuda()


@pytest.mark.parametrize("name", list(OFFSETS))
def test_rows_of_every_entry_point(name):
    off = OFFSETS[name]
    ranges, owner = _ranges(off)
    E, o = len(off) - 1, torch.tensor(off, dtype=torch.int64).to(torch.int32).cuda()
    counts = torch.tensor([hi - lo for lo, hi in ranges], device="cuda")
    held = owner >= 0
    one = torch.ones(1, device="cuda")

    # the activation gradient: codes of held rows alone, each expert's sum its own rows
    ring, stats = torch.empty(20, dtype=torch.int32, device="cuda"), torch.empty(2, device="cuda")
    fp8.fp8_ring_init(ring, 1.0)
    g = torch.ones(ROWS, COLS, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((ROWS, COLS), 9, dtype=torch.uint8, device="cuda")
    db = torch.full((E, COLS), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_act_grad_experts(g, None, ROWS, COLS, E, o, 0, 1, ring, 0, codes, stats[0:1], stats[1:2], db)
    assert torch.equal(db.float(), counts[:, None].float().expand(E, COLS))
    assert torch.equal(codes, torch.where(held[:, None], ONE[1], 9).to(torch.uint8).expand(ROWS, COLS))

    # forward and input gradient: products of zeros and the expert's own bias, its number
    a, b = torch.zeros(ROWS, COLS, dtype=torch.uint8, device="cuda"), torch.zeros(E, COLS, COLS, dtype=torch.uint8, device="cuda")
    bias = (torch.arange(E, device="cuda") % 256).bfloat16()[:, None].expand(E, COLS).contiguous()
    want = torch.where(held, owner % 256, 333).bfloat16()[:, None].expand(ROWS, COLS)
    for layout in (fp8.FP8_NT, fp8.FP8_NN):
        out = torch.full((ROWS, COLS), 333.0, dtype=torch.bfloat16, device="cuda")
        fp8.fp8_mm_experts(a, 0, b, 0, one, one, 0, layout, ROWS, COLS, COLS, E, o, bias, 0, None, out)
        assert torch.equal(out, want)

    # weight gradient: ones times ones count the rows
    a = torch.full((ROWS, COLS), ONE[1], dtype=torch.uint8, device="cuda")
    b = torch.full((ROWS, COLS), ONE[0], dtype=torch.uint8, device="cuda")
    dw = torch.empty(E, COLS, COLS, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_mm_experts(a, 1, b, 0, one, one, 0, fp8.FP8_TN, COLS, COLS, ROWS, E, o, None, 0, None, dw)
    assert torch.equal(dw.float(), counts[:, None, None].float().expand(E, COLS, COLS))

    # zeros in the other rows, before or after the product
    out = torch.full((ROWS, COLS), 5.0, dtype=torch.bfloat16, device="cuda")
    fp8.fp8_experts_zero_rest(out, ROWS, 2 * COLS, E, o)
    assert torch.equal(out, torch.where(held, 5.0, 0.0).bfloat16()[:, None].expand(ROWS, COLS))
    assert fp8.fp8_last_device_error() == fp8.FP8_OK
