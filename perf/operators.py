"""What is measured of the operators around the FP8 GEMM: products with bias, activation and residual in their
epilogue, the gradient through that activation as it is quantized, and products grouped by expert.

`own` says which side `run` computes: the plain form, in elementary torch operations on fp32 values, or the library's
entry points on the same buffers. The operands of every product are FP8 codes with the scale that they were
quantized with, as a training step or a server holds them between a quantize and a GEMM.
"""

import math
import random

import torch

own = False

E4M3, E5M2 = 0, 1
NT, NN, TN = 0, 1, 2
NONE, RELU, GELU, GELU_TANH, SILU = 0, 1, 2, 3, 4
FMAX = {E4M3: 448.0, E5M2: 57344.0}
F8 = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}


def listed():
    return [
        # the MLP's first linear of a dim-1024 layer at 2048 tokens: GELU, its input kept for the backward pass, the
        # output as FP8 codes under a delayed ring, ready for the second linear
        dict(name="mlp_up_gelu_out8", op="mm_act", layout=NT, M=2048, N=4096, K=1024, act=GELU_TANH, residual=False,
             preact=True, out8=True, bias=True),
        # its second linear: bias and the residual stream added before the one rounding
        dict(name="mlp_down_residual", op="mm_act", layout=NT, M=2048, N=1024, K=4096, act=NONE, residual=True,
             preact=False, out8=False, bias=True),
        # one token of a served model: the smallest call, bound by latency and by reading the weight
        dict(name="one_token_silu", op="mm_act", layout=NT, M=1, N=4096, K=4096, act=SILU, residual=True,
             preact=False, out8=False, bias=True),
        # the backward pass of a residual branch: dX = g W + g_residual, a ragged token count, E5M2 x E4M3
        dict(name="dx_residual_ragged", op="mm_act", layout=NN, M=1001, N=1040, K=2064, act=NONE, residual=True,
             preact=False, out8=False, bias=False),
        # the largest product
        dict(name="square_8192_relu", op="mm_act", layout=NT, M=8192, N=8192, K=8192, act=RELU, residual=True,
             preact=False, out8=False, bias=True),
        # gradient through the GELU of the MLP above, its E5M2 codes for dX and dW, and the bias gradient
        dict(name="grad_gelu_mlp", op="act_grad", rows=2048, cols=4096, act=GELU_TANH, dbias=True),
        # the same of a long batch with SiLU
        dict(name="grad_silu_long", op="act_grad", rows=32768, cols=4096, act=SILU, dbias=True),
        # a few odd rows, as the last micro-batch of an epoch leaves them
        dict(name="grad_gelu_few", op="act_grad", rows=37, cols=1040, act=GELU, dbias=True),
        # 2048 tokens sent to 8 of 32 experts each: the experts' first product, forward
        dict(name="experts_up_silu", op="experts", layout=NT, rows=16384, d1=4096, d2=1024, experts=32, act=SILU,
             bias=True, preact=True, skew=1.0, behind=0),
        # its input gradient
        dict(name="experts_dx", op="experts", layout=NN, rows=16384, d1=1024, d2=4096, experts=32, act=NONE,
             bias=False, preact=False, skew=1.0, behind=0),
        # its weight gradient: the ragged rows are summed over, some experts have none
        dict(name="experts_dw", op="experts", layout=TN, rows=16384, d1=4096, d2=1024, experts=32, act=NONE,
             bias=False, preact=False, skew=1.0, behind=0),
        # a decoding step of 8 sequences, 8 of 64 experts each: one row or none for most experts, rows behind the last
        dict(name="experts_decode", op="experts", layout=NT, rows=80, d1=2048, d2=1024, experts=64, act=SILU,
             bias=True, preact=False, skew=0.5, behind=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["mm_act", "mm_act", "act_grad", "experts", "experts"])
    if op == "mm_act":
        layout = rng.choice([NT, NT, NN])
        while True:
            M, N, K = _log(rng, 1, 8192), 16 * _log(rng, 8, 512), 16 * _log(rng, 8, 512)
            if M * N * K <= 8192 ** 3 // 4:
                break
        out8 = rng.random() < 0.3
        return dict(op=op, layout=layout, M=M, N=N, K=K, act=rng.choice([NONE, RELU, GELU, GELU_TANH, SILU]),
                    residual=not out8 and rng.random() < 0.6, preact=rng.random() < 0.4, out8=out8,
                    bias=rng.random() < 0.7)
    if op == "act_grad":
        return dict(op=op, rows=_log(rng, 1, 32768), cols=8 * _log(rng, 8, 512),
                    act=rng.choice([RELU, GELU, GELU_TANH, SILU]), dbias=rng.random() < 0.8)
    layout, behind = rng.choice([NT, NT, NN, TN]), rng.choice([0, 0, 3])
    while True:
        rows, d1, d2 = _log(rng, 1, 32768), 16 * _log(rng, 16, 256), 16 * _log(rng, 16, 256)
        experts = _log(rng, 2, 128)
        if rows * d1 * d2 <= 16384 * 4096 * 1024 and experts * d1 * d2 <= 1 << 28:
            break
    behind = min(behind, rows - 1)
    if layout == TN:
        return dict(op=op, layout=layout, rows=rows, d1=d1, d2=d2, experts=experts, act=NONE, bias=False,
                    preact=False, skew=rng.choice([0.0, 0.5, 1.0]), behind=behind)
    return dict(op=op, layout=layout, rows=rows, d1=d1, d2=d2, experts=experts, act=rng.choice([NONE, GELU, SILU]),
                bias=rng.random() < 0.5, preact=rng.random() < 0.3, skew=rng.choice([0.0, 0.5, 1.0]),
                behind=behind)


# ------------------------------------------------------------------------------------------------ inputs ---


def _codes(gen, shape, fmt):
    """Codes of a normal tensor whose largest value is near the format's maximum, and the format's share of it: what
    a delayed quantize leaves (amax at about 5 standard deviations)."""
    v = torch.randn(shape, generator=gen, device="cuda") * (FMAX[fmt] / 5.0)
    return v.clamp_(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8)


def _bf16(gen, shape, std):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _scale(std, fmt):
    return torch.full((1,), FMAX[fmt] / (5.0 * std), dtype=torch.float32, device="cuda")


def _ring(gen, amax):
    """A delayed-scaling ring in use: 16 amaxes near `amax`, the scale that they give, the next slot."""
    hist = amax * (0.5 + torch.rand(16, generator=gen, device="cuda"))
    ring = torch.zeros(20, dtype=torch.int32, device="cuda")
    ring[:16] = hist.view(torch.int32)
    return ring


def _offsets(case, seed):
    """Rows of each expert: tokens choose experts with unequal odds (skew 0: equal), one expert in eight gets none;
    `behind` rows come after the last expert's."""
    g = torch.Generator().manual_seed(seed)
    E, n = case["experts"], max(0, case["rows"] - case["behind"])
    w = torch.exp(case["skew"] * torch.randn(E, generator=g, dtype=torch.float64))
    w = w * (torch.rand(E, generator=g) >= 0.125)
    if float(w.sum()) == 0.0:
        w[0] = 1.0
    edge = torch.cat([torch.zeros(1, dtype=torch.float64), (w / w.sum()).cumsum(0)])
    cut = torch.bincount(torch.bucketize(torch.rand(n, generator=g, dtype=torch.float64), edge[1:-1], right=True),
                         minlength=E) if E > 1 else torch.tensor([n])
    return torch.cat([torch.zeros(1, dtype=torch.long), cut.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    x_std, w_std, g_std = 1.0, 0.02, 1e-3
    if op == "mm_act":
        M, N, K = case["M"], case["N"], case["K"]
        s["fa"], a_std = (E4M3, x_std) if case["layout"] == NT else (E5M2, g_std)
        s["a8"], s["sa"] = _codes(gen, (M, K), s["fa"]), _scale(a_std, s["fa"])
        s["b8"], s["sb"] = _codes(gen, (N, K) if case["layout"] == NT else (K, N), E4M3), _scale(w_std, E4M3)
        std = a_std * w_std * math.sqrt(K)
        s["bias_t"] = _bf16(gen, (N,), 0.1 * std) if case["bias"] else None
        s["residual_t"] = _bf16(gen, (M, N), std) if case["residual"] else None
        s["preact_t"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda") if case["preact"] else None
        if case["out8"]:
            s["ring"] = _ring(gen, 5.0 * std)
            s["ring"][16:17] = (FMAX[E4M3] / s["ring"][:16].view(torch.float32).max()).view(1).view(torch.int32)
            s["ring"][17] = seed % 16
            s["out8_t"] = torch.empty(M, N, dtype=torch.uint8, device="cuda")
            s["stats"] = torch.empty(2, dtype=torch.float32, device="cuda")
            s["amax_t"], s["scale_t"] = s["stats"][0:1], s["stats"][1:2]
        else:
            s["out_t"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    elif op == "act_grad":
        rows, cols = case["rows"], case["cols"]
        s["g"], s["z"] = _bf16(gen, (rows, cols), g_std), _bf16(gen, (rows, cols), 0.7)
        s["ring"] = _ring(gen, 5.0 * g_std)
        s["ring"][16:17] = (FMAX[E5M2] / s["ring"][:16].view(torch.float32).max()).view(1).view(torch.int32)
        s["ring"][17] = seed % 16
        s["out8_t"] = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
        s["stats"] = torch.empty(2, dtype=torch.float32, device="cuda")
        s["amax_t"], s["scale_t"] = s["stats"][0:1], s["stats"][1:2]
        s["dbias_t"] = torch.empty(cols, dtype=torch.bfloat16, device="cuda") if case["dbias"] else None
    else:
        T, d1, d2, E = case["rows"], case["d1"], case["d2"], case["experts"]
        off = _offsets(case, seed)
        s["offsets"] = off.cuda()
        s["cap"] = int((off[1:] - off[:-1]).max())  # the plain form's padding; the kernels read the offsets alone
        if case["layout"] == TN:
            s["fa"] = E5M2
            s["a8"], s["sa"] = _codes(gen, (T, d1), E5M2), _scale(g_std, E5M2)
            s["b8"], s["sb"] = _codes(gen, (T, d2), E4M3), _scale(x_std, E4M3)
            s["out_t"] = torch.empty(E, d1, d2, dtype=torch.bfloat16, device="cuda")
        else:
            s["fa"], a_std = (E4M3, x_std) if case["layout"] == NT else (E5M2, g_std)
            s["a8"], s["sa"] = _codes(gen, (T, d2), s["fa"]), _scale(a_std, s["fa"])
            s["b8"] = _codes(gen, (E, d1, d2) if case["layout"] == NT else (E, d2, d1), E4M3)
            s["sb"] = _scale(w_std, E4M3) * (0.5 + torch.rand(E, generator=gen, device="cuda"))
            s["bias_t"] = _bf16(gen, (E, d1), 0.1) if case["bias"] else None
            s["out_t"] = _bf16(gen, (T, d1), 1.0)  # rows behind the last expert keep what they hold
            s["preact_t"] = _bf16(gen, (T, d1), 1.0) if case["preact"] else None
    return s


# ------------------------------------------------------------------------------------------- plain forms ---


def _val(codes, fmt):
    return codes.view(F8[fmt]).float()


def _act(z, act):
    if act == RELU:
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == GELU:
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == GELU_TANH:
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == SILU:
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == RELU:
        return (z > 0).to(z.dtype)
    if act == GELU:
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == GELU_TANH:
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == SILU:
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    return torch.ones_like(z)


def _quantize(s, y, fmt):
    """Codes of y under the ring's scale, then y's amax folded into the ring."""
    hist, scale = s["ring"][:16].view(torch.float32), s["ring"][16:17].view(torch.float32)
    s["scale_t"].copy_(scale)
    s["amax_t"].copy_(y.abs().amax().view(1))
    q = (y * scale).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])
    hist.index_copy_(0, s["ring"][17:18].long(), s["amax_t"])
    top = hist.amax().view(1)
    scale.copy_(torch.where((top > 0) & torch.isfinite(top), torch.full_like(top, FMAX[fmt]) / top, scale))
    s["ring"][17] = (s["ring"][17] + 1) % 16
    return q


def _ring_out(s):
    return [s["ring"][:17].view(torch.float32), s["ring"][17:18], s["amax_t"], s["scale_t"]]


def _plain_mm_act(s):
    b = _val(s["b8"], E4M3)
    acc = _val(s["a8"], s["fa"]) @ (b.t() if s["layout"] == NT else b)
    z = acc / (s["sa"] * s["sb"])
    if s["bias"]:
        z = z + s["bias_t"].float()
    y = _act(z, s["act"])
    if s["residual"]:
        y = y + s["residual_t"].float()
    pre = z.to(torch.bfloat16) if s["preact"] else None
    if s["out8"]:
        return {"codes": _quantize(s, y, E4M3), "preact": pre, "ring": _ring_out(s)}
    return {"out": y.to(torch.bfloat16), "preact": pre}


def _plain_act_grad(s):
    dz = s["g"].float() * _act_grad(s["z"].float(), s["act"])
    db = dz.sum(0).to(torch.bfloat16) if s["dbias"] else None
    return {"codes": _quantize(s, dz, E5M2), "dbias": db, "ring": _ring_out(s)}


def _plain_experts(s):
    off, E, cap, T = s["offsets"].long(), s["experts"], max(1, s["cap"]), s["rows"]
    row = torch.arange(T, device="cuda")
    e = torch.bucketize(row, off[1:], right=True).clamp_(max=E - 1)
    held = ((row >= off[0]) & (row < off[-1])).unsqueeze(1)
    at = torch.where(held.squeeze(1), e * cap + row - off[e], torch.full_like(row, E * cap))  # the last row: a bin

    def padded(v):
        p = torch.zeros(E * cap + 1, v.shape[1], device="cuda")
        p.index_copy_(0, at, torch.where(held, v, torch.zeros_like(v)))
        return p[:E * cap].view(E, cap, v.shape[1])

    if s["layout"] == TN:
        acc = torch.bmm(padded(_val(s["a8"], s["fa"])).transpose(1, 2), padded(_val(s["b8"], E4M3)))
        return {"out": (acc / (s["sa"] * s["sb"])).to(torch.bfloat16)}
    b = _val(s["b8"], E4M3)
    z = torch.bmm(padded(_val(s["a8"], s["fa"])), b.transpose(1, 2) if s["layout"] == NT else b)
    z = z / (s["sa"] * s["sb"]).view(E, 1, 1)
    if s["bias"]:
        z = z + s["bias_t"].float().unsqueeze(1)
    at = at.clamp(max=E * cap - 1)
    z = z.view(E * cap, -1)[at]
    out = torch.where(held, _act(z, s["act"]).to(torch.bfloat16), s["out_t"])
    pre = torch.where(held, z.to(torch.bfloat16), s["preact_t"]) if s["preact"] else None
    return {"out": out, "preact": pre}


# ---------------------------------------------------------------------------------------------- the calls ---


def _own_mm_act(s):
    import fp8_delayed_scaling_quantize_b200 as fp8
    if s["out8"]:
        fp8.fp8_mm_act_out8(s["a8"], s["fa"], s["b8"], E4M3, s["sa"], s["sb"], s["layout"], s["M"], s["N"], s["K"], 1,
                            0, 0, 0, s["bias_t"], None, 0, s["act"], s["preact_t"], E4M3, s["ring"], s["out8_t"],
                            s["amax_t"], s["scale_t"])
        return {"codes": s["out8_t"].view(F8[E4M3]), "preact": s["preact_t"], "ring": _ring_out(s)}
    fp8.fp8_mm_act(s["a8"], s["fa"], s["b8"], E4M3, s["sa"], s["sb"], s["layout"], s["M"], s["N"], s["K"], 1, 0, 0, 0,
                   s["bias_t"], None, 0, s["act"], s["residual_t"], 0, s["preact_t"], s["out_t"])
    return {"out": s["out_t"], "preact": s["preact_t"]}


def _own_act_grad(s):
    import fp8_delayed_scaling_quantize_b200 as fp8
    fp8.fp8_act_grad(s["g"], s["z"], s["rows"], s["cols"], s["act"], E5M2, s["ring"], 0, s["out8_t"], s["amax_t"],
                     s["scale_t"], s["dbias_t"])
    return {"codes": s["out8_t"].view(F8[E5M2]), "dbias": s["dbias_t"], "ring": _ring_out(s)}


def _own_experts(s):
    import fp8_delayed_scaling_quantize_b200 as fp8
    T, d1, d2 = s["rows"], s["d1"], s["d2"]
    if s["layout"] == TN:
        fp8.fp8_mm_experts(s["a8"], s["fa"], s["b8"], E4M3, s["sa"], s["sb"], 0, TN, d1, d2, T, s["experts"],
                           s["offsets"], None, NONE, None, s["out_t"])
        return {"out": s["out_t"]}
    fp8.fp8_mm_experts(s["a8"], s["fa"], s["b8"], E4M3, s["sa"], s["sb"], 1, s["layout"], T, d1, d2, s["experts"],
                       s["offsets"], s["bias_t"], s["act"], s["preact_t"], s["out_t"])
    return {"out": s["out_t"], "preact": s["preact_t"]}


def run(state):
    op = state["op"]
    if own:
        return {"mm_act": _own_mm_act, "act_grad": _own_act_grad, "experts": _own_experts}[op](state)
    return {"mm_act": _plain_mm_act, "act_grad": _plain_act_grad, "experts": _plain_experts}[op](state)


# ------------------------------------------------------------------------------------------- definitions ---


def _exact_ring(s, y, fmt):
    """What a delayed quantize leaves: the values before their rounding to codes, the ring, amax and scale. E5M2 has
    none for its codes: its steps of a quarter alone are 5 % of the result, so the value before them says little."""
    hist, scale = s["ring"][:16].view(torch.float32).double(), s["ring"][16:17].view(torch.float32).double()
    idx = int(s["ring"][17])
    amax = y.abs().max()
    q = torch.minimum(torch.maximum(y * scale, torch.full_like(y, -FMAX[fmt])), torch.full_like(y, FMAX[fmt]))
    hist[idx] = amax
    after = torch.cat([hist, (FMAX[fmt] / hist.max()).view(1)])
    return q if fmt == E4M3 else None, [after, torch.tensor([(idx + 1) % 16], dtype=torch.int32), amax.view(1), scale]


def _exact_act(z, act):
    if act == RELU:
        return z.clamp(min=0)
    if act == GELU:
        return z * torch.special.ndtr(z)
    if act == GELU_TANH:
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == SILU:
        return z * torch.sigmoid(z)
    return z


def _exact_slope(z, act):
    z = z.clone().requires_grad_(True)
    return torch.autograd.grad(_exact_act(z, act).sum(), z)[0]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    dec = lambda c, f: c.view(F8[f]).double()  # noqa: E731
    if op == "mm_act":
        w = dec(s["b8"], E4M3)
        z = torch.matmul(dec(s["a8"], s["fa"]), w.T if case["layout"] == NT else w) / (s["sa"].double() * s["sb"].double())
        if case["bias"]:
            z += s["bias_t"].double()
        y = _exact_act(z, case["act"])
        if case["residual"]:
            y = y + s["residual_t"].double()
        pre = z if case["preact"] else None
        if case["out8"]:
            q, ring = _exact_ring(s, y, E4M3)
            return {"codes": q, "preact": pre, "ring": ring}
        return {"out": y, "preact": pre}
    if op == "act_grad":
        dz = s["g"].double() * _exact_slope(s["z"].double(), case["act"])
        q, ring = _exact_ring(s, dz, E5M2)
        return {"codes": q, "dbias": dz.sum(0) if case["dbias"] else None, "ring": ring}
    off = s["offsets"].tolist()
    k = s["sa"].double() * s["sb"].double()
    if case["layout"] == TN:
        out = torch.zeros(case["experts"], case["d1"], case["d2"], dtype=torch.float64, device="cuda")
        for i, (lo, hi) in enumerate(zip(off, off[1:])):
            out[i] = torch.matmul(dec(s["a8"][lo:hi], s["fa"]).T, dec(s["b8"][lo:hi], E4M3)) / k
        return {"out": out}
    out, pre = s["out_t"].double(), s["preact_t"].double() if case["preact"] else None
    for i, (lo, hi) in enumerate(zip(off, off[1:])):
        w = dec(s["b8"][i], E4M3)
        z = torch.matmul(dec(s["a8"][lo:hi], s["fa"]), w.T if case["layout"] == NT else w) / k[i]
        if case["bias"]:
            z += s["bias_t"][i].double()
        out[lo:hi] = _exact_act(z, case["act"])
        if case["preact"]:
            pre[lo:hi] = z
    return {"out": out, "preact": pre}


def work(case):
    if case["op"] == "mm_act":
        M, N, K = case["M"], case["N"], case["K"]
        n = M * K + N * K + M * N * ((1 if case["out8"] else 2) + 2 * case["residual"] + 2 * case["preact"])
        return {"bytes": n + 2 * N * case["bias"], "flops": 2 * M * N * K}
    if case["op"] == "act_grad":
        n = case["rows"] * case["cols"]
        return {"bytes": 5 * n + 2 * case["cols"] * case["dbias"], "flops": 12 * n}
    T, d1, d2, E = max(0, case["rows"] - case["behind"]), case["d1"], case["d2"], case["experts"]
    if case["layout"] == TN:
        return {"bytes": T * (d1 + d2) + 2 * E * d1 * d2, "flops": 2 * T * d1 * d2}
    read = min(T, E - E // 8)  # experts that have rows: their weights alone are read
    return {"bytes": T * d2 + read * d1 * d2 + T * d1 * (2 + 2 * case["preact"]), "flops": 2 * T * d1 * d2}
