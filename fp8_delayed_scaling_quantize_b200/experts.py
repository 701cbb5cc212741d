"""FP8 training linear layer of a mixture of experts (torch.autograd).

The rows of the input are sorted by expert: rows [offsets[e], offsets[e+1])
belong to expert e. The offsets stay on the device; nothing is synchronised,
so a layer whose routing changes from step to step can be captured into a CUDA
graph. Each of the layer's products is one launch over all experts
(fp8_mm_experts: forward NT with bias and activation, input gradient NN,
weight gradient TN), and the gradient through the activation is quantized with
the experts' bias gradients in one pass (fp8_act_grad_experts).

Scaling is delayed and per tensor: one ring each for the input, the weights of
all experts and the gradient, kept in `fp8_rings` with the state_dict.
"""

import torch
from torch.autograd.function import once_differentiable

from . import (FP8_ACT_NONE, FP8_E4M3, FP8_E5M2, FP8_MM_MAX_EXPERTS, FP8_NN, FP8_NT, FP8_TN, fp8_act_grad_experts,
               fp8_experts_zero_rest, fp8_mm_experts)
from .linear import Fp8Layer, _act_code, _dense, _on_input, _quantize_many, _rows_of


class Fp8ExpertsFunction(torch.autograd.Function):
    """y[r] = act(x[r] W[e]^T + b[e]) for the rows r of expert e; rows of no
    expert give zeros and get zero gradients."""

    @staticmethod
    def forward(ctx, x, offsets, weight, bias, rings, act, learn=True):
        E, N, K = weight.shape
        x2 = _rows_of(x, K, "input")
        if x.dim() != 2:
            raise ValueError("experts take token-sorted rows [T, features]")
        if offsets.dtype != torch.int32 or offsets.shape != (E + 1,) or offsets.device != x.device:
            raise ValueError(f"offsets must be int32 [{E + 1}] on the input's device")
        T, dev = x2.shape[0], x.device
        offsets = offsets.contiguous()
        (x8, sx), (w8, sw) = _quantize_many([(x2, FP8_E4M3, rings[0]), (_dense(weight), FP8_E4M3, rings[1])], dev)
        y = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
        fp8_experts_zero_rest(y, T, 2 * N, E, offsets)
        z = None
        if act != FP8_ACT_NONE and learn and (ctx.needs_input_grad[0] or any(ctx.needs_input_grad[2:4])):
            z = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
        b = bias.contiguous() if bias is not None else None
        fp8_mm_experts(x8, FP8_E4M3, w8, FP8_E4M3, sx, sw, 0, FP8_NT, T, N, K, E, offsets, b, act, z, y)
        ctx.save_for_backward(x8, w8, sx, sw, rings, offsets, z)
        ctx.dims, ctx.act, ctx.has_bias = (T, N, K, E), act, bias is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        x8, w8, sx, sw, rings, offsets, z = ctx.saved_tensors
        T, N, K, E = ctx.dims
        need_x, need_w, need_b = ctx.needs_input_grad[0], ctx.needs_input_grad[2], ctx.needs_input_grad[3]
        dx = dw = db = None
        dev = gy.device
        g2 = _dense(gy.to(torch.bfloat16))
        g8 = torch.empty(T * N, dtype=torch.uint8, device=dev)
        stats = torch.empty(2, dtype=torch.float32, device=dev)
        if need_b and ctx.has_bias:
            db = torch.empty(E, N, dtype=torch.bfloat16, device=dev)
        fp8_act_grad_experts(g2, z, T, N, E, offsets, ctx.act, FP8_E5M2, rings[2], 0, g8, stats[0:1], stats[1:2], db)
        sg = stats[1:2]
        if need_x:
            dx = torch.empty(T, K, dtype=torch.bfloat16, device=dev)
            fp8_experts_zero_rest(dx, T, 2 * K, E, offsets)
            fp8_mm_experts(g8, FP8_E5M2, w8, FP8_E4M3, sg, sw, 0, FP8_NN, T, K, N, E, offsets, None, FP8_ACT_NONE, None, dx)
        if need_w:
            dw = torch.empty(E, N, K, dtype=torch.bfloat16, device=dev)
            fp8_mm_experts(g8, FP8_E5M2, x8, FP8_E4M3, sg, sx, 0, FP8_TN, N, K, T, E, offsets, None, FP8_ACT_NONE, None, dw)
        return dx, None, dw, db, None, None, None


class Fp8Experts(Fp8Layer):
    """The linears of `experts` experts (bf16 parameters, FP8 compute).

    in_features and out_features must be multiples of 16, experts at most
    FP8_MM_MAX_EXPERTS (512). forward(x, offsets):
    x bf16 [T, in_features] sorted by expert, offsets int32 [experts + 1] on the
    same device. activation as Fp8Linear's. Rows of no expert give zeros; their
    input values still count for the input's scale.
    """

    def __init__(self, experts, in_features, out_features, bias=True, device=None, activation=None):
        super().__init__()
        if in_features % 16 or out_features % 16:
            raise ValueError("Fp8Experts needs in_features and out_features divisible by 16")
        if not 1 <= experts <= FP8_MM_MAX_EXPERTS:
            raise ValueError(f"Fp8Experts takes 1 to {FP8_MM_MAX_EXPERTS} experts, not {experts}")
        self.experts, self.in_features, self.out_features = experts, in_features, out_features
        self.activation = activation
        self._act = _act_code(activation)
        kw = {"device": device, "dtype": torch.bfloat16}
        self.weight = torch.nn.Parameter(torch.empty(experts, out_features, in_features, **kw))
        self.bias = torch.nn.Parameter(torch.zeros(experts, out_features, **kw)) if bias else None
        self._make_rings(device)
        torch.nn.init.normal_(self.weight, std=in_features ** -0.5)

    def forward(self, x, offsets):
        rings, weight, bias = self.fp8_rings, self.weight, self.bias
        with _on_input(x, rings, weight, bias):
            if not self._rings_ready:
                self.reset_scaling()
            return Fp8ExpertsFunction.apply(x, offsets, weight, bias, rings, self._act, torch.is_grad_enabled())
