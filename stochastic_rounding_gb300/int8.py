"""A linear layer whose three products run in 8-bit integers.

    y  = x W^T       tokens and weight rows quantised, one scale each, to nearest
    dx = dy W        dy's rows and W's columns
    dw = dy^T x      dy's columns and x's columns

The gradient operand is rounded stochastically, so that what it contributes is
right on average (to within 2^-16 of a step, from 16 random bits); the others to
nearest.  Sums of integers are exact.  Outputs and gradients are bf16, whatever
the inputs' types: the operands hold 8 bits, and what those lose is larger.
The weight itself stays bf16 (or float32) and is what an optimizer of this
package updates.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._lib import asr_linear_int8, asr_linear_int8_grads, asr_quantize_int8, int8_empty


def int8_linear(x, qweight, weight_scale, *, rounding="rne", step: int = 0, seed: int = 0, out=None):
    """``x`` (tokens, k), float32 or bfloat16, times the transpose of an int8
    weight (n, k) with one scale a row: (tokens, n), bfloat16 unless ``out`` says
    otherwise.  ``rounding="sr"`` rounds the outputs stochastically."""
    if out is None:
        out = torch.empty(x.shape[0], qweight.shape[0], dtype=torch.bfloat16, device=x.device)
    return asr_linear_int8(x, qweight, weight_scale, out, rounding=rounding, step=step, seed=seed)


def int8_linear_grads(dy, x, weight, *, step: int = 0, seed: int = 0, need_dx=True, need_dw=True):
    """Gradients of ``y = x weight^T`` from ``dy`` (tokens, n): (dx, dw) in
    bfloat16, either None where it is not needed."""
    dx = torch.empty(x.shape, dtype=torch.bfloat16, device=dy.device) if need_dx else None
    dw = torch.empty(weight.shape, dtype=torch.bfloat16, device=dy.device) if need_dw else None
    asr_linear_int8_grads(dy, x, weight, dx, dw, step=step, seed=seed)
    return dx, dw


def _by_rows(t):
    """``t``, or a copy of it where its rows are not contiguous or overlap."""
    rows, cols = t.shape
    ok = (cols <= 1 or t.stride(1) == 1) and (rows <= 1 or t.stride(0) >= cols)
    return t if ok else t.contiguous()


class _Int8LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, step, seed):
        x, weight = _by_rows(x), _by_rows(weight)
        ctx.save_for_backward(x, weight)
        ctx.key = (step, seed)
        q = int8_empty(*weight.shape, weight.device)
        scale = torch.empty(weight.shape[0], dtype=torch.float32, device=weight.device)
        asr_quantize_int8(weight, q, scale)
        return int8_linear(x, q, scale)

    @staticmethod
    @once_differentiable                    # the calls record nothing: a second derivative through them is an error
    def backward(ctx, dy):
        x, weight = ctx.saved_tensors
        step, seed = ctx.key
        dx, dw = int8_linear_grads(dy.contiguous(), x, weight, step=step, seed=seed, need_dx=ctx.needs_input_grad[0],
                                   need_dw=ctx.needs_input_grad[1])
        return (dx.to(x.dtype) if dx is not None else None, dw.to(weight.dtype) if dw is not None else None, None,
                None)


class Int8Linear(torch.nn.Module):
    """``torch.nn.Linear`` without a bias on the 8-bit products: a bf16 (or
    float32) weight of shape (out_features, in_features), quantised in every
    forward pass.  ``seed`` keys the stochastic rounding of the gradients; it
    is drawn anew for every forward pass that records gradients (``calls``, the
    number of such passes, is the Philox step).  ``calls`` is part of the state
    dict (``_extra_state``), so a run repeats bit for bit, resumed from a checkpoint or
    not; a state dict without it, such as ``torch.nn.Linear``'s, loads too and
    leaves it as it is (the other way, ``torch.nn.Linear`` takes the weight with
    ``strict=False``).

    The random bits of an output gradient's element are those of its index in
    (tokens, out_features), from position 0 on, under (seed, pass).  Layers that share a
    seed share them, as do data-parallel ranks, and an optimizer of that seed
    uses them for its first parameters: give each layer and rank a seed of its
    own where the errors are to be independent."""

    def __init__(self, in_features: int, out_features: int, *, seed: int = 0, device=None, dtype=torch.bfloat16):
        super().__init__()
        self.in_features, self.out_features, self.seed, self.calls = in_features, out_features, int(seed), 0
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features, device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=in_features ** -0.5)

    def forward(self, x):
        if torch.is_grad_enabled() and (x.requires_grad or self.weight.requires_grad):
            self.calls += 1
        flat = x.reshape(-1, self.in_features)
        y = _Int8LinearFunction.apply(flat, self.weight, self.calls, self.seed)
        return y.reshape(*x.shape[:-1], self.out_features)

    def get_extra_state(self):
        return torch.tensor(self.calls, device="cpu")

    def set_extra_state(self, state):
        self.calls = int(state)

    def _load_from_state_dict(self, state_dict, prefix, local_metadata, strict, missing_keys, unexpected_keys,
                              error_msgs):
        super()._load_from_state_dict(state_dict, prefix, local_metadata, strict, missing_keys, unexpected_keys,
                                      error_msgs)
        if prefix + "_extra_state" in missing_keys:
            missing_keys.remove(prefix + "_extra_state")

    def extra_repr(self):
        return f"in_features={self.in_features}, out_features={self.out_features}, seed={self.seed}"
