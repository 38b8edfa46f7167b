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

from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import asr_linear_int8, asr_linear_int8_grads, asr_quantize_int8, int8_empty


class Int8Checkpoint(NamedTuple):
    """A matrix kept in 8 bits.  A row of ``data`` (uint8) holds its codes, up to a
    multiple of 16 bytes, and behind them the power of two (plus 127) of each 32 of its
    values."""
    data: torch.Tensor
    cols: int
    dtype: torch.dtype                      # of what it was made from

    @property
    def q(self):
        """The codes: int8, the matrix's shape."""
        return self.data.view(torch.int8)[:, :self.cols]

    @property
    def power(self):
        at = (self.cols + 15) // 16 * 16
        return self.data[:, at:at + (self.cols + _lib.CHECKPOINT_GROUP - 1) // _lib.CHECKPOINT_GROUP]

    def _struct(self, *key):
        """For the library, with the key of its rounding where it is made."""
        p, ld = self.data.data_ptr(), self.data.shape[1]
        return _lib._pack_checkpoint(p, p + (self.cols + 15) // 16 * 16, ld, ld, *key)


def empty_checkpoint(rows: int, cols: int, device, dtype) -> Int8Checkpoint:
    """An uninitialised checkpoint of a rows x cols matrix."""
    width = (cols + 15) // 16 * 16 + ((cols + 31) // 32 + 15) // 16 * 16
    return Int8Checkpoint(torch.empty((rows, width), dtype=torch.uint8, device=device), cols, dtype)


# The functions that return new tensors check what they are given and call the library
# themselves: going through the calls that fill a caller's tensors would check the new
# ones too, and cost as much again as the launch.  For small tensors the host's time is
# the call's: a launch 3 us, an allocation beside it 3 to 5.

_FLOATS = (torch.bfloat16, torch.float32)


def _elsewhere(device: int) -> bool:
    """Whether a CUDA device is not the current one."""
    return device != _get_device()


def _python_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _python_stream


def checkpoint_int8(x, *, rounding="rne", base_index: int = 0, step: int = 0, seed: int = 0) -> Int8Checkpoint:
    """``x`` (2-D, float32 or bfloat16) kept in 8 bits for a backward pass: 32 values
    of a row share a power of two.  ``rounding="sr"`` rounds stochastically, so that
    what is read back is x on average (to within 2^-16 of a step)."""
    px, rows, cols, ld, code, d = _lib._rows_of(x, "x")
    _lib._check_rounding(rounding)
    if _elsewhere(d):
        with torch.cuda.device(d):
            return checkpoint_int8(x, rounding=rounding, base_index=base_index, step=step, seed=seed)
    c = empty_checkpoint(rows, cols, x.device, x.dtype)
    _lib._check(_lib.lib().asr_checkpoint_int8(px, code, rows, cols, ld, c._struct(rounding, base_index, step, seed),
                                               _raw_stream(d)), "asr_checkpoint_int8")
    return c


def _checked(c: Int8Checkpoint, rows, cols, device):
    """The C struct of a checkpoint that a caller gives."""
    t, n = c.data, c.cols
    if not t.is_cuda or t.dtype != torch.uint8 or t.dim() != 2 or not t.is_contiguous():
        raise ValueError("a checkpoint's data must be a contiguous 2-D uint8 CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"the checkpoint is on {t.device}; the call's other tensors are on cuda:{device}")
    have, width = t.shape
    at = (n + 15) // 16 * 16
    if n != cols or have != rows or width != at + ((n + 31) // 32 + 15) // 16 * 16:
        raise ValueError(f"a checkpoint of {(rows, cols)} is wanted, not of {(have, n)} in {tuple(t.shape)}")
    p = t.data_ptr()
    return _lib._pack_checkpoint(p, p + at, width, width)


def restore_int8(checkpoint: Int8Checkpoint, dtype=None):
    """The values that a checkpoint stands for, in ``dtype`` (the original's unless given); exact in either."""
    if not isinstance(checkpoint, Int8Checkpoint):
        raise TypeError(f"an Int8Checkpoint is wanted, not {type(checkpoint).__name__}")
    dtype = dtype or checkpoint.dtype
    if dtype not in _FLOATS:
        raise TypeError(f"values come as float32 or bfloat16, not {dtype}")
    t, cols = checkpoint.data, checkpoint.cols
    rows, d = t.shape[0], t.get_device()
    s = _checked(checkpoint, rows, cols, d)
    if _elsewhere(d):
        with torch.cuda.device(d):
            return restore_int8(checkpoint, dtype)
    out = torch.empty((rows, cols), dtype=dtype, device=t.device)
    _lib._check(_lib.lib().asr_restore_int8(s, rows, cols, out.data_ptr(), _lib._dt(out), cols, _raw_stream(d)),
                "asr_restore_int8")
    return out


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
    def forward(ctx, x, weight, step, seed, save):
        x, weight = _by_rows(x), _by_rows(weight)
        ctx.key, ctx.x_dtype, ctx.save = (step, seed), x.dtype, save
        if save == "int8" and ctx.needs_input_grad[1]:
            ctx.save_for_backward(weight, checkpoint_int8(x, rounding="sr", step=step, seed=seed).data)
        elif save == "int8":                # dx does not read x
            ctx.save_for_backward(weight)
        elif save:
            ctx.save_for_backward(weight, x)
        q = int8_empty(*weight.shape, weight.device)
        scale = torch.empty(weight.shape[0], dtype=torch.float32, device=weight.device)
        asr_quantize_int8(weight, q, scale)
        return int8_linear(x, q, scale)

    @staticmethod
    @once_differentiable                    # the calls record nothing: a second derivative through them is an error
    def backward(ctx, dy):
        weight, *x = ctx.saved_tensors
        step, seed = ctx.key
        dy = dy.contiguous()
        need_dx, need_dw = ctx.needs_input_grad[:2]
        if not x:
            x = dy.new_empty(dy.shape[0], weight.shape[1])
        elif ctx.save == "int8":            # what 8 bits stand for is exact in bf16
            x = restore_int8(Int8Checkpoint(x[0], weight.shape[1], torch.bfloat16))
        else:
            x = x[0]
        dx, dw = int8_linear_grads(dy, x, weight, step=step, seed=seed, need_dx=need_dx, need_dw=need_dw)
        return (dx.to(ctx.x_dtype) if dx is not None else None, dw.to(weight.dtype) if dw is not None else None, None,
                None, None)


class _CountedModule(torch.nn.Module):
    """A module whose passes that record gradients are counted: ``calls`` is the
    Philox step of what a pass rounds stochastically, and part of the state dict
    (``_extra_state``), so that a run repeats bit for bit, resumed from a checkpoint or
    not.  A state dict without it loads too and leaves the count as it is."""

    def __init__(self, seed: int):
        super().__init__()
        self.seed, self.calls = int(seed), 0

    def _count(self, *tensors):
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
            self.calls += 1
            return True
        return False

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


class Int8Linear(_CountedModule):
    """``torch.nn.Linear`` without a bias on the 8-bit products: a bf16 (or
    float32) weight of shape (out_features, in_features), quantised in every
    forward pass.  ``seed`` keys the stochastic rounding of the gradients; it
    is drawn anew for every forward pass that records gradients (``calls``, the
    number of such passes, is the Philox step).  ``calls`` is part of the state
    dict (``_extra_state``), so a run repeats bit for bit, resumed from a checkpoint or
    not; a state dict without it, such as ``torch.nn.Linear``'s, loads too and
    leaves it as it is (the other way, ``torch.nn.Linear`` takes the weight with
    ``strict=False``).

    ``save="int8"`` keeps the input in 8 bits for the backward pass, rounded
    stochastically, in place of the input itself: a little over half of a bf16
    input's memory, and a weight's gradient that is right on average.  The forward pass
    reads the input once more for it, and the backward pass restores the whole input in
    bf16 for as long as its products take (a step of 8,192 tokens of 4,096 x 4,096 bf16:
    695 us, 653 with the input itself).

    The random bits of an output gradient's element are those of its index in
    (tokens, out_features), from position 0 on, under (seed, pass).  Layers that share a
    seed share them, as do data-parallel ranks, and an optimizer of that seed
    uses them for its first parameters: give each layer and rank a seed of its
    own where the errors are to be independent.  (The kept input's are others, but
    also shared by layers of one seed.)"""

    def __init__(self, in_features: int, out_features: int, *, seed: int = 0, device=None, dtype=torch.bfloat16,
                 save: str = "input"):
        if save not in ("input", "int8"):
            raise ValueError(f"save must be 'input' or 'int8', not {save!r}")
        super().__init__(seed)
        self.in_features, self.out_features, self.save = in_features, out_features, save
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features, device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=in_features ** -0.5)

    def forward(self, x):
        save = self.save if self._count(x, self.weight) else None
        flat = x.reshape(-1, self.in_features)
        y = _Int8LinearFunction.apply(flat, self.weight, self.calls, self.seed, save)
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self):
        return (f"in_features={self.in_features}, out_features={self.out_features}, seed={self.seed}" +
                ("" if self.save == "input" else f", save={self.save!r}"))
