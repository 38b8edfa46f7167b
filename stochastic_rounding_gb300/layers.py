"""What stands between a layer's 8-bit products: the norm, the activation and the
embedding, forward and backward, their inputs kept for the backward pass as they are
or in 8 bits (``checkpoint_int8`` in ``stochastic_rounding_gb300.int8``).

The functions work on 2-D tensors whose rows are contiguous and return new ones; the
modules take any shape and layout, record gradients, and hold parameters for this
package's optimizers.  Nothing here has a second derivative.

A pass that is kept in 8 bits and rounded stochastically takes its random numbers from
(seed, step), the same for every call with these: modules count their passes (``calls``)
and go on counting from a state dict.  These numbers are not an optimizer's, nor those
of ``Int8Linear``'s gradients, whatever the seed; modules that share a seed share them.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Union

import torch
from torch.autograd.function import once_differentiable

from ._lib import (asr_activation, asr_activation_grads, asr_embedding, asr_embedding_grads, asr_layer_norm,
                   asr_layer_norm_grads)
from .int8 import Int8Checkpoint, _by_rows, _CountedModule, empty_checkpoint

_SAVE = (None, "input", "int8")


def _check_save(save, allowed=_SAVE):
    if save not in allowed:
        raise ValueError(f"save must be one of {allowed}, not {save!r}")


# -------------------------------------------------------------- activation


def activation(x, function="silu", *, gated=False, save=None, rounding="rne", step: int = 0, seed: int = 0):
    """f(x) for ``x`` (rows, columns), or, ``gated``, f of its first half of columns
    times its second half.  ``function``: "silu", or "gelu" (its tanh form).  With
    ``save`` returns (y, saved) for ``activation_grads``: "input" saves x itself,
    "int8" its 8-bit checkpoint, made in the same pass."""
    _check_save(save)
    rows, width = x.shape
    if gated and width % 2:
        raise ValueError(f"a gated activation takes an even number of columns, not {width}")
    y = torch.empty(rows, width // 2 if gated else width, dtype=x.dtype, device=x.device)
    kept = empty_checkpoint(rows, width, x.device, x.dtype) if save == "int8" else None
    asr_activation(x, y, function, gated=gated, keep=kept, rounding=rounding, step=step, seed=seed)
    return y if save is None else (y, x if kept is None else kept)


def activation_grads(dy, saved: Union[torch.Tensor, Int8Checkpoint], function="silu", *, gated=False):
    """dx from ``dy`` and what ``activation`` saved."""
    kept = saved if isinstance(saved, Int8Checkpoint) else None
    dx = torch.empty(dy.shape[0], dy.shape[1] * (2 if gated else 1), dtype=dy.dtype, device=dy.device)
    return asr_activation_grads(dy, saved if kept is None else None, dx, function, gated=gated, kept=kept)


class _ActivationFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, function, gated, save, rounding, step, seed):
        x = _by_rows(x)
        ctx.kind = (function, gated)
        ctx.x_dtype = x.dtype
        if not ctx.needs_input_grad[0]:
            return activation(x, function, gated=gated)
        y, saved = activation(x, function, gated=gated, save=save, rounding=rounding, step=step, seed=seed)
        ctx.save_for_backward(*(saved[:2] if save == "int8" else (saved,)))
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        function, gated = ctx.kind
        saved = ctx.saved_tensors
        saved = Int8Checkpoint(*saved, ctx.x_dtype) if len(saved) == 2 else saved[0]
        return activation_grads(_by_rows(dy), saved, function, gated=gated), None, None, None, None, None, None


class Activation(_CountedModule):
    """A layer's activation, its input kept in 8 bits for the backward pass
    (``save="int8"``) or as it is (``"input"``).  ``gated``: the first half of the
    last dimension through the function, times the second half."""

    def __init__(self, function: str = "silu", *, gated: bool = False, save: str = "int8", rounding: str = "rne",
                 seed: int = 0):
        _check_save(save, _SAVE[1:])
        if function not in ("silu", "gelu"):
            raise ValueError(f"function must be 'silu' or 'gelu', not {function!r}")
        if rounding not in ("sr", "rne"):
            raise ValueError(f"rounding must be 'sr' or 'rne', not {rounding!r}")
        super().__init__(seed)
        self.function, self.gated, self.save, self.rounding = function, bool(gated), save, rounding

    def forward(self, x):
        self._count(x)
        flat = x.reshape(-1, x.shape[-1])
        y = _ActivationFunction.apply(flat, self.function, self.gated, self.save, self.rounding, self.calls, self.seed)
        return y.reshape(*x.shape[:-1], y.shape[-1])

    def extra_repr(self):
        return f"{self.function!r}, gated={self.gated}, save={self.save!r}, rounding={self.rounding!r}, seed={self.seed}"


# -------------------------------------------------------------- layer norm


class NormSaved(NamedTuple):
    """What a norm's backward pass reads."""
    input: Union[torch.Tensor, Int8Checkpoint]
    mean: Optional[torch.Tensor]            # None if not centred
    rstd: torch.Tensor


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, centred=True, save=None, rounding="rne", step: int = 0,
               seed: int = 0):
    """(x - mean) rstd weight + bias for each row of ``x`` (2-D); ``centred=False`` is
    the norm by the root mean square.  With ``save`` returns (y, saved) for
    ``layer_norm_grads``: "input" saves x itself, "int8" its 8-bit checkpoint, made in
    the same pass."""
    _check_save(save)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if save is None:
        return asr_layer_norm(x, weight, bias, y, eps=eps, centred=centred)
    rows = x.shape[0]
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    mean = torch.empty(rows, dtype=torch.float32, device=x.device) if centred else None
    kept = empty_checkpoint(*x.shape, x.device, x.dtype) if save == "int8" else None
    asr_layer_norm(x, weight, bias, y, mean, rstd, eps=eps, centred=centred, keep=kept, rounding=rounding, step=step,
                   seed=seed)
    return y, NormSaved(x if kept is None else kept, mean, rstd)


def layer_norm_grads(dy, saved: NormSaved, weight=None, *, need_dx=True, need_dweight=True, need_dbias=True,
                     dbias_dtype=None):
    """(dx, dweight, dbias) from ``dy`` and what ``layer_norm`` saved, each None where it
    is not needed; dx of dy's dtype, dweight of the weight's (dy's, if the norm has none),
    dbias of ``dbias_dtype`` (dweight's unless given)."""
    cols = dy.shape[1]
    kept = saved.input if isinstance(saved.input, Int8Checkpoint) else None
    dx = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device) if need_dx else None
    dtype = dy.dtype if weight is None else weight.dtype
    dweight = torch.empty(cols, dtype=dtype, device=dy.device) if need_dweight else None
    dbias = torch.empty(cols, dtype=dbias_dtype or dtype, device=dy.device) if need_dbias else None
    asr_layer_norm_grads(dy, saved.input if kept is None else None, weight, saved.mean, saved.rstd, dx, dweight, dbias,
                         centred=saved.mean is not None, kept=kept)
    return dx, dweight, dbias


class _LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, centred, save, rounding, step, seed):
        x = _by_rows(x)
        if not any(ctx.needs_input_grad):
            return layer_norm(x, weight, bias, eps=eps, centred=centred)
        ctx.x_dtype, ctx.bias_dtype = x.dtype, None if bias is None else bias.dtype
        y, saved = layer_norm(x, weight, bias, eps=eps, centred=centred, save=save, rounding=rounding, step=step, seed=seed)
        ctx.save_for_backward(weight, saved.mean, saved.rstd, *(saved.input[:2] if save == "int8" else (saved.input,)))
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        weight, mean, rstd, *x = ctx.saved_tensors
        saved = NormSaved(Int8Checkpoint(*x, ctx.x_dtype) if len(x) == 2 else x[0], mean, rstd)
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_grads(_by_rows(dy), saved, weight, need_dx=need[0], need_dweight=need[1], need_dbias=need[2],
                                      dbias_dtype=ctx.bias_dtype)
        return dx, dw, db, None, None, None, None, None, None


class LayerNorm(_CountedModule):
    """``torch.nn.LayerNorm`` over the last dimension, of size ``width``, or,
    ``centred=False``, the norm by the root mean square (no bias unless asked for); its
    input is kept as it is for the backward pass, or in 8 bits (``save="int8"``)."""

    def __init__(self, width: int, eps: float = 1e-5, *, centred: bool = True, bias: Optional[bool] = None,
                 save: str = "input", rounding: str = "rne", seed: int = 0, device=None, dtype=torch.bfloat16):
        _check_save(save, _SAVE[1:])
        if rounding not in ("sr", "rne"):
            raise ValueError(f"rounding must be 'sr' or 'rne', not {rounding!r}")
        super().__init__(seed)
        self.width, self.eps, self.centred, self.save, self.rounding = int(width), float(eps), bool(centred), save, rounding
        self.weight = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))
        if centred if bias is None else bias:
            self.bias = torch.nn.Parameter(torch.zeros(width, device=device, dtype=dtype))
        else:
            self.register_parameter("bias", None)

    def forward(self, x):
        self._count(x, self.weight, self.bias)
        flat = x.reshape(-1, self.width)
        y = _LayerNormFunction.apply(flat, self.weight, self.bias, self.eps, self.centred, self.save, self.rounding,
                                     self.calls, self.seed)
        return y.reshape(x.shape)

    def extra_repr(self):
        return (f"{self.width}, eps={self.eps}, centred={self.centred}, bias={self.bias is not None}, save={self.save!r}, "
                f"rounding={self.rounding!r}, seed={self.seed}")


# --------------------------------------------------------------- embedding


def embedding(ids, table, *, scale: float = 1.0):
    """``scale * table[ids]`` for ``ids`` (1-D, int64 or int32): (tokens, dim).  An id
    outside the table gives a row of NaN."""
    y = torch.empty(ids.shape[0], table.shape[1], dtype=table.dtype, device=table.device)
    return asr_embedding(ids, table, y, scale=scale)


def embedding_grads(ids, dy, vocab: int, *, scale: float = 1.0, padding_idx: Optional[int] = None, dtype=None):
    """The whole table's gradient, (vocab, dim) in ``dtype`` (dy's unless given): for each
    row, scale times the sum of ``dy`` over its tokens, in their order."""
    dtable = torch.empty(int(vocab), dy.shape[1], dtype=dtype or dy.dtype, device=dy.device)
    return asr_embedding_grads(ids, dy, dtable, scale=scale, padding_idx=padding_idx)


class _EmbeddingFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale, padding_idx):
        table = _by_rows(table)
        ctx.save_for_backward(ids)
        ctx.kind = (table.shape[0], scale, padding_idx, table.dtype)
        return embedding(ids, table, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (ids,) = ctx.saved_tensors
        vocab, scale, padding_idx, dtype = ctx.kind
        return None, embedding_grads(ids, _by_rows(dy), vocab, scale=scale, padding_idx=padding_idx, dtype=dtype), None, None


class Embedding(torch.nn.Module):
    """``torch.nn.Embedding`` with a factor on what is looked up (``scale``, such as the
    root of ``dim``).  Its gradient is dense, for this package's optimizers; tokens of
    ``padding_idx`` add nothing to it."""

    def __init__(self, vocab: int, dim: int, *, scale: float = 1.0, padding_idx: Optional[int] = None, device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        if padding_idx is not None and not 0 <= int(padding_idx) < vocab:
            raise ValueError(f"padding_idx must be a row of the table (0 to {vocab - 1}), not {padding_idx}")
        self.vocab, self.dim, self.scale, self.padding_idx = int(vocab), int(dim), float(scale), padding_idx
        self.weight = torch.nn.Parameter(torch.empty(vocab, dim, device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=0.02)

    def forward(self, ids):
        y = _EmbeddingFunction.apply(ids.reshape(-1).contiguous(), self.weight, self.scale, self.padding_idx)
        return y.reshape(*ids.shape, self.dim)

    def extra_repr(self):
        return f"{self.vocab}, {self.dim}, scale={self.scale}, padding_idx={self.padding_idx}"
