"""What stands between a layer's 8-bit products: the norm, the activation and the
embedding, forward and backward, their inputs kept for the backward pass as they are
or in 8 bits (``checkpoint_int8`` in ``stochastic_rounding_gb300.int8``).

The functions work on 2-D tensors whose rows are contiguous and return new ones; the
modules take any shape and layout, record gradients, and hold parameters for this
package's optimizers.  Nothing here has a second derivative.

A pass that is kept in 8 bits and rounded stochastically takes its random numbers from
(seed, step), the same for every call with these: modules count their passes (``calls``)
and go on counting from a state dict.  A pass captured into a CUDA graph keeps its
number, and every replay its random numbers.  These numbers are not an optimizer's, nor
those of ``Int8Linear``'s gradients, whatever the seed; modules that share a seed share
them.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Union

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .int8 import (_FLOATS, Int8Checkpoint, _by_rows, _checked, _CountedModule, _elsewhere, _raw_stream,
                   empty_checkpoint)

_SAVE = (None, "input", "int8")


def _check_save(save, allowed=_SAVE):
    if save not in allowed:
        raise ValueError(f"save must be one of {allowed}, not {save!r}")


# -------------------------------------------------------------- activation


def activation(x, function="silu", *, gated=False, save=None, rounding="rne", step: int = 0, seed: int = 0):
    """f(x) for ``x`` (rows, columns), or, ``gated``, f of its first half of columns
    times its second half.  ``function``: "silu", or "gelu" (its tanh form).  With
    ``save`` returns (y, saved) for ``activation_grads``: "input" saves x itself,
    "int8" its 8-bit checkpoint, made in the same pass (in one of its own where a gated
    half is no multiple of 32 columns)."""
    _check_save(save)
    _lib._check_rounding(rounding)
    code = _lib._function(function)
    px, rows, width, ld, dtype, d = _lib._rows_of(x, "x")
    if gated and width % 2:
        raise ValueError(f"a gated activation takes an even number of columns, not {width}")
    if _elsewhere(d):
        with torch.cuda.device(d):
            return activation(x, function, gated=gated, save=save, rounding=rounding, step=step, seed=seed)
    cols = width // 2 if gated else width
    y = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
    kept = key = None
    if save == "int8":
        kept = empty_checkpoint(rows, width, x.device, x.dtype)
        key = kept._struct(rounding, 0, step, seed)
    _lib._check(_lib.lib().asr_activation(px, ld, y.data_ptr(), cols, dtype, rows, cols, code, 1 if gated else 0, key,
                                          _raw_stream(d)), "asr_activation")
    return y if save is None else (y, x if kept is None else kept)


def activation_grads(dy, saved: Union[torch.Tensor, Int8Checkpoint], function="silu", *, gated=False):
    """dx from ``dy`` and what ``activation`` saved."""
    code = _lib._function(function)
    pg, rows, cols, g_ld, dtype, d = _lib._rows_of(dy, "dy")
    width = 2 * cols if gated else cols
    px, x_ld, kept = _saved_input(saved, rows, width, dtype, d)
    if _elsewhere(d):
        with torch.cuda.device(d):
            return activation_grads(dy, saved, function, gated=gated)
    dx = torch.empty((rows, width), dtype=dy.dtype, device=dy.device)
    _lib._check(_lib.lib().asr_activation_grads(pg, g_ld, px, x_ld, kept, dx.data_ptr(), width, dtype, rows, cols, code,
                                                1 if gated else 0, _raw_stream(d)), "asr_activation_grads")
    return dx


def _saved_input(saved, rows, cols, dtype, device):
    """(pointer, pitch, checkpoint) of what a forward pass saved, the pointer or the checkpoint None."""
    if isinstance(saved, Int8Checkpoint):
        return None, cols, _checked(saved, rows, cols, device)
    px, xr, xc, ld, xt, xd = _lib._rows_of(saved, "the saved input")
    if xr != rows or xc != cols or xt != dtype or xd != device:
        raise ValueError(f"the saved input has shape {(xr, xc)} and type {saved.dtype} on cuda:{xd}; it must have {(rows, cols)}, "
                         f"dy's type and dy's device (cuda:{device})")
    return px, ld, None


class _ActivationFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, function, gated, save, rounding, step, seed):
        x = _by_rows(x)
        ctx.kind = (function, gated, x.shape[1], x.dtype)
        if save is None:
            return activation(x, function, gated=gated)
        y, saved = activation(x, function, gated=gated, save=save, rounding=rounding, step=step, seed=seed)
        ctx.kept = save == "int8"
        ctx.save_for_backward(saved.data if ctx.kept else saved)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        function, gated, width, dtype = ctx.kind
        (saved,) = ctx.saved_tensors
        if ctx.kept:
            saved = Int8Checkpoint(saved, width, dtype)
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
        save = self.save if self._count(x) else None
        flat = x.reshape(x.shape[:-1].numel(), x.shape[-1])
        y = _ActivationFunction.apply(flat, self.function, self.gated, save, self.rounding, self.calls, self.seed)
        return y.reshape(*x.shape[:-1], y.shape[-1])

    def extra_repr(self):
        return f"{self.function!r}, gated={self.gated}, save={self.save!r}, rounding={self.rounding!r}, seed={self.seed}"


# -------------------------------------------------------------- layer norm


class NormSaved(NamedTuple):
    """What a norm's backward pass reads."""
    input: Union[torch.Tensor, Int8Checkpoint]
    stats: torch.Tensor                     # float32, (1 or 2, rows): rstd, and, centred, the mean

    @property
    def rstd(self):
        return self.stats[0]

    @property
    def mean(self):
        return self.stats[1] if self.stats.shape[0] == 2 else None


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, centred=True, save=None, rounding="rne", step: int = 0,
               seed: int = 0):
    """(x - mean) rstd weight + bias for each row of ``x`` (2-D); ``centred=False`` is
    the norm by the root mean square.  With ``save`` returns (y, saved) for
    ``layer_norm_grads``: "input" saves x itself, "int8" its 8-bit checkpoint, made in
    the same pass."""
    _check_save(save)
    _lib._check_rounding(rounding)
    px, rows, cols, ld, dtype, d = _lib._rows_of(x, "x")
    p = _lib._norm_params(rows, cols, dtype, weight, bias, eps, centred, d)
    if _elsewhere(d):
        with torch.cuda.device(d):
            return layer_norm(x, weight, bias, eps=eps, centred=centred, save=save, rounding=rounding, step=step, seed=seed)
    y = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
    rstd = mean = kept = key = None
    if save is not None:
        stats = torch.empty((2 if centred else 1, rows), dtype=torch.float32, device=x.device)
        rstd = stats.data_ptr()
        mean = rstd + 4 * rows if centred else None
        if save == "int8":
            kept = empty_checkpoint(rows, cols, x.device, x.dtype)
            key = kept._struct(rounding, 0, step, seed)
    _lib._check(_lib.lib().asr_layer_norm(p, px, ld, y.data_ptr(), cols, mean, rstd, key, _raw_stream(d)), "asr_layer_norm")
    return y if save is None else (y, NormSaved(x if kept is None else kept, stats))


def layer_norm_grads(dy, saved: NormSaved, weight=None, *, need_dx=True, need_dweight=True, need_dbias=True,
                     dbias_dtype=None):
    """(dx, dweight, dbias) from ``dy`` and what ``layer_norm`` saved, each None where it
    is not needed; dx of dy's dtype, dweight of the weight's (dy's, if the norm has none),
    dbias of ``dbias_dtype`` (dweight's unless given)."""
    pg, rows, cols, g_ld, code, d = _lib._rows_of(dy, "dy")
    px, x_ld, kept = _saved_input(saved.input, rows, cols, code, d)
    stats = saved.stats
    centred = stats.shape[0] == 2
    rstd = _lib._dev_ptr(stats, "stats", (torch.float32,), (2 if centred else 1) * rows, d)
    p = _lib._norm_params(rows, cols, code, weight, None, 0.0, centred, d)
    dtype = dy.dtype if weight is None else weight.dtype
    if dbias_dtype is not None and dbias_dtype not in _FLOATS:
        raise TypeError(f"a gradient comes as float32 or bfloat16, not {dbias_dtype}")
    if _elsewhere(d):
        with torch.cuda.device(d):
            return layer_norm_grads(dy, saved, weight, need_dx=need_dx, need_dweight=need_dweight, need_dbias=need_dbias,
                                    dbias_dtype=dbias_dtype)
    device = dy.device
    dx = dweight = dbias = buf = None
    to_x = to_w = to_b = to_ws = None
    w_type = b_type = need = 0
    if need_dx:
        dx = torch.empty((rows, cols), dtype=dy.dtype, device=device)
        to_x = dx.data_ptr()
    if need_dweight:
        dweight = torch.empty(cols, dtype=dtype, device=device)
        to_w, w_type = dweight.data_ptr(), _lib._dt(dweight)
    if need_dbias:
        dbias = torch.empty(cols, dtype=dbias_dtype or dtype, device=device)
        to_b, b_type = dbias.data_ptr(), _lib._dt(dbias)
    if need_dweight or need_dbias:
        need = _lib.asr_layer_norm_grads_workspace(rows, cols)
        buf = torch.empty(need, dtype=torch.uint8, device=device)
        to_ws = buf.data_ptr()
    _lib._check(_lib.lib().asr_layer_norm_grads(p, pg, g_ld, px, x_ld, kept, rstd + 4 * rows if centred else None, rstd, to_x, cols,
                                                to_w, w_type, to_b, b_type, to_ws, need, _raw_stream(d)), "asr_layer_norm_grads")
    return dx, dweight, dbias


class _LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, centred, save, rounding, step, seed):
        x = _by_rows(x)
        if save is None:
            return layer_norm(x, weight, bias, eps=eps, centred=centred)
        ctx.kept, ctx.kind = save == "int8", (x.dtype, None if bias is None else bias.dtype)
        y, saved = layer_norm(x, weight, bias, eps=eps, centred=centred, save=save, rounding=rounding, step=step, seed=seed)
        ctx.save_for_backward(weight, saved.stats, saved.input.data if ctx.kept else saved.input)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        weight, stats, x = ctx.saved_tensors
        x_dtype, bias_dtype = ctx.kind
        saved = NormSaved(Int8Checkpoint(x, dy.shape[1], x_dtype) if ctx.kept else x, stats)
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_grads(_by_rows(dy), saved, weight, need_dx=need[0], need_dweight=need[1], need_dbias=need[2],
                                      dbias_dtype=bias_dtype)
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
        if x.shape[-1:] != (self.width,):
            raise ValueError(f"the last dimension must be {self.width}, not that of {tuple(x.shape)}")
        save = self.save if self._count(x, self.weight, self.bias) else None
        flat = x.reshape(x.shape[:-1].numel(), self.width)
        y = _LayerNormFunction.apply(flat, self.weight, self.bias, self.eps, self.centred, save, self.rounding, self.calls,
                                     self.seed)
        return y.reshape(x.shape)

    def extra_repr(self):
        return (f"{self.width}, eps={self.eps}, centred={self.centred}, bias={self.bias is not None}, save={self.save!r}, "
                f"rounding={self.rounding!r}, seed={self.seed}")


# --------------------------------------------------------------- embedding


def embedding(ids, table, *, scale: float = 1.0):
    """``scale * table[ids]`` for ``ids`` (1-D, int64 or int32): (tokens, dim).  An id
    outside the table gives a row of NaN."""
    pt, vocab, dim, ld, dtype, d = _lib._rows_of(table, "table")
    pi, index, tokens = _lib._ids(ids, d)
    if _elsewhere(d):
        with torch.cuda.device(d):
            return embedding(ids, table, scale=scale)
    y = torch.empty((tokens, dim), dtype=table.dtype, device=table.device)
    _lib._check(_lib.lib().asr_embedding(pi, index, tokens, pt, ld, vocab, dim, scale, y.data_ptr(), dim, dtype, _raw_stream(d)),
                "asr_embedding")
    return y


def embedding_grads(ids, dy, vocab: int, *, scale: float = 1.0, padding_idx: Optional[int] = None, dtype=None):
    """The whole table's gradient, (vocab, dim) in ``dtype`` (dy's unless given): for each
    row, scale times the sum of ``dy`` over its tokens, in their order."""
    pg, rows, dim, ld, code, d = _lib._rows_of(dy, "dy")
    pi, index, tokens = _lib._ids(ids, d)
    if rows != tokens:
        raise ValueError(f"dy has {rows} rows; expected {tokens}")
    if padding_idx is not None and not 0 <= padding_idx < vocab:
        raise ValueError(f"padding_idx must be a row of the table (0 to {vocab - 1}), not {padding_idx}")
    if dtype is not None and dtype not in _FLOATS:
        raise TypeError(f"a gradient comes as float32 or bfloat16, not {dtype}")
    if _elsewhere(d):
        with torch.cuda.device(d):
            return embedding_grads(ids, dy, vocab, scale=scale, padding_idx=padding_idx, dtype=dtype)
    need = _lib.asr_embedding_grads_workspace(tokens, dim)
    out = torch.empty((vocab, dim), dtype=dtype or dy.dtype, device=dy.device)
    buf = torch.empty(need, dtype=torch.uint8, device=dy.device) if need else None
    _lib._check(_lib.lib().asr_embedding_grads(pi, index, tokens, pg, ld, code, vocab, dim, scale,
                                               -1 if padding_idx is None else padding_idx, out.data_ptr(), _lib._dt(out),
                                               None if buf is None else buf.data_ptr(), need, _raw_stream(d)),
                "asr_embedding_grads")
    return out


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
    ``padding_idx`` add nothing to it.  That row is drawn like the others (from a normal
    distribution of deviation 0.02), and not zeros as in ``torch.nn.Embedding``: zero it,
    or load a table, where its values matter."""

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
