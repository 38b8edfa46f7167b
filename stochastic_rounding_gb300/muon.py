"""``MuonSR``: Muon for matrices kept in bf16, without a float32 copy.

It takes the place of ``torch.optim.Muon``, with the same arguments plus a seed:
the momentum (float32) is orthogonalised by Newton-Schulz products, and the
bfloat16 parameters are decayed, stepped and rounded stochastically in place.
The rounding bits are keyed by (seed, step) and indexed by each element's global
parameter position, as ``AdamWSR``'s are (``stochastic_rounding_gb300.optim``
says how positions are given, and when the device error bit is read), so a
model's matrices can go to ``MuonSR`` and its other parameters to ``AdamWSR``:
with one seed, at positions of their own (``base_offset`` of the second: the
number of elements of the first), or the two would round with the same bits.
An update depends on the whole matrix: unlike AdamW's, a step of a matrix cannot
be cut into shards.

All matrices of one shape and type are worked on together, in one call of the
library for each group, device and step count.
"""
from __future__ import annotations

from typing import Dict, List

import torch

from . import _lib
from .optim import _PlacedOptimizer


class MuonSR(_PlacedOptimizer):
    """Muon with stochastic rounding of bf16 parameters.

    Arguments follow ``torch.optim.Muon`` (``lr``, ``weight_decay``,
    ``momentum``, ``nesterov``, ``ns_coefficients``, ``eps``, ``ns_steps``,
    ``adjust_lr_fn``: ``"original"`` (or None), the rate times sqrt(max(1, rows
    / cols)), or ``"match_rms_adamw"``, times 0.2 sqrt(max(rows, cols))) plus
    ``seed``, ``rounding``, ``base_offset`` and ``check_errors`` as ``AdamWSR``
    has them.  Parameters must be contiguous CUDA matrices (2-D) or stacks of
    matrices (3-D, such as a layer's experts) of float32 or bfloat16; gradients
    dense float32 or bfloat16."""

    def __init__(self, params, lr: float = 1e-3, weight_decay: float = 0.1, momentum: float = 0.95,
                 nesterov: bool = True, ns_coefficients=_lib.NS_COEFFICIENTS, eps: float = 1e-7, ns_steps: int = 5,
                 adjust_lr_fn=None, *, seed: int = 0, rounding: str = "sr", base_offset: int = 0, check_errors=True):
        if not 0.0 <= lr:
            raise ValueError(f"Invalid learning rate: {lr}")
        if not 0.0 <= weight_decay:
            raise ValueError(f"Invalid weight_decay value: {weight_decay}")
        if not 0.0 <= momentum < 1.0:
            raise ValueError(f"Invalid momentum value: {momentum}")
        if not 0.0 < eps:
            raise ValueError(f"Invalid epsilon value: {eps}")
        if not 1 <= ns_steps <= 100:
            raise ValueError(f"ns_steps must be between 1 and 100, not {ns_steps}")
        if len(ns_coefficients) != 3:
            raise ValueError("ns_coefficients must be three numbers")
        if adjust_lr_fn not in (None, "original", "match_rms_adamw"):
            raise ValueError(f"adjust_lr_fn must be 'original' or 'match_rms_adamw', not {adjust_lr_fn!r}")
        if rounding not in ("sr", "rne"):
            raise ValueError(f"rounding must be 'sr' or 'rne', not {rounding!r}")
        if not 0 <= int(seed) < 2**64:
            raise ValueError("seed must fit in 64 bits")
        self._place(base_offset, check_errors)
        defaults = dict(lr=lr, weight_decay=weight_decay, momentum=momentum, nesterov=nesterov,
                        ns_coefficients=tuple(ns_coefficients), eps=eps, ns_steps=ns_steps,
                        adjust_lr_fn=adjust_lr_fn or "original", seed=int(seed), rounding=rounding, base_index=None)
        super().__init__(params, defaults)
        self._assign_positions()

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        for p in self.param_groups[-1]["params"]:
            if p.dim() not in (2, 3):
                self.param_groups.pop()
                if hasattr(self, "_base"):
                    self._assign_positions()
                raise ValueError(f"MuonSR takes matrices (2-D) and stacks of them (3-D), not {p.dim()}-D parameters")

    @staticmethod
    def _settings(group):
        return dict(lr=group["lr"], momentum=group["momentum"], weight_decay=group["weight_decay"],
                    nesterov=group["nesterov"], steps=group["ns_steps"], coefficients=group["ns_coefficients"],
                    eps=group["eps"], adjust=group["adjust_lr_fn"], seed=group["seed"], rounding=group["rounding"])

    @staticmethod
    def _check(p: torch.Tensor):
        if not p.is_cuda:
            raise ValueError("MuonSR parameters must live on a CUDA device")
        if p.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"MuonSR supports float32 and bfloat16 parameters, not {p.dtype}")
        if not p.is_contiguous():
            raise ValueError("MuonSR parameters must be contiguous")
        g = p.grad
        if g.is_sparse:
            raise RuntimeError("MuonSR does not support sparse gradients")
        if g.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"MuonSR supports float32 and bfloat16 gradients, not {g.dtype}")
        if not g.is_contiguous() or g.shape != p.shape or g.get_device() != p.get_device():
            raise ValueError("gradient must be contiguous, on the parameter's device and of its shape")

    @torch.no_grad()
    def step(self, closure=None, *, check_errors=None):
        """One step of every parameter that has a gradient.  ``check_errors``
        overrides the optimizer's setting for this call."""
        mode = self.check_errors if check_errors is None else self._error_mode(check_errors)
        if self._pending:
            self.poll_errors()
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        # every parameter, and every group's settings (by a step over no matrices), are
        # checked before anything is launched or counted
        for group in self.param_groups:
            live = [p for p in group["params"] if p.grad is not None]
            for p in live:
                self._check(p)
            if live:
                _lib.asr_muon_sr_multi_tensor([], step=1, **self._settings(group))
        devices = set()
        for group in self.param_groups:
            batches: Dict[tuple, List[tuple]] = {}
            for p in group["params"]:
                if p.grad is None:
                    continue
                state = self.state[p]
                if len(state) == 0:
                    state["step"] = 0
                    state["momentum_buffer"] = torch.zeros_like(p, dtype=torch.float32,
                                                                memory_format=torch.contiguous_format)
                state["step"] = int(state["step"]) + 1
                batches.setdefault((p.device, state["step"]), []).append(
                    (p, p.grad, state["momentum_buffer"], self._base[id(p)]))
            for (device, step), entries in batches.items():
                _lib.asr_muon_sr_multi_tensor(entries, step=step, **self._settings(group))
                devices.add(device)
        self._finish_step(devices, mode)
        return loss

    def load_state_dict(self, state_dict):
        """Like torch's, but the momentum stays float32."""
        from itertools import chain
        super().load_state_dict(state_dict)
        saved_ids = chain.from_iterable(g["params"] for g in state_dict["param_groups"])
        params = chain.from_iterable(g["params"] for g in self.param_groups)
        id_map = dict(zip(saved_ids, params))
        for pid, st in state_dict["state"].items():
            p = id_map[pid]
            if "momentum_buffer" in st:
                self.state[p]["momentum_buffer"] = st["momentum_buffer"].to(device=p.device, dtype=torch.float32,
                                                                            copy=True)
            if "step" in self.state[p]:
                self.state[p]["step"] = int(self.state[p]["step"])
        for group in self.param_groups:
            group.setdefault("base_index", None)
        self._assign_positions()
