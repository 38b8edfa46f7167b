"""Int8Linear's own logic without a GPU: the library's three calls are replaced
by plain products on the CPU."""
import pytest
import torch

import stochastic_rounding_gb300.int8 as int8


class Calls:
    """What the module asked the library for."""

    def __init__(self):
        self.inputs, self.steps, self.seeds = [], [], []


@pytest.fixture
def calls(monkeypatch):
    seen = Calls()

    def rows_ok(t):
        assert t.dim() == 2 and (t.shape[1] <= 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1]), \
            "rows must be contiguous and must not overlap"

    def quantize(w, q, scale, **kw):
        rows_ok(w)
        scale.copy_(w.detach().float().abs().amax(1) / 127)
        q.copy_(torch.round(w.detach().float() / scale[:, None]))
        return q, scale

    def linear(x, q, scale, y, **kw):
        rows_ok(x)
        seen.inputs.append(x)
        return y.copy_(x.detach().float() @ (q.float() * scale[:, None]).t())

    def grads(dy, x, w, dx, dw, *, step, seed, **kw):
        for t in (dy, x, w):
            rows_ok(t)
        seen.steps.append(step)
        seen.seeds.append(seed)
        if dx is not None:
            dx.copy_(dy.detach().float() @ w.detach().float())
        if dw is not None:
            dw.copy_(dy.detach().float().t() @ x.detach().float())

    monkeypatch.setattr(int8, "asr_quantize_int8", quantize)
    monkeypatch.setattr(int8, "asr_linear_int8", linear)
    monkeypatch.setattr(int8, "asr_linear_int8_grads", grads)
    return seen


def test_second_derivatives_are_refused(calls):
    """The backward pass records nothing, so what is asked through it again has
    to be an error, not a gradient of zero."""
    torch.manual_seed(0)
    layer = int8.Int8Linear(8, 6, dtype=torch.float32)
    x = torch.randn(5, 8, requires_grad=True)
    loss = layer(x).float().square().sum()
    (dx,) = torch.autograd.grad(loss, x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (loss + dx.square().sum()).backward()        # a gradient penalty
