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


def _inputs():
    torch.manual_seed(1)
    return {"transposed": torch.randn(1, 8, 5).transpose(1, 2),      # a view whose rows are not contiguous
            "transposed_two": torch.randn(2, 8, 5).transpose(1, 2),
            "expanded": torch.randn(1, 8).expand(5, 8),              # rows that overlap
            "expanded_batch": torch.randn(1, 1, 8).expand(3, 5, 8),
            "every_other": torch.randn(5, 16)[:, ::2],
            "pitched": torch.randn(5, 11)[:, :8],
            "vector": torch.randn(8),
            "none": torch.randn(0, 8)}


@pytest.mark.parametrize("name", list(_inputs()))
def test_inputs_of_any_layout(calls, name):
    """What torch.nn.Linear takes: any strides, and the gradients of each."""
    x = _inputs()[name].requires_grad_()
    layer = int8.Int8Linear(8, 6, dtype=torch.float32)
    y = layer(x)
    g = torch.randn(6).expand(y.shape)
    y.backward(g.to(y.dtype))
    want = x.detach().clone().requires_grad_()
    w = layer.weight.detach().clone().requires_grad_()
    torch.nn.functional.linear(want, w).backward(g.to(y.dtype).float())
    # bf16 outputs and gradients of sums of eight and five products, and a weight in 8 bits
    assert y.shape == x.shape[:-1] + (6,) and x.grad.shape == x.shape
    for a, b in ((x.grad, want.grad), (layer.weight.grad, w.grad)):
        assert torch.allclose(a, b, rtol=2.0 ** -7, atol=2.0 ** -7 * float(b.abs().max()) if b.numel() else 0.0)


def test_pitched_rows_are_not_copied(calls):
    layer = int8.Int8Linear(8, 6, dtype=torch.float32)
    x = torch.randn(5, 11)[:, :8]
    layer(x)
    assert calls.inputs[0].data_ptr() == x.data_ptr()


def test_weight_of_any_layout(calls):
    """A weight tied to another module's as its transpose."""
    layer = int8.Int8Linear(8, 6, dtype=torch.float32)
    base = torch.randn(8, 6)
    layer.weight = torch.nn.Parameter(base.t())
    x = torch.randn(5, 8)
    layer(x).float().sum().backward()
    assert torch.allclose(layer.weight.grad, x.sum(0).expand(6, 8), rtol=2.0 ** -7, atol=2.0 ** -7 * 5)
