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


def _train(layer, passes, calls, evaluate=0):
    for _ in range(passes):
        for _ in range(evaluate):
            with torch.no_grad():
                layer(torch.ones(2, 8))
        layer(torch.ones(2, 8)).float().sum().backward()
    return calls.steps


def test_a_resumed_layer_goes_on_with_its_random_numbers(calls):
    """The count of passes is part of the state, so passes after a checkpoint draw
    what they draw without one."""
    whole = _train(int8.Int8Linear(8, 6), 5, calls)[:]
    calls.steps.clear()
    first = int8.Int8Linear(8, 6)
    _train(first, 2, calls)
    second = int8.Int8Linear(8, 6)
    second.load_state_dict(first.state_dict())
    assert _train(second, 3, calls) == whole == [1, 2, 3, 4, 5]


def test_passes_without_gradients_draw_nothing(calls):
    """A run that is evaluated in between draws the numbers of one that is not."""
    assert _train(int8.Int8Linear(8, 6), 3, calls, evaluate=2) == [1, 2, 3]
    frozen = int8.Int8Linear(8, 6)
    frozen.weight.requires_grad_(False)
    frozen(torch.ones(2, 8))
    assert frozen.calls == 0
    frozen(torch.ones(2, 8, requires_grad=True))
    assert frozen.calls == 1


def test_state_of_other_modules_and_of_older_checkpoints(calls):
    """A dictionary with the weight alone loads, and leaves the count as it is."""
    layer = int8.Int8Linear(8, 6)
    _train(layer, 2, calls)
    plain = torch.nn.Linear(8, 6, bias=False)
    assert not layer.load_state_dict(plain.state_dict()).missing_keys and layer.calls == 2
    net = torch.nn.Sequential(int8.Int8Linear(8, 6), int8.Int8Linear(6, 8))
    net.load_state_dict({k: v for k, v in net.state_dict().items() if k.endswith("weight")})
    with pytest.raises(RuntimeError):
        layer.load_state_dict({})
    with pytest.raises(RuntimeError):
        layer.load_state_dict({**plain.state_dict(), "bias": torch.zeros(6)})
