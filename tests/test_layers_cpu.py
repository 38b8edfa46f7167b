"""The calls between a layer's 8-bit products without a GPU: what the library and the binding refuse before
anything is launched, and the modules' own logic."""
import ctypes

import pytest
import torch

import stochastic_rounding_gb300 as asr
from stochastic_rounding_gb300 import _lib, int8, layers
from test_binding_cpu import _on

BAD, TYPE, OK = _lib.ASR_ERR_INVALID_VALUE, _lib.ASR_ERR_UNSUPPORTED_DTYPE, _lib.ASR_OK
P = 4096            # stands for memory: never read here


@pytest.fixture(scope="module")
def L():
    from stochastic_rounding_gb300 import build
    build.build()
    return asr.lib()


def kept(q=P, power=P, q_ld=64, power_ld=2, base=0, rounding=_lib.ASR_ROUND_RNE):
    return ctypes.byref(_lib.Checkpoint(q, power, q_ld, power_ld, base, 0, 1, rounding))


def test_checkpoint_refusals(L):
    def call(x=P, dtype=1, rows=4, cols=64, ld=64, to=kept()):
        return L.asr_checkpoint_int8(x, dtype, rows, cols, ld, to, None)
    assert call(rows=0) == OK and call(cols=0, x=None) == OK
    assert call(dtype=2) == TYPE and call(to=kept(rounding=5)) == TYPE
    for k in (dict(x=None), dict(to=None), dict(ld=63), dict(ld=2 ** 32), dict(x=P + 1), dict(dtype=0, x=P + 2),
              dict(to=kept(q=None)), dict(to=kept(power=None)), dict(to=kept(q_ld=63)), dict(to=kept(power_ld=1)),
              dict(to=kept(base=8)), dict(to=kept(base=2 ** 64 - 32)), dict(rows=2 ** 30 + 1), dict(cols=2 ** 24 + 1, ld=2 ** 25)):
        assert call(**k) == BAD, k

    def back(c=kept(), rows=4, cols=64, out=P, dtype=1, ld=64):
        return L.asr_restore_int8(c, rows, cols, out, dtype, ld, None)
    assert back(rows=0) == OK and back(dtype=7) == TYPE
    for k in (dict(c=None), dict(out=None), dict(ld=10), dict(out=P + 1), dict(c=kept(q_ld=8)), dict(c=kept(power_ld=1))):
        assert back(**k) == BAD, k


def test_activation_refusals(L):
    def call(x=P, x_ld=64, y=P, y_ld=64, dtype=1, rows=4, cols=32, function=0, gated=1, to=None):
        return L.asr_activation(x, x_ld, y, y_ld, dtype, rows, cols, function, gated, to, None)
    assert call(rows=0, x=None) == OK
    assert call(dtype=3) == TYPE and call(function=2) == TYPE and call(to=kept(rounding=9)) == TYPE
    for k in (dict(x=None), dict(y=None), dict(gated=2), dict(x_ld=63), dict(y_ld=31), dict(x=P + 1),
              dict(to=kept(q_ld=32)), dict(to=kept(base=3)), dict(cols=2 ** 24 + 1)):
        assert call(**k) == BAD, k

    def back(dy=P, g_ld=32, x=P, x_ld=64, c=None, dx=P, d_ld=64, dtype=1, rows=4, cols=32, function=0, gated=1):
        return L.asr_activation_grads(dy, g_ld, x, x_ld, c, dx, d_ld, dtype, rows, cols, function, gated, None)
    assert back(rows=0) == OK and back(dtype=5) == TYPE
    for k in (dict(x=None), dict(c=kept()), dict(dy=None), dict(dx=None), dict(d_ld=63), dict(g_ld=31), dict(x_ld=32),
              dict(x=None, c=kept(q_ld=32))):
        assert back(**k) == BAD, k


def norm_params(rows=4, cols=64, weight=P, bias=P, eps=1e-5, dtype=1, wt=1, bt=1, centred=1, reserved=0):
    return ctypes.byref(_lib.NormParams(rows, cols, weight, bias, eps, dtype, wt, bt, centred, reserved))


def test_norm_refusals(L):
    def call(p=norm_params(), x=P, x_ld=64, y=P, y_ld=64, mean=P, rstd=P, to=None):
        return L.asr_layer_norm(p, x, x_ld, y, y_ld, mean, rstd, to, None)
    assert call(p=norm_params(rows=0), x=None) == OK and call(p=norm_params(cols=0)) == OK
    for k in (dict(dtype=2), dict(wt=4), dict(bt=-1)):
        assert call(p=norm_params(**k)) == TYPE, k
    for k in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(centred=2), dict(reserved=1),
              dict(weight=P + 1), dict(bias=P + 1), dict(rows=2 ** 30 + 1)):
        assert call(p=norm_params(**k)) == BAD, k
    for k in (dict(p=None), dict(x=None), dict(y=None), dict(x_ld=63), dict(y_ld=63), dict(rstd=None), dict(mean=P + 2),
              dict(rstd=P + 1), dict(to=kept(q_ld=32)), dict(to=kept(q=None))):
        assert call(**k) == BAD, k
    need = ctypes.c_uint64(0)
    assert L.asr_layer_norm_grads_workspace(4, 64, ctypes.byref(need)) == OK and need.value > 0
    assert L.asr_layer_norm_grads_workspace(4, 64, None) == BAD
    assert L.asr_layer_norm_grads_workspace(2 ** 31, 64, ctypes.byref(need)) == BAD

    def back(p=norm_params(), dy=P, g_ld=64, x=P, x_ld=64, c=None, mean=P, rstd=P, dx=P, d_ld=64, dw=P, wt=1, db=P, bt=1, ws=P,
             size=need.value):
        return L.asr_layer_norm_grads(p, dy, g_ld, x, x_ld, c, mean, rstd, dx, d_ld, dw, wt, db, bt, ws, size, None)
    assert back(dx=None, dw=None, db=None, dy=None) == OK
    assert back(wt=2) == TYPE and back(bt=3) == TYPE
    for k in (dict(p=None), dict(dy=None), dict(x=None), dict(c=kept()), dict(x=None, c=kept(power_ld=1)), dict(mean=None),
              dict(rstd=None), dict(dw=P + 1), dict(db=P + 1), dict(dx=P + 1), dict(d_ld=60), dict(ws=None), dict(ws=P + 16),
              dict(size=need.value - 1)):
        assert back(**k) == BAD, k


def test_embedding_refusals(L):
    def call(ids=P, index=1, tokens=4, table=P, t_ld=64, vocab=10, dim=64, scale=1.0, y=P, y_ld=64, dtype=1):
        return L.asr_embedding(ids, index, tokens, table, t_ld, vocab, dim, scale, y, y_ld, dtype, None)
    assert call(tokens=0, ids=None) == OK and call(dim=0) == OK
    assert call(index=2) == TYPE and call(dtype=9) == TYPE
    for k in (dict(ids=None), dict(ids=P + 4), dict(index=0, ids=P + 2), dict(table=None), dict(y=None), dict(t_ld=63),
              dict(scale=float("inf")), dict(scale=float("nan")), dict(vocab=2 ** 28 + 1), dict(tokens=2 ** 28 + 1),
              dict(y_ld=2 ** 32)):
        assert call(**k) == BAD, k
    need = ctypes.c_uint64(0)
    assert L.asr_embedding_grads_workspace(4, 64, ctypes.byref(need)) == OK and need.value > 0
    assert L.asr_embedding_grads_workspace(0, 64, ctypes.byref(ctypes.c_uint64(1))) == OK
    assert L.asr_embedding_grads_workspace(2 ** 29, 64, ctypes.byref(need)) == BAD

    def back(ids=P, index=1, tokens=4, dy=P, g_ld=64, dtype=1, vocab=10, dim=64, scale=1.0, padding=-1, out=P, ot=1, ws=P,
             size=need.value):
        return L.asr_embedding_grads(ids, index, tokens, dy, g_ld, dtype, vocab, dim, scale, padding, out, ot, ws, size, None)
    assert back(vocab=0) == OK and back(dim=0) == OK
    assert back(index=-1) == TYPE and back(dtype=2) == TYPE and back(ot=2) == TYPE
    for k in (dict(ids=None), dict(dy=None), dict(out=None), dict(out=P + 1), dict(ws=None), dict(ws=P + 8),
              dict(size=need.value - 1), dict(g_ld=63), dict(scale=float("nan")), dict(vocab=2 ** 28 + 1)):
        assert back(**k) == BAD, k


@pytest.mark.parametrize("tokens,dim", [(1, 1), (33, 4096), (8192, 4096), (16384, 8192), (16385, 40), (10 ** 6, 64), (2 ** 28, 8)])
def test_embedding_workspace_holds_what_it_says(L, tokens, dim):
    """Keys and places of every token, and two rows of binary32 sums a chunk, of which there are at most 8,192."""
    need = asr.asr_embedding_grads_workspace(tokens, dim)
    pitch = -(-dim // 8) * 8
    assert need >= 8 * tokens + 8 * pitch
    assert need <= 16 * tokens + 2 * 4 * pitch * min(tokens, 8192) + 4096 * (-(-tokens // 4096)) + 8192 * 64 + 8192


class Library:
    """Takes the C calls and counts them; none is expected."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            def size(*args):
                args[-1]._obj.value = 1024
                return 0
            return size
        return lambda *args: self.calls.append(name) or 0


@pytest.fixture
def fake(monkeypatch):
    import contextlib
    lib = Library()
    monkeypatch.setattr(_lib, "_lib", lib)
    monkeypatch.setattr(_lib, "_on_device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(_lib, "_stream_handle", lambda d, s: ctypes.c_void_p(None))
    for module in (int8, layers):
        monkeypatch.setattr(module, "_raw_stream", lambda i: 0)
        monkeypatch.setattr(module, "_elsewhere", lambda d: False)
    yield lib
    _lib.asr_layer_norm_grads_workspace.cache_clear()
    _lib.asr_embedding_grads_workspace.cache_clear()


def test_binding_refuses_before_any_call(fake):
    bf, f32 = torch.bfloat16, torch.float32
    x, y = _on(0, 4, 64, dtype=bf), _on(0, 4, 64, dtype=bf)
    q, p = _on(0, 4, 64, dtype=torch.int8), _on(0, 4, 2, dtype=torch.uint8)
    stat, vec, ids = _on(0, 4), _on(0, 64), _on(0, 4, dtype=torch.int64)
    wrong = [
        lambda: asr.asr_checkpoint_int8(x, q, _on(0, 4, 3, dtype=torch.uint8)),
        lambda: asr.asr_checkpoint_int8(x, _on(0, 4, 63, dtype=torch.int8), p),
        lambda: asr.asr_checkpoint_int8(x, q, p, rounding="up"),
        lambda: asr.asr_checkpoint_int8(x, _on(1, 4, 64, dtype=torch.int8), p),
        lambda: asr.asr_checkpoint_int8(_on(0, 4, 64, dtype=torch.float64), q, p),
        lambda: asr.asr_checkpoint_int8(torch.zeros(4, 64), q, p),
        lambda: asr.asr_restore_int8(q, p, _on(0, 4, 65)),
        lambda: asr.asr_activation(x, y, "relu"),
        lambda: asr.asr_activation(x, y, gated=True),
        lambda: asr.asr_activation(x, _on(0, 4, 64)),
        lambda: asr.asr_activation(x, y, keep=(q, q)),
        lambda: asr.asr_activation_grads(x, None, y),
        lambda: asr.asr_activation_grads(x, x, y, kept=(q, p)),
        lambda: asr.asr_activation_grads(x, x, y, gated=True),
        lambda: asr.asr_activation_grads(x, _on(1, 4, 64, dtype=bf), y),
        lambda: asr.asr_layer_norm(x, _on(0, 63), None, y),
        lambda: asr.asr_layer_norm(x, vec, None, _on(0, 4, 64)),
        lambda: asr.asr_layer_norm(x, vec, None, y, stat, _on(0, 5)),
        lambda: asr.asr_layer_norm(x, _on(0, 64, dtype=torch.float16), None, y),
        lambda: asr.asr_layer_norm_grads(x, x, vec, None, stat, y, None, None),
        lambda: asr.asr_layer_norm_grads(x, x, vec, stat, None, y, None, None),
        lambda: asr.asr_layer_norm_grads(x, None, vec, stat, stat, y, None, None),
        lambda: asr.asr_layer_norm_grads(x, x, vec, stat, stat, y, _on(0, 3), None),
        lambda: asr.asr_embedding(_on(0, 4), _on(0, 10, 64, dtype=bf), y),
        lambda: asr.asr_embedding(_on(0, 2, 2, dtype=torch.int64), _on(0, 10, 64, dtype=bf), y),
        lambda: asr.asr_embedding(_on(0, 5, dtype=torch.int64), _on(0, 10, 64, dtype=bf), y),
        lambda: asr.asr_embedding(_on(1, 4, dtype=torch.int64), _on(0, 10, 64, dtype=bf), y),
        lambda: asr.asr_embedding_grads(ids, x, _on(0, 10, 63)),
        lambda: asr.asr_embedding_grads(ids, x, _on(0, 10, 64), padding_idx=10),
        lambda: asr.asr_embedding_grads(ids, x, _on(0, 640)),
        lambda: asr.checkpoint_int8(_on(0, 64)),
        lambda: asr.checkpoint_int8(x[:, ::2]),
        lambda: asr.checkpoint_int8(x, rounding="down"),
        lambda: asr.activation(_on(0, 4, 63), gated=True),
        lambda: asr.activation(x, save="bf16"),
        lambda: asr.activation(x, "tanh"),
        lambda: asr.activation_grads(x, _on(0, 4, 65, dtype=bf)),
        lambda: asr.activation_grads(x, _on(0, 4, 64)),
        lambda: asr.layer_norm(x, _on(1, 64)),
        lambda: asr.layer_norm(x, save="yes"),
        lambda: asr.embedding(ids, _on(1, 10, 64)),
        lambda: asr.embedding_grads(_on(0, 3, dtype=torch.int64), x, 10),
        lambda: asr.embedding_grads(ids, x, 10, padding_idx=-1),
        lambda: asr.embedding_grads(ids, x, 10, dtype=torch.float16),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises((ValueError, TypeError)):
            call()
        assert not fake.calls, i
    # the ones they differ from
    asr.asr_checkpoint_int8(x, q, p)
    asr.asr_restore_int8(q, p, y)
    asr.asr_activation(_on(0, 4, 128, dtype=bf), y, gated=True)
    asr.asr_activation_grads(x, None, y, kept=(q, p))
    asr.asr_layer_norm(x, vec, None, y, stat, stat)
    asr.asr_embedding(ids, _on(0, 10, 64, dtype=bf), y)
    assert len(fake.calls) == 6


def test_a_checkpoint_of_another_shape_or_device_is_refused(fake):
    def made(device, rows, width, cols):
        return int8.Int8Checkpoint(_on(device, rows, width, dtype=torch.uint8), cols, torch.bfloat16)
    dy = _on(0, 4, 64, dtype=torch.bfloat16)
    for bad in (made(1, 4, 80, 64), made(0, 5, 80, 64), made(0, 4, 80, 60), made(0, 4, 96, 64)):
        with pytest.raises(ValueError):
            asr.activation_grads(dy, bad)
    with pytest.raises(ValueError):
        asr.restore_int8(int8.Int8Checkpoint(torch.zeros(4, 80, dtype=torch.uint8), 64, torch.bfloat16))
    with pytest.raises(TypeError):
        asr.restore_int8(made(0, 4, 80, 64), torch.float16)
    assert not fake.calls


# ------------------------------------------------------------------ modules

def test_module_arguments():
    for call in (lambda: asr.Activation("relu"), lambda: asr.Activation(save=None), lambda: asr.Activation(rounding="up"),
                 lambda: asr.LayerNorm(8, save="half"), lambda: asr.LayerNorm(8, rounding="up"),
                 lambda: asr.Embedding(8, 4, padding_idx=8), lambda: asr.Embedding(8, 4, padding_idx=-1),
                 lambda: asr.Int8Linear(8, 4, save="fp8")):
        with pytest.raises(ValueError):
            call()
    norm = asr.LayerNorm(8, dtype=torch.float32)
    with pytest.raises(ValueError, match="last dimension"):
        norm(torch.zeros(4, 6))
    assert asr.LayerNorm(8).bias is not None and asr.LayerNorm(8, centred=False).bias is None
    assert asr.LayerNorm(8, bias=False).bias is None and asr.LayerNorm(8, centred=False, bias=True).bias is not None


def test_parameters_are_those_of_torchs_modules():
    norm = asr.LayerNorm(8, dtype=torch.float32)
    assert not norm.load_state_dict(torch.nn.LayerNorm(8).state_dict()).missing_keys and norm.calls == 0
    e = asr.Embedding(10, 4, dtype=torch.float32)
    other = torch.nn.Embedding(10, 4)
    e.load_state_dict(other.state_dict())
    assert torch.equal(e.weight, other.weight)


@pytest.fixture
def plain(monkeypatch):
    """The modules' calls as plain torch on the CPU; what each was asked for."""
    seen = []

    def activation(x, function="silu", *, gated=False, save=None, rounding="rne", step=0, seed=0):
        seen.append((save, rounding, step, seed))
        n = x.shape[1] // 2 if gated else x.shape[1]
        y = torch.nn.functional.silu(x[:, :n]) * (x[:, n:] if gated else 1)
        kept = int8.Int8Checkpoint(x.clone(), x.shape[1], x.dtype) if save == "int8" else x
        return y if save is None else (y, kept)

    def activation_grads(dy, saved, function="silu", *, gated=False):
        x = (saved.data if isinstance(saved, int8.Int8Checkpoint) else saved).detach().requires_grad_()
        with torch.enable_grad():
            y = activation(x, function, gated=gated)
        return torch.autograd.grad(y, x, dy)[0]

    def layer_norm(x, weight=None, bias=None, *, eps=1e-5, centred=True, save=None, rounding="rne", step=0, seed=0):
        seen.append((save, rounding, step, seed))
        y = torch.nn.functional.layer_norm(x, x.shape[1:], weight, bias, eps)
        return y if save is None else (y, layers.NormSaved(x, torch.zeros(2, x.shape[0])))

    def layer_norm_grads(dy, saved, weight=None, *, need_dx=True, need_dweight=True, need_dbias=True, dbias_dtype=None):
        return (dy.clone() if need_dx else None, dy.sum(0) if need_dweight else None, dy.sum(0) if need_dbias else None)

    for f in (activation, activation_grads, layer_norm, layer_norm_grads):
        monkeypatch.setattr(layers, f.__name__, f)
    return seen


def test_passes_are_counted_where_gradients_are_recorded(plain):
    act = asr.Activation(gated=True, rounding="sr", seed=5)
    x = torch.randn(3, 2, 8, requires_grad=True)
    act(x).sum().backward()
    with torch.no_grad():
        act(x)
    act(x.detach())
    act(x)
    # the plain backward pass's own call, and those that record nothing, save nothing
    assert plain == [("int8", "sr", 1, 5), (None, "rne", 0, 0), (None, "rne", 0, 0), (None, "rne", 0, 0), ("int8", "sr", 2, 5)]
    assert act.calls == 2
    other = asr.Activation(gated=True)
    other.load_state_dict(act.state_dict())
    assert other.calls == 2
    want = x.detach().clone().requires_grad_()
    (torch.nn.functional.silu(want[..., :4]) * want[..., 4:]).sum().backward()
    assert torch.allclose(x.grad, want.grad, atol=1e-6)


@pytest.mark.parametrize("shape", [(8,), (5, 8), (2, 3, 8), (0, 8), (2, 0, 8)])
def test_shapes(plain, shape):
    norm, act = asr.LayerNorm(8, dtype=torch.float32), asr.Activation(gated=True)
    x = torch.randn(shape).requires_grad_()
    y = norm(x)
    assert y.shape == x.shape
    z = act(y)
    assert z.shape == shape[:-1] + (4,)
    z.sum().backward()
    assert x.grad.shape == x.shape and norm.weight.grad.shape == (8,) and norm.bias.grad.shape == (8,)


def test_second_derivatives_are_refused(plain):
    x = torch.randn(4, 8, requires_grad=True)
    (g,) = torch.autograd.grad(asr.Activation()(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_int8_linear_keeps_its_input_in_8_bits(monkeypatch):
    """What is saved is the checkpoint, not the input; nothing is kept where only dx is wanted or no gradient is recorded."""
    made = []

    def checkpoint(x, *, rounding, step, seed):
        made.append((rounding, step, seed))
        return int8.Int8Checkpoint(x.detach().clone(), x.shape[1], x.dtype)

    def quantize(w, q, scale, **kw):
        scale.fill_(1 / 127)
        q.copy_(torch.round(w.detach().float() * 127))
        return q, scale

    def grads(dy, x, w, dx, dw, **kw):
        if dx is not None:
            dx.copy_(dy.float() @ w.float())
        if dw is not None:
            dw.copy_(dy.float().t() @ x.float())

    monkeypatch.setattr(int8, "checkpoint_int8", checkpoint)
    monkeypatch.setattr(int8, "restore_int8", lambda c, dtype=None: c.data)
    monkeypatch.setattr(int8, "asr_quantize_int8", quantize)
    monkeypatch.setattr(int8, "asr_linear_int8", lambda x, q, s, y, **kw: y.copy_(x.float() @ (q.float() * s[:, None]).t()))
    monkeypatch.setattr(int8, "asr_linear_int8_grads", grads)
    layer = int8.Int8Linear(8, 6, dtype=torch.float32, save="int8", seed=3)
    x = torch.randn(5, 8, requires_grad=True)
    y = layer(x)
    saved = y.grad_fn.next_functions[0][0].saved_tensors if not hasattr(y.grad_fn, "saved_tensors") else y.grad_fn.saved_tensors
    assert all(t.data_ptr() != x.data_ptr() for t in saved)
    g = torch.randn(5, 6)
    y.backward(g.to(y.dtype))
    assert made == [("sr", 1, 3)]
    assert torch.allclose(layer.weight.grad, g.bfloat16().float().t() @ x.detach(), rtol=2 ** -6, atol=2 ** -6)
    with torch.no_grad():
        layer(x)
    layer.weight.requires_grad_(False)
    layer(x).sum().backward()
    assert len(made) == 1
