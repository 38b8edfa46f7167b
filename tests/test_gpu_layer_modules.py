"""The norm, the activation, the embedding and 8-bit checkpoints as they are used: through autograd, together in a
network that the package's optimizers train, in graphs, on other streams, with workspaces of the caller's."""
import io

import numpy as np
import pytest

import layer_reference as ref
from gpu_util import assert_same_bits, host, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asr():
    torch_cuda()
    from stochastic_rounding_gb300 import build
    build.build()
    import stochastic_rounding_gb300 as m
    yield m
    assert m.asr_take_device_error() == 0


def relative(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("save", ["input", "int8"])
@pytest.mark.parametrize("shape", [(24,), (5, 24), (2, 3, 24), (0, 24), (2, 0, 24)])
def test_autograd_is_the_functions(asr, save, shape):
    """A module's gradients are those of the two calls, whatever the input's shape."""
    import torch
    torch.manual_seed(len(shape))
    x = torch.randn(shape, device="cuda")
    rows = x.reshape(x.shape[:-1].numel(), 24)
    norm = asr.LayerNorm(24, save=save, rounding="sr", seed=4, device="cuda", dtype=torch.float32)
    with torch.no_grad():
        norm.weight.copy_(torch.rand(24)), norm.bias.copy_(torch.rand(24))
    a = x.clone().requires_grad_()
    y = norm(a)
    g = torch.randn_like(y)
    y.backward(g)
    w, b = norm.weight.detach(), norm.bias.detach()
    want, saved = asr.layer_norm(rows, w, b, save=save, rounding="sr", step=1, seed=4)
    dx, dw, db = asr.layer_norm_grads(g.reshape(rows.shape), saved, w)
    for p, q in ((y, want), (a.grad, dx), (norm.weight.grad, dw), (norm.bias.grad, db)):
        assert p.numel() == q.numel() and torch.equal(p.reshape(q.shape), q)
    act = asr.Activation("gelu", gated=True, save=save, rounding="sr", seed=9)
    a = x.clone().requires_grad_()
    y = act(a)
    g = torch.randn_like(y)
    y.backward(g)
    want, saved = asr.activation(rows, "gelu", gated=True, save=save, rounding="sr", step=1, seed=9)
    assert torch.equal(y.reshape(want.shape), want)
    assert torch.equal(a.grad.reshape(rows.shape), asr.activation_grads(g.reshape(want.shape), saved, "gelu", gated=True))


def test_inputs_of_any_layout(asr):
    """Transposed, broadcast and strided inputs and output gradients give what their contiguous copies give."""
    import torch
    torch.manual_seed(1)
    inputs = [torch.randn(24, 6, device="cuda").t(), torch.randn(1, 24, device="cuda").expand(6, 24),
              torch.randn(6, 48, device="cuda")[:, ::2], torch.randn(6, 31, device="cuda")[:, 3:27]]
    grads = [torch.randn(12, 6, device="cuda").t(), torch.randn(1, 12, device="cuda").expand(6, 12)]
    for x in inputs:
        for g in grads:
            got = []
            for copy in (False, True):
                norm = asr.LayerNorm(24, device="cuda", dtype=torch.float32, save="int8")
                act = asr.Activation(gated=True)
                a = (x.contiguous() if copy else x).detach().requires_grad_()
                act(norm(a)).backward(g.contiguous() if copy else g)
                got.append([t.contiguous() for t in (a.grad, norm.weight.grad, norm.bias.grad)])
            assert all(torch.equal(p, q) for p, q in zip(*got))
    table = torch.randn(24, 30, device="cuda").t().requires_grad_()
    e = asr.Embedding(30, 24, device="cuda", dtype=torch.float32)
    e.weight = torch.nn.Parameter(table)
    ids = torch.arange(12, device="cuda").reshape(3, 4).t()
    y = e(ids)
    assert torch.equal(y, table.detach()[ids])
    y.backward(torch.randn(1, 1, 24, device="cuda").expand(4, 3, 24))


def test_parameters_that_need_no_gradient(asr):
    import torch
    x = torch.randn(6, 24, device="cuda", requires_grad=True)
    for frozen in ("weight", "bias"):
        norm = asr.LayerNorm(24, device="cuda", dtype=torch.float32)
        getattr(norm, frozen).requires_grad_(False)
        norm(x).square().sum().backward()
        assert getattr(norm, frozen).grad is None
    norm(x.detach()).square().sum().backward()
    with torch.no_grad():
        assert not norm(x).requires_grad and not asr.Activation()(x).requires_grad
    assert not asr.Activation()(x.detach()).requires_grad


def test_what_is_kept_is_smaller(asr):
    """Between forward and backward an 8-bit norm, activation and linear layer hold a little over half of the bf16 input."""
    import torch
    x = torch.randn(2048, 1024, device="cuda").to(torch.bfloat16).requires_grad_()

    def held(module):
        y = module(x)
        del y
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        y = module(x)
        return torch.cuda.memory_allocated() - before - y.numel() * y.element_size()
    size = x.numel()
    for module, more in ((asr.LayerNorm(1024, save="int8", device="cuda"), 2048 * 8), (asr.Activation(), 0),
                         (asr.Int8Linear(1024, 64, save="int8", device="cuda"), 0)):
        assert size <= held(module) <= size * 17 / 16 + more + 4096


def test_int8_linear_from_its_checkpoint(asr):
    """The weight's gradient is the product's with the values that the checkpoint stands for, the input's the same as
    without one."""
    import torch
    torch.manual_seed(3)
    x = torch.randn(300, 200, device="cuda").to(torch.bfloat16)
    g = torch.randn(300, 96, device="cuda").to(torch.bfloat16)
    grads = {}
    for save in ("input", "int8"):
        layer = asr.Int8Linear(200, 96, seed=5, device="cuda", save=save)
        with torch.no_grad():
            layer.weight.copy_(torch.randn(96, 200, generator=torch.Generator().manual_seed(1)) * 0.1)
        a = x.clone().requires_grad_()
        y = layer(a)
        y.backward(g)
        grads[save] = (y, a.grad, layer.weight.grad)
    kept = asr.restore_int8(asr.checkpoint_int8(x, rounding="sr", step=1, seed=5))
    _, dw = asr.int8_linear_grads(g, kept, layer.weight.detach(), step=1, seed=5)
    assert torch.equal(grads["int8"][2], dw)
    assert torch.equal(grads["int8"][0], grads["input"][0]) and torch.equal(grads["int8"][1], grads["input"][1])
    # 127 levels and the powers' bit: a value is off by at most a 64th of its group's largest, a fifth of that on average
    assert relative(grads["int8"][2], grads["input"][2]) < 0.03


class Block:
    """A decoder's feed-forward layer on tokens, all of it kept in bf16 and 8 bits."""

    def __init__(self, asr, width=96, hidden=160, vocab=211, save="int8"):
        import torch
        torch.manual_seed(7)
        self.embed = asr.Embedding(vocab, width, scale=width ** 0.5, padding_idx=0, device="cuda")
        self.norm = asr.LayerNorm(width, centred=False, save=save, rounding="sr", seed=1, device="cuda")
        self.up = asr.Int8Linear(width, 2 * hidden, seed=2, device="cuda", save=save)
        self.act = asr.Activation(gated=True, save=save, rounding="sr", seed=3)
        self.down = asr.Int8Linear(hidden, width, seed=4, device="cuda", save=save)
        self.last = asr.LayerNorm(width, save=save, device="cuda")
        self.net = torch.nn.ModuleList([self.embed, self.norm, self.up, self.act, self.down, self.last])

    def __call__(self, ids):
        h = self.embed(ids)
        h = h + self.down(self.act(self.up(self.norm(h))))
        return self.last(h)


def batches(count, vocab=211):
    import torch
    g = torch.Generator().manual_seed(5)
    return [torch.randint(0, vocab, (4, 40), generator=g).cuda() for _ in range(count)]


def optimizers(asr, block):
    matrices = [block.up.weight, block.down.weight]
    rest = [block.embed.weight, block.norm.weight, block.last.weight, block.last.bias]
    return (asr.MuonSR(matrices, lr=0.01, seed=11),
            asr.AdamWSR(rest, lr=1e-3, seed=11, base_offset=sum(p.numel() for p in matrices)))


def train(block, opts, steps):
    for ids in steps:
        for o in opts:
            o.zero_grad()
        (block(ids).float() - 1).square().mean().backward()
        for o in opts:
            o.step()


def test_a_network_of_them(asr):
    """Gradients of the whole against 64 bits with the weights as they are; the 8-bit products and checkpoints are what
    separates them (at most 3 % each of five in a row, the products' operands and results)."""
    import torch
    block = Block(asr)
    ids = batches(1)[0]
    ids[0, :5] = 0
    y = block(ids)
    g = torch.randn(y.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    y.backward(g)
    params = {n: p.detach().double().requires_grad_() for n, p in
              (("e", block.embed.weight), ("n", block.norm.weight), ("u", block.up.weight), ("d", block.down.weight),
               ("w", block.last.weight), ("b", block.last.bias))}
    h = params["e"][ids.reshape(-1)] * 96 ** 0.5
    z = h * (h.square().mean(1, keepdim=True) + 1e-5).rsqrt() * params["n"]
    z = ref.activation(z @ params["u"].t(), "silu", True) @ params["d"].t()
    h = h + z
    m = h.mean(1, keepdim=True)
    want = (h - m) * ((h - m).square().mean(1, keepdim=True) + 1e-5).rsqrt() * params["w"] + params["b"]
    want.backward(g.double().reshape(want.shape))
    assert relative(y.reshape(want.shape), want) < 0.05
    params["e"].grad[0] = 0
    for p, q in zip((block.embed.weight, block.norm.weight, block.up.weight, block.down.weight, block.last.weight, block.last.bias),
                    params.values()):
        assert relative(p.grad, q.grad) < 0.15
    assert (block.embed.weight.grad[0] == 0).all()
    used = torch.zeros(211, dtype=torch.bool, device="cuda")
    used[ids.reshape(-1)] = True
    assert (block.embed.weight.grad[~used] == 0).all()


def test_a_run_repeats_and_resumes(asr):
    """Four steps in one go, the same again, and two, a checkpoint (saved and loaded), evaluation and two more: the same
    weights bit for bit."""
    import torch
    data = batches(4)

    def weights(block):
        return [host(p) for p in block.net.parameters()]
    whole = Block(asr)
    train(whole, optimizers(asr, whole), data)
    again = Block(asr)
    train(again, optimizers(asr, again), data)
    half = Block(asr)
    opts = optimizers(asr, half)
    train(half, opts, data[:2])
    with torch.no_grad():
        half(data[0])
    file = io.BytesIO()
    torch.save([half.net.state_dict()] + [o.state_dict() for o in opts], file)
    file.seek(0)
    net, *states = torch.load(file, weights_only=True)
    rest = Block(asr)
    rest.net.load_state_dict(net)
    opts = optimizers(asr, rest)
    for o, s in zip(opts, states):
        o.load_state_dict(s)
    train(rest, opts, data[2:])
    for a, b, c in zip(weights(whole), weights(again), weights(rest)):
        assert_same_bits(a, b)
        assert_same_bits(a, c)


def all_calls(asr, inputs, out, ws):
    """Every call that fills a caller's tensors, on these inputs."""
    x, dy, w, ids, dt = inputs
    kw = dict(rounding="sr", step=2, seed=3)
    asr.asr_checkpoint_int8(x, out["q"], out["p"], **kw)
    asr.asr_restore_int8(out["q"], out["p"], out["restored"])
    asr.asr_activation(x, out["act"], gated=True, keep=(out["q2"], out["p2"]), **kw)
    asr.asr_activation_grads(out["act"], None, out["dact"], gated=True, kept=(out["q2"], out["p2"]))
    asr.asr_layer_norm(x, w, None, out["norm"], out["mean"], out["rstd"])
    asr.asr_layer_norm_grads(dy, x, w, out["mean"], out["rstd"], out["dx"], out["dw"], out["db"], workspace=ws[0])
    asr.asr_embedding(ids, dt, out["rows"], scale=2.0)
    asr.asr_embedding_grads(ids, out["rows"], out["dt"], workspace=ws[1])


def buffers(asr, rows, cols, vocab, dtype):
    import torch
    e = lambda *s, t=dtype: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    out = dict(q=asr.int8_empty(rows, cols), p=e(rows, -(-cols // 32), t=torch.uint8), restored=e(rows, cols),
               act=e(rows, cols // 2), q2=asr.int8_empty(rows, cols), p2=e(rows, -(-cols // 32), t=torch.uint8), dact=e(rows, cols),
               norm=e(rows, cols), mean=e(rows, t=torch.float32), rstd=e(rows, t=torch.float32), dx=e(rows, cols), dw=e(cols),
               db=e(cols), rows=e(rows, cols), dt=e(vocab, cols))
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (asr.asr_layer_norm_grads_workspace(rows, cols),
                                                                    asr.asr_embedding_grads_workspace(rows, cols))]
    return out, ws


def inputs_of(rows, cols, vocab, dtype, seed):
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    x, dy = (torch.randn(rows, cols, device="cuda", generator=g).to(dtype) for _ in range(2))
    return (x, dy, torch.rand(cols, device="cuda", generator=g).to(dtype),
            torch.randint(0, vocab, (rows,), device="cuda", generator=g) ** 2 % vocab,
            torch.randn(vocab, cols, device="cuda", generator=g).to(dtype))


SIZES = [(70, 96, 40), (33, 512, 300), (700, 1030, 50), (9, 18000, 7), (20000, 64, 130)]


@pytest.mark.parametrize("rows,cols,vocab", SIZES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_graphs_and_streams(asr, rows, cols, vocab, dtype):
    """Captured and replayed with other inputs, on a stream of their own, by the stream's handle, and two at a time: the
    bits that the calls give one after another."""
    import torch
    dtype = getattr(torch, dtype)
    sets = [inputs_of(rows, cols, vocab, dtype, s) for s in range(3)]
    want = []
    for i in sets:
        out, ws = buffers(asr, rows, cols, vocab, dtype)
        all_calls(asr, i, out, ws)
        want.append({k: v.clone() for k, v in out.items()})
    torch.cuda.synchronize()

    def same(out, n, what):
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(out[k], want[n][k]), (what, k)
    # a graph, replayed three times on inputs copied into the first
    inputs = [t.clone() for t in sets[0]]
    out, ws = buffers(asr, rows, cols, vocab, dtype)
    for v in out.values():
        v.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_calls(asr, inputs, out, ws)
    for n in (1, 2, 0):
        for a, b in zip(inputs, sets[n]):
            a.copy_(b)
        graph.replay()
        same(out, n, "graph")
    # two streams at once, with workspaces of their own
    streams = [torch.cuda.Stream() for _ in range(2)]
    pairs = [buffers(asr, rows, cols, vocab, dtype) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for n, (s, (o, w)) in enumerate(zip(streams, pairs)):
            with torch.cuda.stream(s):
                all_calls(asr, sets[n], o, w)
    for n, (o, _) in enumerate(pairs):
        same(o, n, "streams")
    # a stream given to the call, workspaces made for it
    o, _ = buffers(asr, rows, cols, vocab, dtype)
    x, dy, w, ids, dt = sets[1]
    torch.cuda.synchronize()
    for s in (streams[0], streams[1].cuda_stream):
        asr.asr_layer_norm(x, w, None, o["norm"], o["mean"], o["rstd"], stream=s)
        asr.asr_layer_norm_grads(dy, x, w, o["mean"], o["rstd"], o["dx"], o["dw"], o["db"], stream=s)
        asr.asr_embedding(ids, dt, o["rows"], scale=2.0, stream=s)
        asr.asr_embedding_grads(ids, o["rows"], o["dt"], stream=s)
        torch.cuda.synchronize()
    for k in ("norm", "dx", "dw", "db", "rows", "dt"):
        assert torch.equal(o[k], want[1][k]), k


def test_a_training_step_in_a_graph(asr):
    """The functions' whole forward and backward pass captured: new tensors come from the graph's pool."""
    import torch
    x, dy, w, ids, table = inputs_of(300, 192, 77, torch.bfloat16, 1)

    def step():
        e = asr.embedding(ids, table, scale=3.0)
        y, s = asr.layer_norm(e, w, save="int8", rounding="sr", step=1, seed=2)
        z, t = asr.activation(y, gated=True, save="int8", rounding="sr", step=1, seed=3)
        dy = asr.activation_grads(z, t, gated=True)
        dx, dw, db = asr.layer_norm_grads(dy, s, w)
        return z, dw, db, asr.embedding_grads(ids, dx, 77, scale=3.0, padding_idx=1)
    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_same_workspace_call_after_call(asr):
    """Whatever a workspace held before, and whatever the call before it left there."""
    import torch
    need = max(asr.asr_embedding_grads_workspace(t, 40) for t in (1, 50, 3000, 17000))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for tokens in (3000, 1, 17000, 50, 3000, 17000):
        ids = torch.randint(0, 9, (tokens,), device="cuda", generator=torch.Generator("cuda").manual_seed(tokens))
        dy = torch.randn(tokens, 40, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
        out = torch.empty(9, 40, device="cuda")
        asr.asr_embedding_grads(ids, dy, out, workspace=ws)
        assert torch.equal(out, asr.embedding_grads(ids, dy, 9))
    norm_ws = torch.full((asr.asr_layer_norm_grads_workspace(5000, 100),), 255, dtype=torch.uint8, device="cuda")
    for rows in (5000, 3, 700):
        x = torch.randn(rows, 100, device="cuda")
        y, s = asr.layer_norm(x, save="input")
        dw, db = torch.empty(100, device="cuda"), torch.empty(100, device="cuda")
        asr.asr_layer_norm_grads(y, x, None, s.mean, s.rstd, None, dw, db, workspace=norm_ws)
        want = asr.layer_norm_grads(y, s)
        assert torch.equal(dw, want[1]) and torch.equal(db, want[2])


def test_kernels_that_ran(asr):
    """Each call's launches are counted under its kind: no call is answered by anything else."""
    import torch
    x = torch.randn(40, 64, device="cuda")
    before = asr.asr_kernel_launches()
    c = asr.checkpoint_int8(x)
    asr.restore_int8(c)
    y, s = asr.activation(x, save="int8")
    asr.activation_grads(y, s)
    y, s = asr.layer_norm(x, save="input")
    asr.layer_norm_grads(y, s)
    ids = torch.zeros(40, dtype=torch.int64, device="cuda")
    asr.embedding(ids, x)
    asr.embedding_grads(ids, x, 40)
    after = asr.asr_kernel_launches()
    ran = {k: after[k] - before[k] for k in after if after[k] != before[k]}
    assert ran == {"checkpoint": 2, "activation": 2, "norm": 3, "embedding": 3}


@pytest.mark.parametrize("rows,cols", [(1, 16384), (200_000, 8), (3, 2 ** 20)])
def test_large_and_lopsided(asr, rows, cols):
    """Rows that no block holds, and more rows than blocks, against 64 bits over all values at once."""
    import torch
    x = torch.randn(rows, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    y, s = asr.layer_norm(x, save="int8")
    want, mean, rstd, _ = ref.norm(x, None, None, 1e-5, True)
    assert float((y.double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) + 1e-4
    kept = asr.restore_int8(s.input)
    dx, dw, db = asr.layer_norm_grads(x, s)
    wx, ww, wb = ref.norm_grads(x, kept, None, mean, rstd, True)
    for a, b in ((dx, wx), (dw, ww), (db, wb)):
        assert relative(a, b) <= 2.0 ** -8
    z = asr.activation(x)
    assert relative(z, ref.activation(x, "silu", False)) <= 2.0 ** -8


def test_places_past_32_bits(asr):
    """A matrix of more than 2^32 values, its last rows' codes, powers and random numbers among them."""
    import torch
    rows, cols = 131_200, 32_800
    assert rows * cols > 2 ** 32
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(7, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(torch.bfloat16)
    x[-7:] = tail
    whole = asr.checkpoint_int8(x, rounding="sr", step=1, seed=2)
    part = asr.checkpoint_int8(tail, rounding="sr", step=1, seed=2, base_index=(rows - 7) * (-(-cols // 32) * 32))
    assert torch.equal(whole.q[-7:], part.q) and torch.equal(whole.power[-7:], part.power)
    assert int(whole.data[:-7, :cols].max()) == 0
    back = asr.restore_int8(whole)
    assert torch.equal(back[-7:], asr.restore_int8(part))
    assert torch.equal(asr.activation(x)[-7:], asr.activation(tail))
    y, s = asr.layer_norm(back, save="input")
    want, t = asr.layer_norm(back[-7:].contiguous(), save="input")
    assert torch.equal(y[-7:], want)
    dx = asr.layer_norm_grads(x, s, need_dweight=False, need_dbias=False)[0]
    assert torch.equal(dx[-7:], asr.layer_norm_grads(tail, t, need_dweight=False, need_dbias=False)[0])
    # the same memory as a table: rows past 2^32 values, looked up and summed
    ids = torch.tensor([rows - 1, 5, rows - 7, rows - 1], device="cuda")
    assert torch.equal(asr.embedding(ids, x), x[ids])
    g = asr.embedding_grads(ids, x[ids], rows)
    assert torch.equal(g[-1], 2 * x[-1]) and torch.equal(g[-7], x[-7]) and int(g[:-7].count_nonzero()) == 0
