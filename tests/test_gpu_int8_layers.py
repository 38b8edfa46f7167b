"""The linear layer's 8-bit calls and the module on them, beyond single
products: calls one after another, gradients on their own, the module's inputs
and state."""
import numpy as np
import pytest

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


def _want_product(a, b, sa, sb):
    """Of int8 matrices, as the product is defined: the exact sum, then binary32."""
    s = a.double() @ b.double().t()              # whole numbers below 2^53: exact in any order
    return (s.float() * sa[:, None]) * sb[None]


def _quantised(asr, v, axis="rows", **kw):
    import torch
    q = asr.int8_empty(*(v.shape if axis == "rows" else v.shape[::-1]))
    return asr.asr_quantize_int8(v, q, torch.empty(q.shape[0], device="cuda"), axis=axis, **kw)


def test_scales_of_one_call_after_another(asr):
    """Calls in a row through one workspace, of operands whose scales differ by
    powers of two: each has the scales of its own operands, not those that the
    same memory held for the call before."""
    import torch
    torch.manual_seed(1)
    t, n, k = 300, 400, 260
    x, w, dy = (torch.randn(*s, device="cuda").to(torch.bfloat16) for s in ((t, k), (n, k), (t, n)))
    qw, sw = _quantised(asr, w)
    size = max(asr.asr_linear_int8_workspace(t, n, k), asr.asr_linear_int8_grads_workspace(t, n, k))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    y1 = asr.asr_linear_int8(x, qw, sw, torch.empty(t, n, device="cuda"), workspace=ws)
    dx1, dw1 = asr.int8_linear_grads(dy, x, w, step=1)
    xs, dys, ys, dxs, dws = [], [], [], [], []
    scales = [2.0 ** (i % 7 - 3) for i in range(40)]
    for f in scales:
        xs.append(x * f)
        dys.append(dy * f)
        ys.append(torch.empty(t, n, device="cuda"))
        dxs.append(torch.empty(t, k, device="cuda", dtype=torch.bfloat16))
        dws.append(torch.empty(n, k, device="cuda", dtype=torch.bfloat16))
    for a, d, y, gx, gw in zip(xs, dys, ys, dxs, dws):
        asr.asr_linear_int8(a, qw, sw, y, workspace=ws)
        asr.asr_linear_int8_grads(d, a, w, gx, gw, step=1, workspace=ws)
    for f, y, gx, gw in zip(scales, ys, dxs, dws):
        assert torch.equal(y, y1 * f)
        assert torch.equal(gx, dx1 * f)
        assert torch.equal(gw, dw1 * (f * f))


def test_module_inputs_of_any_layout(asr):
    """Transposed and broadcast inputs, and a transposed weight, give what their
    contiguous copies give."""
    import torch
    torch.manual_seed(2)
    base = torch.randn(72, 40, device="cuda", dtype=torch.bfloat16)
    inputs = [torch.randn(1, 72, 50, device="cuda", dtype=torch.bfloat16).transpose(1, 2),
              torch.randn(1, 72, device="cuda", dtype=torch.bfloat16).expand(50, 72)]
    for x in inputs:
        got = []
        for copy in (False, True):
            layer = asr.Int8Linear(72, 40, seed=3, device="cuda")
            layer.weight = torch.nn.Parameter(base.t().contiguous() if copy else base.t())
            v = (x.contiguous() if copy else x).detach().requires_grad_()
            y = layer(v)
            y.float().square().sum().backward()
            got.append([host(t.detach().contiguous()) for t in (y, v.grad, layer.weight.grad)])
        for a, b in zip(*got):
            assert_same_bits(a, b)


def test_a_run_resumed_from_a_checkpoint_repeats(asr):
    """Six steps in one go, and three, a checkpoint (saved and loaded), evaluation
    and three more: the same weights and momentum, bit for bit."""
    import io
    import torch
    rows = [torch.randn(48, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).bfloat16()
            for i in range(6)]

    def make():
        torch.manual_seed(4)
        net = torch.nn.Sequential(asr.Int8Linear(64, 96, seed=11, device="cuda"), torch.nn.ReLU(),
                                  asr.Int8Linear(96, 64, seed=12, device="cuda"))
        return net, asr.MuonSR(net.parameters(), lr=0.02, seed=13)

    def steps(net, opt, batches):
        for x in batches:
            opt.zero_grad()
            (net(x).float() - x.float()).square().mean().backward()
            opt.step()
    net, opt = make()
    steps(net, opt, rows)
    half, half_opt = make()
    steps(half, half_opt, rows[:3])
    with torch.no_grad():
        half(rows[0])
    file = io.BytesIO()
    torch.save({"net": half.state_dict(), "opt": half_opt.state_dict()}, file)
    file.seek(0)
    saved = torch.load(file, weights_only=True)
    rest, rest_opt = make()
    rest.load_state_dict(saved["net"])
    rest_opt.load_state_dict(saved["opt"])
    steps(rest, rest_opt, rows[3:])
    for p, q in zip(net.parameters(), rest.parameters()):
        assert_same_bits(host(p), host(q))
        assert_same_bits(host(opt.state[p]["momentum_buffer"]), host(rest_opt.state[q]["momentum_buffer"]))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("size", [(131072, 40, 72), (150001, 72, 40), (24, 151936, 200), (300, 131073, 272)])
def test_gradients_of_long_sums(asr, size, dtype):
    """More tokens, or outputs (a vocabulary), than int32 sums can hold: exact, of
    random operands and of constant ones (whose sums pass 2^31)."""
    import torch
    t, n, k = size
    torch.manual_seed(n)
    for constant in (False, True):
        mk = lambda *s: (torch.full(s, 0.75, device="cuda") if constant else torch.randn(s, device="cuda")  # noqa: E731
                         ).to(getattr(torch, dtype))
        dy, x, w = mk(t, n), mk(t, k), mk(n, k)
        dx, dw = asr.int8_linear_grads(dy, x, w, step=2, seed=5)
        sr = dict(rounding="sr", step=2, seed=5)
        a, sa = _quantised(asr, dy, **sr)
        b, sb = _quantised(asr, w, axis="columns")
        assert_same_bits(host(dx), host(_want_product(a, b, sa, sb).bfloat16()))
        a, sa = _quantised(asr, dy, axis="columns", **sr)
        b, sb = _quantised(asr, x, axis="columns")
        assert_same_bits(host(dw), host(_want_product(a, b, sa, sb).bfloat16()))
        assert not constant or (a == 127).all() and (b == 127).all()


@pytest.mark.parametrize("axis", ["rows", "columns"])
def test_quantise_rows_of_no_elements(asr, axis):
    """Their scales are those of zeros, not what the memory held."""
    import torch
    x = torch.empty((300, 0) if axis == "rows" else (0, 300), device="cuda")
    scale = torch.full((300,), 3.0, device="cuda")
    asr.asr_quantize_int8(x, asr.int8_empty(300, 0), scale, axis=axis)
    assert (scale == 0).all()
    none = torch.empty((0, 5) if axis == "rows" else (5, 0), device="cuda")
    asr.asr_quantize_int8(none, asr.int8_empty(0, 5), scale[:0], axis=axis)
    assert (scale == 0).all()


@pytest.mark.parametrize("axis", ["rows", "columns"])
def test_stochastic_comparison_is_exact(asr, orc, axis):
    """Fractions just above a random number, of values below zero: y - floor(y)
    rounded to binary32 would come out equal to it, and the integer one too low."""
    import torch
    rows, cols, step, seed = 64, 512, 3, 21
    words = (orc.philox_fill(rows * cols // 4, 0, step, 0, seed).reshape(rows, cols) & 0xFFFF).astype(np.float64)
    near = words >= 49152                                   # 24 bits hold 65536 - r - 2^-10
    rng = np.random.default_rng(0)
    x = np.where(near, -(65536 - words - 2.0 ** -10) / 65536, rng.normal(size=words.shape).astype(np.float32))
    line = (slice(None), 0) if axis == "rows" else (0, slice(None))
    x[line], near[line] = 127.0, False                      # scale 1, so that y = x
    x = x.astype(np.float32)
    y = x.astype(np.float64)
    low = np.floor(y)
    want = low + (65536 * (y - low) > words)
    rounded = np.floor(x) + ((x - np.floor(x)) * np.float32(65536) > words.astype(np.float32))
    assert near.sum() > 5000 and (want[near] == 0).all() and (rounded[near] == -1).all()
    q, scale = _quantised(asr, torch.from_numpy(x).cuda(), axis, rounding="sr", step=step, seed=seed)
    assert (scale == 1).all()
    assert np.array_equal(q.cpu().numpy() if axis == "rows" else q.t().cpu().numpy(), want.astype(np.int8))


# Tiles of 256 x 256 on 76 pairs of SMs, whole rounds of them and what is left: 0 and
# 50 (whole tiles), 1 and 14 (in quarters), 1 and 24 (in halves), 2 and 68, 4 and 37.
@pytest.mark.parametrize("size", [(1277, 2500, 1100), (2300, 2560, 130), (2300, 2700, 2049), (2309, 5500, 1025),
                                  (2600, 7800, 515)])
def test_products_of_several_rounds_of_tiles(asr, orc, size):
    import torch
    m, n, k = size
    g = torch.Generator(device="cuda").manual_seed(m)
    a, b = asr.int8_empty(m, k), asr.int8_empty(n, k)
    for v in (a, b):
        v.copy_(torch.randint(-128, 128, v.shape, device="cuda", generator=g, dtype=torch.int8))
    sa, sb = (torch.rand(s, device="cuda", generator=g) + 0.5 for s in (m, n))
    want = _want_product(a, b, sa, sb)
    c = torch.empty(m, n, device="cuda")
    asr.asr_gemm_int8_sr(a, b, sa, sb, c)
    assert_same_bits(host(c), host(want))
    pitched = torch.full((m, n + 3), 7.0, device="cuda", dtype=torch.bfloat16)
    asr.asr_gemm_int8_sr(a, b, sa, sb, pitched[:, :n], rounding="sr", step=3, seed=8)
    assert_same_bits(host(pitched[:, :n].contiguous()).reshape(-1), orc.sr_fill(host(want).reshape(-1), 0, 3, 8))
    assert (pitched[:, n:] == 7.0).all()


# Weights of more rows than the tests of single products have: dot products of one CTA a
# row block, stretches of pieces over several row blocks, passes over the weight.
@pytest.mark.parametrize("size", [(1, 14336, 4096), (3, 20001, 1030), (4, 9700, 2050), (7, 30000, 515), (33, 14336, 4096),
                                  (128, 9001, 4096), (200, 5000, 8192), (16, 40003, 130)])
def test_few_rows_with_large_weights(asr, size):
    import torch
    m, n, k = size
    torch.manual_seed(n)
    x = torch.randn(m, k, device="cuda").bfloat16()
    (a, sa), (b, sb) = _quantised(asr, x), _quantised(asr, torch.randn(n, k, device="cuda"))
    want = _want_product(a, b, sa, sb)
    c, y = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    asr.asr_gemm_int8_sr(a, b, sa, sb, c)
    assert_same_bits(host(c), host(want))
    asr.int8_linear(x, b, sb, out=y)
    assert_same_bits(host(y), host(want))


# The same of two products in a launch, either first; 1, 2, 4, 8, 16 and 32 rows a warp of
# the quantiser, the last of them part empty.
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("size", [(517, 901, 515), (701, 1301, 901), (1285, 2563, 1285), (2051, 1031, 2053),
                                  (2051, 4104, 2064), (2051, 4102, 2060), (4102, 2051, 2064), (8201, 1030, 1029), (4101, 8203, 2056)])
def test_gradients_of_several_rounds_of_tiles(asr, size, dtype):
    import torch
    t, n, k = size
    torch.manual_seed(t)
    dy, x, w = (torch.randn(*s, device="cuda").to(getattr(torch, dtype)) for s in ((t, n), (t, k), (n, k)))
    dx, dw = asr.int8_linear_grads(dy, x, w, step=4, seed=6)
    sr = dict(rounding="sr", step=4, seed=6)
    (a, sa), (b, sb) = _quantised(asr, dy, **sr), _quantised(asr, w, "columns")
    assert_same_bits(host(dx), host(_want_product(a, b, sa, sb).bfloat16()))
    (a, sa), (b, sb) = _quantised(asr, dy, "columns", **sr), _quantised(asr, x, "columns")
    assert_same_bits(host(dw), host(_want_product(a, b, sa, sb).bfloat16()))
    assert torch.equal(asr.int8_linear_grads(dy, x, w, step=4, seed=6, need_dw=False)[0], dx)
    assert torch.equal(asr.int8_linear_grads(dy, x, w, step=4, seed=6, need_dx=False)[1], dw)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("size", [(1, 300, 515), (40, 64, 1000), (200, 130, 77), (513, 1001, 257), (1285, 515, 1365)])
def test_both_gradients_of_strided_operands(asr, dtype, size):
    """Views at odd starts and pitches: each gradient from the quantiser's integers."""
    import torch
    torch.manual_seed(size[1])
    t, n, k = size
    mk = lambda r, c: torch.randn(r + 1, c + 5, device="cuda").to(getattr(torch, dtype))[1:, 2:c + 2]  # noqa: E731
    x, w, dy = mk(t, k), mk(n, k), mk(t, n)
    dx, dw = asr.int8_linear_grads(dy, x, w, step=1, seed=2)
    sr = dict(rounding="sr", step=1, seed=2)
    (a, sa), (b, sb) = _quantised(asr, dy, **sr), _quantised(asr, w, "columns")
    assert_same_bits(host(dx), host(_want_product(a, b, sa, sb).bfloat16()))
    (a, sa), (b, sb) = _quantised(asr, dy, "columns", **sr), _quantised(asr, x, "columns")
    assert_same_bits(host(dw), host(_want_product(a, b, sa, sb).bfloat16()))
