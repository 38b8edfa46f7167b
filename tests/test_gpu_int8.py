"""The 8-bit quantiser and product against plain forms: the integers and the
scales bit for bit (numpy binary32, the oracle's Philox words), the product
against the exact integer sum times the scales, rounded the same way."""
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


def _words(orc, n, base, step, seed):
    """Low 16 bits of the Philox words of indices base .. base+n-1."""
    first = base >> 2
    w = orc.philox_fill((n + 7) // 4 + 1, first, step, 0, seed).reshape(-1)
    return (w[base - 4 * first:][:n] & 0xFFFF).astype(np.float32)


def _want_rows(x, bits=None):
    """Scales and integers of the rows of a float32 array, each operation
    rounded to binary32."""
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(x).all(1)
        top = np.abs(x).max(1).astype(np.float32)
        top[np.isnan(x).any(1)] = np.nan
        pre = np.where(top < np.float32(2.0 ** -64), np.float32(2.0 ** 64), np.float32(1)).astype(np.float32)
        inv = np.where((top > 0) & ~bad, np.float32(127) / (top * pre), np.float32(0)).astype(np.float32)
        y = (np.where(bad[:, None], 0, x).astype(np.float32) * pre[:, None]) * inv[:, None]
        if bits is None:
            q = np.rint(y)
        else:
            low = np.floor(y)
            q = low + ((y - low) * np.float32(65536) > bits)
        scale = (top / np.float32(127)).astype(np.float32)
    return np.clip(q, -127, 127).astype(np.int8), scale


ROWS = [(1, 1), (1, 4096), (3, 7), (5, 8), (2, 130), (33, 2049), (700, 515), (64, 8191), (2, 40000)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("axis", ["rows", "columns"])
@pytest.mark.parametrize("rounding", ["rne", "sr"])
@pytest.mark.parametrize("shape", ROWS)
def test_quantise_bit_exact(asr, orc, shape, rounding, axis, dtype):
    import torch
    torch.manual_seed(shape[1] + 7)
    x = torch.randn(shape, device="cuda").to(getattr(torch, dtype))
    rows, cols = shape
    q = asr.int8_empty(*(shape if axis == "rows" else shape[::-1]))
    scale = torch.empty(q.shape[0], device="cuda")
    asr.asr_quantize_int8(x, q, scale, axis=axis, rounding=rounding, base_index=13, step=5, seed=99)
    xn = x.float().cpu().numpy()
    bits = _words(orc, rows * cols, 13, 5, 99).reshape(shape) if rounding == "sr" else None
    if axis == "columns":
        xn = np.ascontiguousarray(xn.T)
        bits = None if bits is None else bits.T
    wq, ws = _want_rows(xn, bits)
    assert np.array_equal(q.cpu().numpy(), wq)
    assert_same_bits(host(scale), ws)


@pytest.mark.parametrize("axis", ["rows", "columns"])
def test_quantise_edges(asr, axis):
    """Zeros, subnormals, the largest values, infinities and NaN, a row each."""
    import torch
    x = torch.randn(8, 50)
    x[0] = 0.0
    x[1] *= 1e-44
    x[2] *= 1e38
    x[3, 7] = float("inf")
    x[4, 49] = float("nan")
    x[5] = 0.0
    x[5, 3] = 1e-45
    x[6] = 0.5
    x[7] *= 1e-20
    wq, ws = _want_rows(x.numpy())
    xd = x.cuda() if axis == "rows" else x.t().contiguous().cuda()
    q, scale = asr.int8_empty(8, 50), torch.empty(8, device="cuda")
    asr.asr_quantize_int8(xd, q, scale, axis=axis)
    assert np.array_equal(q.cpu().numpy(), wq)
    assert_same_bits(host(scale), ws)


def test_quantise_strided_and_unaligned(asr):
    """Row pitches, a start off every alignment, an output without padding;
    bytes beside the rows stay as they were."""
    import torch
    store = torch.randn(40, 101, device="cuda")
    x = store[3:30, 5:92]
    wq, ws = _want_rows(x.cpu().numpy())
    for axis in ("rows", "columns"):
        want = wq if axis == "rows" else _want_rows(np.ascontiguousarray(x.t().cpu().numpy()))[0]
        buf = torch.full((want.shape[0], want.shape[1] + 9), 77, dtype=torch.int8, device="cuda")
        q = buf[:, 3:3 + want.shape[1]]
        scale = torch.empty(want.shape[0], device="cuda")
        asr.asr_quantize_int8(x, q, scale, axis=axis)
        assert np.array_equal(q.cpu().numpy(), want)
        assert (buf[:, :3] == 77).all() and (buf[:, 3 + want.shape[1]:] == 77).all()


def _operands(m, n, k, seed, extreme=False):
    import torch
    import stochastic_rounding_gb300 as asr
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    a, b = asr.int8_empty(m, k), asr.int8_empty(n, k)
    if extreme:                      # sums at the ends of their range, and products that differ by one from them
        a.fill_(-128)
        b.fill_(-128)
        a[:, ::97] = 127
        b[:, 1::89] = 127
        a[::3] = 127
    else:
        a.copy_(torch.randint(-128, 128, (m, k), device="cuda", generator=g, dtype=torch.int8))
        b.copy_(torch.randint(-128, 128, (n, k), device="cuda", generator=g, dtype=torch.int8))
    sa = torch.rand(m, device="cuda", generator=g) * 0.01 + 1e-4
    sb = torch.rand(n, device="cuda", generator=g) * 0.01 + 1e-4
    return a, b, sa, sb


def _want_product(a, b, sa, sb):
    s = a.double() @ b.double().t()              # whole numbers below 2^53: exact in any order
    return (s.float() * sa[:, None]) * sb[None]


SIZES = [(1, 1, 1), (1, 16, 16), (1, 257, 4097), (2, 100, 1000), (4, 64, 64), (5, 333, 129), (8, 515, 2048),
         (9, 40, 31), (16, 512, 1024), (17, 256, 1025), (33, 1000, 1365), (64, 300, 5000), (65, 129, 640),
         (128, 256, 128), (129, 257, 1023), (256, 256, 1024), (300, 511, 2049), (777, 1001, 515), (1024, 2048, 4096)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_product_bit_exact(asr, size, dtype):
    import torch
    m, n, k = size
    a, b, sa, sb = _operands(m, n, k, m + n + k)
    c = torch.empty(m, n, device="cuda", dtype=getattr(torch, dtype))
    asr.asr_gemm_int8_sr(a, b, sa, sb, c, rounding="rne")
    want = _want_product(a, b, sa, sb).to(c.dtype)
    assert_same_bits(host(c), host(want))


@pytest.mark.parametrize("size", [(1, 64, 131071), (3, 48, 131071), (20, 40, 70000), (256, 256, 131071), (200, 300, 9000)])
def test_product_exact_at_the_ends_of_the_range(asr, size):
    import torch
    a, b, sa, sb = _operands(*size, 1, extreme=True)
    c = torch.empty(size[0], size[1], device="cuda")
    asr.asr_gemm_int8_sr(a, b, sa, sb, c)
    assert_same_bits(host(c), host(_want_product(a, b, sa, sb)))


@pytest.mark.parametrize("size", [(1, 515, 300), (6, 77, 100), (40, 130, 257), (300, 271, 513),
                                  (33, 130, 1500), (40, 260, 5000)])
def test_product_stochastic_rounding(asr, orc, size):
    import torch
    m, n, k = size
    a, b, sa, sb = _operands(m, n, k, 3)
    c = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)
    asr.asr_gemm_int8_sr(a, b, sa, sb, c, rounding="sr", step=11, seed=2**40 + 5)
    want = orc.sr_fill(_want_product(a, b, sa, sb).cpu().numpy().reshape(-1), 0, 11, 2**40 + 5)
    assert_same_bits(host(c).reshape(-1), want)


@pytest.mark.parametrize("m", [1, 3, 7, 20, 150])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_product_strided_unaligned(asr, m, dtype):
    """Operands and outputs at odd pitches and starts; what lies beside the
    output stays."""
    import torch
    n, k = 143, 333
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    a = torch.randint(-128, 128, (m + 2, k + 11), device="cuda", generator=g, dtype=torch.int8)[1:m + 1, 3:k + 3]
    b = torch.randint(-128, 128, (n + 2, k + 7), device="cuda", generator=g, dtype=torch.int8)[1:n + 1, 1:k + 1]
    sa, sb = torch.rand(m, device="cuda", generator=g), torch.rand(n, device="cuda", generator=g)
    buf = torch.full((m + 2, n + 6), 7.0, device="cuda", dtype=getattr(torch, dtype))
    c = buf[1:m + 1, 3:n + 3]
    asr.asr_gemm_int8_sr(a, b, sa, sb, c, rounding="rne")
    assert_same_bits(host(c.contiguous()), host(_want_product(a, b, sa, sb).to(c.dtype)))
    rest = buf.clone()
    rest[1:m + 1, 3:n + 3] = 7.0
    assert (rest == 7.0).all()


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
@pytest.mark.parametrize("m,n,k", [(2, 70, 2049), (16, 64, 130), (17, 64, 130), (33, 129, 2051), (64, 130, 2048),
                                   (65, 130, 2048), (150, 133, 5001), (256, 40, 8200), (257, 40, 8200), (300, 70, 12400)])
def test_product_weight_at_any_address(asr, m, n, k, shift):
    """A weight whose rows follow one another without a gap, from any byte on to
    the end of its memory, on both sides of the choice between the kernels."""
    import torch
    a, b, sa, sb = _operands(m, n, k, m + k)
    room = torch.empty(shift + n * k, device="cuda", dtype=torch.int8)
    w = room[shift:].view(n, k)
    w.copy_(b)
    c = torch.empty(m, n, device="cuda")
    asr.asr_gemm_int8_sr(a, w, sa, sb, c)
    assert_same_bits(host(c), host(_want_product(a, b, sa, sb)))


@pytest.mark.parametrize("m", [1, 12, 140])
def test_product_scales_that_are_not_finite(asr, m):
    import torch
    a, b, sa, sb = _operands(m, 64, 80, 1)
    a[0] = 0
    sa[0] = float("inf")
    sb[5] = float("nan")
    c = torch.empty(m, 64, device="cuda", dtype=torch.bfloat16)
    asr.asr_gemm_int8_sr(a, b, sa, sb, c, rounding="sr", step=1)
    assert c[0].isnan().all() and c[:, 5].isnan().all()
    rest = c[1:, [j for j in range(64) if j != 5]]
    assert rest.isfinite().all()


def test_product_empty_and_streams(asr):
    import torch
    a, b, sa, sb = _operands(40, 50, 60, 1)
    c = torch.full((0, 50), 3.0, device="cuda")
    asr.asr_gemm_int8_sr(a[:0], b, sa[:0], sb, c)
    c = torch.full((40, 0), 3.0, device="cuda")
    asr.asr_gemm_int8_sr(a, b[:0], sa, sb[:0], c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = torch.empty(40, 50, device="cuda")
    asr.asr_gemm_int8_sr(a, b, sa, sb, c, stream=s)
    s.synchronize()
    assert_same_bits(host(c), host(_want_product(a, b, sa, sb)))


def test_linear_and_its_gradients(asr):
    """y, dx and dw are the exact products of the quantised operands, times the
    scales, rounded to bf16: bit for bit."""
    import torch
    torch.manual_seed(0)
    t, n, k = 130, 271, 515
    x = torch.randn(t, k, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(n, k, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(t, n, device="cuda", dtype=torch.bfloat16)

    def quant(v, axis, **kw):
        q = asr.int8_empty(*(v.shape if axis == "rows" else v.shape[::-1]))
        s = torch.empty(q.shape[0], device="cuda")
        return asr.asr_quantize_int8(v, q, s, axis=axis, **kw)
    qw, sw = quant(w, "rows")
    y = asr.int8_linear(x, qw, sw)
    dx, dw = asr.int8_linear_grads(dy, x, w, step=3, seed=9)
    sr = dict(rounding="sr", step=3, seed=9)
    operands = [(quant(x, "rows"), (qw, sw)), (quant(dy, "rows", **sr), quant(w, "columns")),
                (quant(dy, "columns", **sr), quant(x, "columns"))]
    for got, ((a, sa), (b, sb)) in zip((y, dx, dw), operands):
        assert_same_bits(host(got), host(_want_product(a, b, sa, sb).bfloat16()))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("size", [(1, 300, 515), (40, 64, 1000), (200, 130, 77), (513, 1001, 257)])
def test_linear_from_either_type_strided(asr, dtype, size):
    """The one call gives what the quantiser and the product give, on strided
    views; each gradient alone as both together."""
    import torch
    torch.manual_seed(size[1])
    t, n, k = size
    mk = lambda r, c: torch.randn(r + 1, c + 5, device="cuda").to(getattr(torch, dtype))[1:, 2:c + 2]  # noqa: E731
    x, w, dy = mk(t, k), mk(n, k), mk(t, n)
    qw, sw = asr.asr_quantize_int8(w, asr.int8_empty(n, k), torch.empty(n, device="cuda"))
    qx, sx = asr.asr_quantize_int8(x, asr.int8_empty(t, k), torch.empty(t, device="cuda"))
    y = torch.empty(t, n, device="cuda")
    asr.int8_linear(x, qw, sw, out=y)
    assert_same_bits(host(y), host(_want_product(qx, qw, sx, sw)))
    dx, dw = asr.int8_linear_grads(dy, x, w, step=1, seed=2)
    a, sa = asr.asr_quantize_int8(dy, asr.int8_empty(t, n), torch.empty(t, device="cuda"), rounding="sr", step=1, seed=2)
    b, sb = asr.asr_quantize_int8(w, asr.int8_empty(k, n), torch.empty(k, device="cuda"), axis="columns")
    assert_same_bits(host(dx), host(_want_product(a, b, sa, sb).bfloat16()))
    only, none = asr.int8_linear_grads(dy, x, w, step=1, seed=2, need_dw=False)
    assert none is None and torch.equal(only, dx)
    none, only = asr.int8_linear_grads(dy, x, w, step=1, seed=2, need_dx=False)
    assert none is None and torch.equal(only, dw)


@pytest.mark.parametrize("tokens", [2, 30, 200])
def test_captured_into_a_graph(asr, tokens):
    """A replay gives the direct calls' bits, on inputs that changed since the capture."""
    import torch
    torch.manual_seed(tokens)
    n, k = 300, 1030
    w = torch.randn(n, k, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(tokens, k, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(tokens, n, device="cuda", dtype=torch.bfloat16)
    qw, sw = asr.int8_empty(n, k), torch.empty(n, device="cuda")
    y, dx, dw = (torch.empty(*s, device="cuda", dtype=torch.bfloat16) for s in ((tokens, n), (tokens, k), (n, k)))

    def call():
        asr.asr_quantize_int8(w, qw, sw)
        asr.int8_linear(x, qw, sw, out=y, rounding="sr", step=1)
        asr.asr_linear_int8_grads(dy, x, w, dx, dw, step=2)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in (w, x, dy):
        t.copy_(torch.randn_like(t))
    graph.replay()
    torch.cuda.synchronize()
    got = [host(t) for t in (y, dx, dw, sw)]
    call()
    for a, b in zip(got, (y, dx, dw, sw)):
        assert_same_bits(a, host(b))


def test_linear_module_gradients_against_differences(asr):
    """Int8Linear's gradients along a direction against differences of the
    unquantised layer.  One entry of an operand is off by at most half a step
    (nearest; a whole one where rounded stochastically), a step is top / 127 and
    top < 5 for these normal values, so a sum of K products of unit variance
    has a standard error below 5/127 sqrt(K) on top of its sqrt(K); averaged
    over the direction's entries, four standard errors relative to the
    derivative's own size stay below a tenth."""
    import torch
    torch.manual_seed(1)
    layer = asr.Int8Linear(256, 192, seed=5, device="cuda")
    x = torch.randn(64, 256, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    target = torch.randn(64, 192, device="cuda")
    y = layer(x)
    loss = ((y.float() - target) ** 2).sum()
    loss.backward()

    def plain(xv, wv):
        return ((xv @ wv.t() - target.double()) ** 2).sum()
    for p, which in ((x, 0), (layer.weight, 1)):
        d = p.grad.double()
        d = d / d.norm()
        h = 1e-4 * p.detach().double().norm()
        v = [x.detach().double(), layer.weight.detach().double()]
        up, down = list(v), list(v)
        up[which], down[which] = v[which] + h * d, v[which] - h * d
        diff = float((plain(*up) - plain(*down)) / (2 * h))
        got = float((p.grad.double() * d).sum())
        assert abs(got - diff) <= 0.1 * abs(diff)
    # repeats bit for bit
    again = asr.Int8Linear(256, 192, seed=5, device="cuda")
    again.weight.data.copy_(layer.weight.data)
    x2 = x.detach().clone().requires_grad_()
    ((again(x2).float() - target) ** 2).sum().backward()
    assert torch.equal(x2.grad, x.grad) and torch.equal(again.weight.grad, layer.weight.grad)


def test_refusals(asr):
    import torch
    a, b, sa, sb = _operands(4, 6, 32, 1)
    c = torch.empty(4, 6, device="cuda")
    with pytest.raises(ValueError):
        asr.asr_gemm_int8_sr(a, b[:, :16], sa, sb, c)
    with pytest.raises(ValueError):
        asr.asr_gemm_int8_sr(a, b, sa[:3], sb, c)
    with pytest.raises(ValueError):
        asr.asr_gemm_int8_sr(a, b, sa, sb, c, rounding="up")
    with pytest.raises(TypeError):
        asr.asr_gemm_int8_sr(a.float(), b, sa, sb, c)
    with pytest.raises(ValueError):
        asr.asr_gemm_int8_sr(a.cpu(), b, sa, sb, c)
    with pytest.raises(ValueError):
        asr.asr_gemm_int8_sr(a, b, sa, sb, c.t().contiguous().t())
    a2, b2, sa2, sb2 = _operands(100, 6, 32, 1)      # with many rows the product needs a workspace
    with pytest.raises(ValueError):
        asr.asr_gemm_int8_sr(a2, b2, sa2, sb2, torch.empty(100, 6, device="cuda"),
                             workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        asr.asr_quantize_int8(c, asr.int8_empty(4, 6), sa, axis="both")
    with pytest.raises(ValueError):
        asr.asr_quantize_int8(c, asr.int8_empty(4, 6), sa, axis="columns")
