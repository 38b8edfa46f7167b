"""Newton-Schulz orthogonalisation and the Muon step against 64-bit forms.

Tolerance of an orthogonalised matrix (relative Frobenius distance).  Each of the
`steps` steps rounds S, P and X' to f16: relative perturbations of at most 2^-11
of each entry, which the rest of the iteration carries along with what it does to
the matrix itself (to first order it multiplies small singular values and what
is added to them by the same factor), so 3 * steps * 2^-11 in all, and the
result's bf16 rounding (at most 2^-8 of an entry, evenly spread: 2^-8 / sqrt 3
times about 0.72 in the norm) adds less than 2^-9.  Singular values far below the others are the
exception: a matrix of low rank is tested on its own."""
import numpy as np
import pytest

from gpu_util import assert_same_bits, host, torch_cuda

pytestmark = pytest.mark.gpu
ABC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def asr():
    torch_cuda()
    from stochastic_rounding_gb300 import build
    build.build()
    import stochastic_rounding_gb300 as m
    yield m
    assert m.asr_take_device_error() == 0


def _exact(g, steps=5, abc=ABC, eps=1e-7):
    x = g.double()
    x = x / max(float(x.norm()), eps)
    a, b, c = abc
    for _ in range(steps):
        if x.shape[0] <= x.shape[1]:
            s = x @ x.t()
            x = a * x + (b * s + c * (s @ s)) @ x
        else:
            s = x.t() @ x
            x = a * x + x @ (b * s + c * (s @ s))
    return x


def _bound(steps):
    return 3 * steps * 2.0 ** -11 + 2.0 ** -9


def _far(got, want):
    return float((got.double() - want).norm() / want.norm())


SHAPES = [(1, 1), (1, 17), (17, 1), (2, 3), (8, 8), (16, 64), (65, 31), (96, 160), (127, 129), (128, 128), (129, 400),
          (256, 256), (257, 255), (300, 513), (515, 1365), (1365, 515), (640, 640), (1024, 256), (512, 2048),
          (2048, 520),
          # a smaller side of at most 128: one to eight CTAs a matrix, just below and above their limits
          (128, 512), (128, 513), (100, 1500), (1025, 77), (128, 4096), (4096, 128), (3, 4000), (4000, 1), (128, 4097),
          (4097, 128)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalise(asr, shape, dtype):
    import torch
    torch.manual_seed(shape[0])
    g = (torch.randn(shape, device="cuda") * 1e-3).to(getattr(torch, dtype))
    out = torch.full(shape, 9.0, device="cuda", dtype=torch.bfloat16)
    asr.asr_newton_schulz([(g, out)])
    assert _far(out, _exact(g)) <= _bound(5)


@pytest.mark.parametrize("scale", [1e-15, 1e-4, 1.0, 1e15])
def test_orthogonalise_scale(asr, scale):
    """The size of the gradient does not matter (eps aside)."""
    import torch
    torch.manual_seed(3)
    g = torch.randn(200, 150, device="cuda") * scale
    out = torch.empty(200, 150, device="cuda", dtype=torch.bfloat16)
    asr.asr_newton_schulz([(g, out)], eps=1e-25)
    assert _far(out, _exact(g, eps=1e-25)) <= _bound(5)


@pytest.mark.parametrize("steps,abc", [(1, ABC), (2, ABC), (3, (1.5, -0.5, 0.0)), (12, (1.5, -0.5, 0.0)), (8, (1.875, -1.25, 0.375))])
def test_orthogonalise_other_polynomials(asr, steps, abc):
    import torch
    torch.manual_seed(4)
    g = torch.randn(90, 333, device="cuda")
    out = torch.empty(90, 333, device="cuda", dtype=torch.bfloat16)
    asr.asr_newton_schulz([(g, out)], steps=steps, coefficients=abc)
    assert _far(out, _exact(g, steps, abc)) <= _bound(steps)


def test_orthogonalise_low_rank(asr):
    """Rank 3 of 256: the null space gets rounding errors of X_0 (2^-11 of its
    entries, so a matrix of norm at most 2^-11) raised by at most a^5 = 485 in
    norm, as random directions do: four standard sizes of a random matrix's
    largest singular value, 2 sqrt(n) 2^-11 / sqrt(12) of an entry's size
    1 / n, stay below 0.02."""
    import torch
    torch.manual_seed(5)
    u, v = torch.randn(256, 3, device="cuda"), torch.randn(3, 256, device="cuda")
    g = u @ v
    out = torch.empty(256, 256, device="cuda", dtype=torch.bfloat16)
    asr.asr_newton_schulz([(g, out)])
    want = _exact((u.double() @ v.double()))
    assert torch.linalg.matrix_norm(out.double() - want, 2) <= 4 * 485 * 2 * 16 * 2.0 ** -11 / 12 ** 0.5 / 256 + 2.0 ** -8


def test_orthogonalise_zero_and_not_finite(asr):
    import torch
    g = torch.randn(4, 100, 60, device="cuda")
    g[0] = 0
    g[1, 5, 7] = float("inf")
    g[2, 99, 59] = float("nan")
    out = torch.empty(4, 100, 60, device="cuda", dtype=torch.bfloat16)
    asr.asr_newton_schulz([(g, out)])
    assert (out[0] == 0).all() and out[1].isnan().all() and out[2].isnan().all()
    assert _far(out[3], _exact(g[3])) <= _bound(5)


def test_orthogonalise_stacks_and_strides(asr):
    """A stack, a transposed-looking pitch, odd starts, matrices of several
    shapes in one call: each as on its own, bit for bit, and nothing written
    beside the outputs."""
    import torch
    torch.manual_seed(6)
    store = torch.randn(70, 50, 110, device="cuda")          # more than one launch's stack
    views = [store[:, 1:40, 3:90], store[0, :, :64], store[:2, :7, 50:], torch.randn(120, 45, device="cuda").bfloat16()]
    pairs, bufs = [], []
    for v in views:
        buf = torch.full((*v.shape[:-1], v.shape[-1] + 5), 7.0, device="cuda", dtype=torch.bfloat16)
        bufs.append(buf)
        pairs.append((v, buf[..., 2:2 + v.shape[-1]]))
    asr.asr_newton_schulz(pairs)
    for v, out in pairs:
        flat = v if v.dim() == 3 else v[None]
        for z in range(0, flat.shape[0], 23):
            alone = torch.empty(flat.shape[1:], device="cuda", dtype=torch.bfloat16)
            asr.asr_newton_schulz([(flat[z].contiguous(), alone)])
            got = out[z] if v.dim() == 3 else out
            assert_same_bits(host(got.contiguous()), host(alone))
            assert _far(got, _exact(flat[z])) <= _bound(5)
    for buf in bufs:
        assert (buf[..., :2] == 7).all() and (buf[..., -3:] == 7).all()


def test_orthogonalise_strided_larger(asr):
    """The same on matrices that go through memory: strided views, odd starts."""
    import torch
    torch.manual_seed(16)
    store = torch.randn(3, 210, 333, device="cuda")
    x = store[:, 1:201, 3:320]
    buf = torch.full((3, 200, 325), 7.0, device="cuda", dtype=torch.bfloat16)
    out = buf[..., 2:319]
    asr.asr_newton_schulz([(x, out)])
    for z in range(3):
        alone = torch.empty(200, 317, device="cuda", dtype=torch.bfloat16)
        asr.asr_newton_schulz([(x[z].contiguous(), alone)])
        assert_same_bits(host(out[z].contiguous()), host(alone))
        assert _far(out[z], _exact(x[z])) <= _bound(5)
    assert (buf[..., :2] == 7).all() and (buf[..., 319:] == 7).all()


@pytest.mark.parametrize("shape", [(128, 700), (700, 128), (150, 200)])
def test_orthogonalise_zero_and_not_finite_each_path(asr, shape):
    import torch
    g = torch.randn(4, *shape, device="cuda")
    g[0] = 0
    g[1, 5, 7] = float("-inf")
    g[2, -1, -1] = float("nan")
    out = torch.empty(4, *shape, device="cuda", dtype=torch.bfloat16)
    asr.asr_newton_schulz([(g, out)])
    assert (out[0] == 0).all() and out[1].isnan().all() and out[2].isnan().all()
    assert _far(out[3], _exact(g[3])) <= _bound(5)


def _momentum(m, g, mu, nesterov):
    """binary32, every operation rounded."""
    f = np.float32
    omu = f(1.0 - float(f(mu)))
    m = (m + (omu * (g - m).astype(f)).astype(f)).astype(f)
    u = (g + (f(mu) * (m - g).astype(f)).astype(f)).astype(f) if nesterov else m
    return m, u


@pytest.mark.parametrize("shape", [(40, 64), (65, 33), (2, 100, 256), (3, 515, 130), (1, 300, 300), (2, 2000, 50),
                                   (60, 1103), (1103, 61), (128, 640)])
@pytest.mark.parametrize("gdt", ["float32", "bfloat16"])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("adjust", ["original", "match_rms_adamw", None])
def test_muon_step(asr, shape, gdt, nesterov, adjust):
    """Momentum bit for bit; f32 parameters to the orthogonalised update's
    bound and three binary32 roundings; bf16 parameters bit for bit the
    stochastic rounding of what the f32 form gives."""
    import torch
    torch.manual_seed(shape[-1])
    p = torch.randn(shape, device="cuda") * 0.02
    g = (torch.randn(shape, device="cuda") * 1e-3).to(getattr(torch, gdt))
    m = torch.randn(shape, device="cuda") * 1e-4
    wm, u = _momentum(host(m), g.float().cpu().numpy(), 0.9, nesterov)
    kw = dict(lr=0.03, momentum=0.9, weight_decay=0.2, nesterov=nesterov, adjust=adjust, step=4, seed=77)
    pb = p.to(torch.bfloat16)
    pf, m1, m2 = pb.float(), m.clone(), m.clone()
    before = pf.double()
    asr.asr_muon_sr_multi_tensor([(pf, g, m1, 6)], **kw)
    assert_same_bits(host(m1), wm)
    rows, cols = shape[-2:]
    factor = {None: 1.0, "original": max(1.0, rows / cols) ** 0.5, "match_rms_adamw": 0.2 * max(rows, cols) ** 0.5}[adjust]
    ud = torch.from_numpy(u).cuda().reshape(-1, rows, cols)
    o = torch.stack([_exact(v) for v in ud]).reshape(shape) * (0.03 * factor)
    want = before * (1 - 0.03 * 0.2) - o
    err = pf.double() - want
    assert float(err.norm()) <= _bound(5) * float(o.norm()) + 3 * 2.0 ** -24 * float(want.norm())
    asr.asr_muon_sr_multi_tensor([(pb, g, m2, 6)], **kw)
    assert_same_bits(host(m2), wm)
    rounded = torch.empty_like(pb)
    asr.asr_stochastic_round_bf16(pf, rounded, base_index=6, step=4, seed=77)
    assert_same_bits(host(pb), host(rounded))


def test_muon_rounding_nearest_and_many(asr):
    """Nearest rounding; 70 matrices over several descriptors equal the steps
    one by one; a zero gradient and momentum only decay."""
    import torch
    torch.manual_seed(2)
    mk = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    sets = [(mk(68, 24, 40).bfloat16(), mk(68, 24, 40), mk(68, 24, 40), 5),
            (mk(24, 40).bfloat16(), mk(24, 40), mk(24, 40), 10 ** 12 + 1),
            (mk(40, 24).bfloat16(), torch.zeros(40, 24, device="cuda"), torch.zeros(40, 24, device="cuda"), 0)]
    one = [tuple(t.clone() for t in s[:3]) + s[3:] for s in sets]
    zero = sets[2][0].clone()
    for rounding in ("rne", "sr"):
        kw = dict(lr=0.02, step=9, seed=1, rounding=rounding)
        asr.asr_muon_sr_multi_tensor(sets, **kw)
        for p, g, m, base in one:
            for z in range(p.shape[0] if p.dim() == 3 else 1):
                v = (p[z], g[z], m[z], base + z * 960) if p.dim() == 3 else (p, g, m, base)
                asr.asr_muon_sr_multi_tensor([v], **kw)
        for a, b in zip(sets, one):
            assert_same_bits(host(a[0]), host(b[0]))
            assert_same_bits(host(a[2]), host(b[2]))
        if rounding == "rne":
            want = (zero.float() * np.float32(1 - 0.02 * 0.1)).bfloat16()
            assert_same_bits(host(sets[2][0]), host(want))


def test_streams_graph_and_workspace(asr):
    import torch
    torch.manual_seed(8)
    g = torch.randn(3, 130, 200, device="cuda")
    want = torch.empty(3, 130, 200, device="cuda", dtype=torch.bfloat16)
    out = torch.zeros_like(want)
    asr.asr_newton_schulz([(g, want)])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    asr.asr_newton_schulz([(g, out)], stream=s)
    s.synchronize()
    assert_same_bits(host(out), host(want))
    ws = torch.empty(asr.asr_newton_schulz_workspace([(g, out)]), dtype=torch.uint8, device="cuda")
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        asr.asr_newton_schulz([(g, out)], workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert_same_bits(host(out), host(want))
    with pytest.raises(ValueError):
        asr.asr_newton_schulz([(g, out)], workspace=ws[:-256])


def test_muon_step_captured_into_a_graph(asr):
    import torch
    torch.manual_seed(3)
    sets = [(torch.randn(s, device="cuda").bfloat16(), torch.randn(s, device="cuda"), torch.zeros(s, device="cuda"), 4)
            for s in ((2, 90, 300), (200, 260), (260, 200))]
    again = [tuple(t.clone() for t in s[:3]) + s[3:] for s in sets]
    kw = dict(lr=0.02, step=9, seed=1)
    asr.asr_muon_sr_multi_tensor([tuple(t.clone() for t in s[:3]) + s[3:] for s in sets], **kw)
    ws = torch.empty(asr.asr_muon_workspace(sets), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        asr.asr_muon_sr_multi_tensor(sets, workspace=ws, **kw)
    for _ in range(2):
        graph.replay()
        asr.asr_muon_sr_multi_tensor(again, **kw)
    torch.cuda.synchronize()
    for a, b in zip(sets, again):
        assert_same_bits(host(a[0]), host(b[0]))
        assert_same_bits(host(a[2]), host(b[2]))


def test_refusals(asr):
    import torch
    g = torch.randn(8, 16, device="cuda")
    o = torch.empty(8, 16, device="cuda", dtype=torch.bfloat16)
    for bad in (dict(steps=0), dict(steps=101)):
        with pytest.raises(ValueError):
            asr.asr_newton_schulz([(g, o)], **bad)
    for bad in (dict(coefficients=(20.0, 0.0, 0.0)), dict(coefficients=(float("nan"), 0, 0)), dict(eps=-1.0),
                dict(coefficients=(3.0, 3.0, 3.0)), dict(eps=0.0)):
        with pytest.raises(asr.AsrError):
            asr.asr_newton_schulz([(g, o)], **bad)
    with pytest.raises(ValueError):
        asr.asr_newton_schulz([(g, o[:, :8])])
    with pytest.raises(ValueError):
        asr.asr_newton_schulz([(g.t(), o.t())])
    with pytest.raises(TypeError):
        asr.asr_newton_schulz([(g, g)])
    with pytest.raises(ValueError):
        asr.asr_newton_schulz([(g[0], o[0])])
    with pytest.raises(ValueError):
        asr.asr_newton_schulz([(g.cpu(), o)])
    p = torch.zeros(8, 16, device="cuda")
    kw = dict(lr=0.1, step=1)
    with pytest.raises(ValueError):
        asr.asr_muon_sr_multi_tensor([(p, g, g[:4], 0)], **kw)
    with pytest.raises(ValueError):
        asr.asr_muon_sr_multi_tensor([(p, g, p.clone(), 0)], lr=0.1, step=1, adjust="other")
    for bad in (dict(lr=-1.0, step=1), dict(lr=0.1, step=0), dict(lr=0.1, step=1, momentum=1.0)):
        with pytest.raises(asr.AsrError):
            asr.asr_muon_sr_multi_tensor([(p, g, p.clone(), 0)], **bad)
    asr.asr_newton_schulz([])
    asr.asr_newton_schulz([(g[:0], o[:0])])
    asr.asr_muon_sr_multi_tensor([], lr=0.1, step=1)
