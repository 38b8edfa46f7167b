"""Newton-Schulz and the Muon step past the sizes and values of the ordinary
tests: gradients whose squares binary32 loses, and products of more tiles than
the GPU takes at once.  The bound is derived in test_gpu_muon.py."""
import pytest

from gpu_util import torch_cuda

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


def _exact(g, eps=1e-7):
    x = g.double()
    x = x / max(float(x.norm()), eps)
    if x.shape[0] > x.shape[1]:
        x = x.t()
    a, b, c = ABC
    for _ in range(5):
        s = x @ x.t()
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.t() if g.shape[0] > g.shape[1] else x


BOUND = 3 * 5 * 2.0 ** -11 + 2.0 ** -9


def _far(got, want):
    return float((got.double() - want).norm() / want.norm())


# one CTA a matrix, clusters, products in memory; wide and tall
@pytest.mark.parametrize("shape", [(96, 160), (700, 128), (100, 4000), (256, 256), (515, 300)])
@pytest.mark.parametrize("size", [1e-12, 1e-18, 1e-20, 1e-23, 3e-26, 1e-29])
def test_gradients_whose_squares_underflow(asr, shape, size):
    import torch
    torch.manual_seed(7)
    g = torch.randn(shape, device="cuda") * size
    out = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    asr.asr_newton_schulz([(g, out)], eps=1e-30)
    assert _far(out, _exact(g, 1e-30)) <= BOUND
    p, m = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
    asr.asr_muon_sr_multi_tensor([(p, g, m, 0)], lr=1.0, momentum=0.5, weight_decay=0.0, nesterov=False, adjust=None,
                                 step=1, eps=1e-30)
    assert _far(-p, _exact(m, 1e-30)) <= BOUND


@pytest.mark.parametrize("shape", [(96, 160), (256, 256)])
def test_gradients_below_eps(asr, shape):
    """A norm below eps: G / eps, not G / |G|."""
    import torch
    torch.manual_seed(8)
    g = torch.randn(shape, device="cuda")
    g *= 0.25e-20 / float(g.norm())
    out = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    asr.asr_newton_schulz([(g, out)], eps=1e-20)
    assert _far(out, _exact(g, 1e-20)) <= BOUND


@pytest.mark.parametrize("shape", [(96, 160), (256, 256)])
def test_small_entries_beside_large_ones(asr, shape):
    """Squares that underflow next to ones that do not, on both sides of where
    the sums change over (a sum of squares of 2^-60)."""
    import torch
    torch.manual_seed(9)
    for top in (1e-8, 2.0 ** -30, 1e-10):
        g = torch.randn(shape, device="cuda") * 1e-22
        g[::7] = torch.randn_like(g[::7]) * (top / 16)
        out = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
        asr.asr_newton_schulz([(g, out)], eps=1e-30)
        got, want = out[::7], _exact(g, 1e-30)[::7]
        assert _far(got, want) <= BOUND


@pytest.mark.parametrize("shape", [(60, 96), (1, 96), (96, 1), (200, 150)])
def test_stacks_whose_rows_alternate(asr, shape):
    """A stack along the middle of a tensor (the heads of a projection), as input
    and as output: what each matrix gives on its own."""
    import torch
    torch.manual_seed(10)
    rows, cols = shape
    g = torch.randn(rows, 5, cols, device="cuda").bfloat16().transpose(0, 1)
    buf = torch.full((rows, 7, cols), 9.0, device="cuda", dtype=torch.bfloat16)
    out = buf[:, 1:6].transpose(0, 1)
    asr.asr_newton_schulz([(g, out)])
    for z in range(5):
        alone = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
        asr.asr_newton_schulz([(g[z].contiguous(), alone)])
        assert torch.equal(out[z], alone)
    assert (buf[:, 0] == 9).all() and (buf[:, 6] == 9).all()


def test_overlapping_outputs_are_refused(asr):
    import torch
    g = torch.randn(3, 4, 8, device="cuda")
    buf = torch.empty(200, device="cuda", dtype=torch.bfloat16)
    for strides in ((31, 8, 1), (0, 8, 1), (7, 24, 1), (8, 23, 1), (8, 8, 1)):
        with pytest.raises(ValueError, match="overlap"):
            asr.asr_newton_schulz([(g, buf.as_strided((3, 4, 8), strides))])
    for strides in ((32, 8, 1), (8, 24, 1), (40, 9, 1), (9, 30, 1)):
        asr.asr_newton_schulz([(g, buf.as_strided((3, 4, 8), strides))])


# Stacks whose products take more tiles (of 256 x 256, on 76 pairs of SMs) than half the
# pairs, and several rounds of them.  Of S and P, and of X', whole rounds and what is
# left: 1 + 24 and 2 + 48; 0 + 54 and 2 + 10; 0 + 48 and 1 + 20; 0 + 45 and 1 + 23.
STACKS = [(10, 1024, 1100), (10, 1100, 1024), (9, 600, 1300), (9, 1300, 600), (16, 500, 700), (16, 700, 500),
          (1, 2300, 2600), (1, 2600, 2300)]


@pytest.mark.parametrize("shape", STACKS)
def test_products_of_several_rounds_of_tiles(asr, shape):
    import torch
    torch.manual_seed(shape[1])
    g = (torch.randn(shape, device="cuda") * 1e-3).bfloat16()
    want = [_exact(v) for v in g]
    out = torch.full(shape, 9.0, device="cuda", dtype=torch.bfloat16)
    asr.asr_newton_schulz([(g, out)])
    for got, w in zip(out, want):
        assert _far(got, w) <= BOUND
    # the same rounded from parameters of zero: f32, and bf16 by its random bits
    kw = dict(lr=1.0, momentum=0.5, weight_decay=0.0, nesterov=False, adjust=None, step=3, seed=5)
    p, m = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
    asr.asr_muon_sr_multi_tensor([(p, g, m, 8)], **kw)
    for got, w in zip(p, want):
        assert _far(-got, w) <= BOUND
    pb, m = torch.zeros(shape, device="cuda", dtype=torch.bfloat16), torch.zeros(shape, device="cuda")
    asr.asr_muon_sr_multi_tensor([(pb, g, m, 8)], **kw)
    rounded = torch.empty_like(pb)
    asr.asr_stochastic_round_bf16(p, rounded, base_index=8, step=3, seed=5)
    assert torch.equal(pb, rounded)


@pytest.mark.parametrize("shape", [(5, 700, 1001), (5, 1001, 700)])
def test_parameters_off_every_alignment(asr, shape):
    """Rows of odd length, bf16 parameters and gradients that start at odd
    elements, with decay and momentum from before."""
    import torch
    torch.manual_seed(11)
    size = shape[0] * shape[1] * shape[2]
    base = torch.randn(size, device="cuda") * 0.02
    g = torch.randn(size + 3, device="cuda").bfloat16()[3:].view(shape)
    m = torch.randn(size + 1, device="cuda")[1:].view(shape)
    kw = dict(lr=0.1, momentum=0.9, weight_decay=0.3, adjust="match_rms_adamw", step=2, seed=9)
    pb = torch.empty(size + 1, device="cuda", dtype=torch.bfloat16)[1:].view(shape)
    pb.copy_(base.view(shape))
    pf, m2 = pb.float(), m.clone()
    before = pf.double()
    asr.asr_muon_sr_multi_tensor([(pb, g, m, 7)], **kw)
    asr.asr_muon_sr_multi_tensor([(pf, g, m2, 7)], **kw)
    assert torch.equal(m, m2)
    rounded = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    asr.asr_stochastic_round_bf16(pf, rounded, base_index=7, step=2, seed=9)
    assert torch.equal(pb, rounded)
    u = g.float() + 0.9 * (m2 - g.float())
    for z in range(shape[0]):
        step = 0.1 * 0.2 * max(shape[1:]) ** 0.5 * _exact(u[z])
        err = pf[z].double() - (before[z] * (1 - 0.1 * 0.3) - step)
        assert float(err.norm()) <= BOUND * float(step.norm()) + 3 * 2.0 ** -24 * float(before[z].norm())


@pytest.mark.parametrize("small", [1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("shape", [(96, 160), (256, 256), (512, 2048), (300, 200)])
def test_small_directions_beside_eight_large_ones(asr, shape, small):
    """Rounding X_0 and X' to f16 puts errors of entries' size 2^-11 / sqrt(12)
    at most into every direction, as a random matrix whose largest singular
    value is that times (sqrt m + sqrt n) / sqrt(m n), and the iteration raises
    the small directions, true or not, by at most a^5 = 485: four such sizes and the
    bf16 rounding of the result, as in the test of a matrix of rank 3.  The small
    directions, raised to 485 times their share, are there to the same bound each."""
    import torch
    torch.manual_seed(12)
    m, n = shape
    r = min(shape)
    u = torch.linalg.qr(torch.randn(m, r, device="cuda", dtype=torch.float64))[0]
    v = torch.linalg.qr(torch.randn(n, r, device="cuda", dtype=torch.float64))[0]
    s = torch.full((r,), small, device="cuda", dtype=torch.float64)
    s[:8] = 1.0
    g = ((u * s) @ v.t()).float()
    out = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    asr.asr_newton_schulz([(g, out)])
    want = _exact(g)
    bound = 4 * 485 * 2.0 ** -11 / 12 ** 0.5 * (m ** 0.5 + n ** 0.5) / (m * n) ** 0.5 + 2.0 ** -8
    assert float(torch.linalg.matrix_norm(out.double() - want, 2)) <= bound
    got, there = ((u.t() @ o @ v).diagonal()[8:] for o in (out.double(), want))
    assert float((got - there).abs().max()) <= bound


@pytest.mark.parametrize("shape", [(1, 137, 7674), (2, 128, 4000), (4, 16, 300), (1, 196, 9939), (3, 2107, 8),
                                   (2, 300, 16), (1, 7674, 137), (2, 30, 6000), (1, 96, 160), (2, 512, 2048)])
def test_as_near_as_independent_roundings_leave_it(asr, shape):
    """Gradients of noise and eight directions at two thirds of the norm.  A
    rounding to f16 is off by at most 2^-11 of an entry, evenly spread: 2^-11 /
    sqrt(3) of it in the mean square; sqrt(3) times that of what the eight
    directions leave.  Fifteen of them (X, S and P of five steps), if they are
    independent, leave sqrt(15) 2^-11; what is the same for a whole diagonal would
    add up faster and is kept out.  The result's own rounding is that of the exact one."""
    import torch
    torch.manual_seed(13)
    count, rows, cols = shape
    rank = min(8, rows, cols)
    g = torch.randn(shape, device="cuda")
    g += 0.5 * torch.randn(count, rows, rank, device="cuda") @ torch.randn(count, rank, cols, device="cuda")
    g *= 1e-3
    out = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    asr.asr_newton_schulz([(g, out)])
    p, m = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
    asr.asr_muon_sr_multi_tensor([(p, g, m, 0)], lr=1.0, momentum=0.5, weight_decay=0.0, nesterov=False, adjust=None,
                                 step=1)
    want = torch.stack([_exact(v) for v in g])
    own = _far(want.bfloat16(), want)
    assert _far(-p, want) <= 15 ** 0.5 * 2.0 ** -11
    assert _far(out, want) <= (own ** 2 + 15 * 2.0 ** -22) ** 0.5
