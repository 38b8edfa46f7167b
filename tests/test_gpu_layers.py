"""The operators between a layer's 8-bit products against 64 bits: 8-bit checkpoints, the
activation, the norm, the embedding, forward and backward.

Tolerances count roundings.  u = 2^-24 is half a step of binary32 relative to the value, and a
result is rounded once more to its type (finfo.eps / 2).  A checkpoint is exact."""
import math

import pytest

import layer_reference as ref
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def asr():
    torch_cuda()
    from stochastic_rounding_gb300 import build
    build.build()
    import stochastic_rounding_gb300 as m
    yield m
    assert m.asr_take_device_error() == 0


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def make(rows, cols, dtype, seed, size=1.0):
    """Values of several sizes and signs, a few strong, some zero."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * size
    x *= torch.exp(1.5 * torch.randn(rows, 1, generator=g))
    x *= 1.0 + 20.0 * (torch.rand(rows, cols, generator=g) < 0.01)
    x *= torch.rand(rows, cols, generator=g) > 0.02
    return x.to(dtype_of(dtype)).cuda()


def placed(x, how):
    """x in other memory: rows with a gap between them, or beginning off alignment."""
    import torch
    rows, cols = x.shape
    if how == "plain":
        return x
    off, ld = {"pitched": (0, cols + 24), "odd": (1, cols + 5), "off": (3, cols)}[how]
    buf = torch.full((off + rows * ld + 64,), 7.0, dtype=x.dtype, device=x.device)
    v = buf[off:off + rows * ld].view(rows, ld)[:, :cols] if rows else x
    return v.copy_(x) if rows else x


def close(got, want, bound, what=""):
    """Every element within `bound` of 64 bits and its own rounding; what is not finite is equal."""
    import torch
    got64, want = got.double(), want.to(got.device)
    bound = bound.to(got.device) if torch.is_tensor(bound) else bound
    both = torch.isfinite(want)
    assert torch.equal(torch.isnan(got64), torch.isnan(want)), what
    assert torch.equal(got64[~both & ~torch.isnan(want)], want[~both & ~torch.isnan(want)]), what
    # the type's rounding, relative to the value, and the smallest number's (f32's, bf16 having the same exponents)
    limit = bound + (want.abs() + bound) * (torch.finfo(got.dtype).eps / 2) + 2.0 ** -133
    worse = ((got64 - want).abs() > limit) & both
    assert not worse.any(), f"{what}: {int(worse.sum())} of {worse.numel()}, worst " \
        f"{float(((got64 - want).abs() / limit)[both].max())} of the bound"


# -------------------------------------------------------------- checkpoints

SHAPES = [(1, 1), (1, 31), (3, 32), (2, 33), (5, 64), (7, 515), (4, 1000), (3, 2049), (33, 4096), (130, 96)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rounding", ["rne", "sr"])
def test_checkpoint(asr, orc, rows, cols, dtype, rounding):
    """Codes, powers and values, all exact, from memory of every alignment."""
    import torch
    x = make(rows, cols, dtype, rows * 10000 + cols)
    bits = ref.words16(rows, cols, 5, 77, orc) if rounding == "sr" else None
    q, power, value = ref.checkpoint(x, bits)
    for how in ("plain", "pitched", "odd", "off"):
        c = asr.checkpoint_int8(placed(x, how), rounding=rounding, step=5, seed=77)
        assert torch.equal(c.power.cpu().long(), power), how
        assert torch.equal(c.q.cpu().double(), q), how
        for out in (torch.bfloat16, torch.float32):
            got = asr.restore_int8(c, out)
            assert torch.equal(got.double().cpu(), value), (how, out)
            other = placed(torch.zeros_like(got), how)
            asr.asr_restore_int8(c.q, c.power, other)
            assert torch.equal(other, got)


def test_checkpoint_writes_no_byte_of_its_neighbours(asr):
    import torch
    rows, cols = 5, 71
    x = make(rows, cols, "bf16", 3)
    for q_off, q_ld, p_ld in ((0, 80, 4), (1, 72, 3), (3, 71, 3)):
        q = torch.full((q_off + rows * q_ld + 32,), 99, dtype=torch.int8, device="cuda")
        p = torch.full((1 + rows * p_ld + 32,), 98, dtype=torch.uint8, device="cuda")
        qv, pv = (t[o:o + rows * ld].view(rows, ld)[:, :n] for t, o, ld, n in ((q, q_off, q_ld, cols), (p, 1, p_ld, 3)))
        qv.fill_(1), pv.fill_(1)
        asr.asr_checkpoint_int8(x, qv, pv)
        want = asr.checkpoint_int8(x)
        assert torch.equal(qv, want.q) and torch.equal(pv, want.power)
        qv.fill_(99), pv.fill_(98)
        assert (q == 99).all() and (p == 98).all()
        # and the values, between rows of others
        out = torch.full((rows, cols + 3), 7.0, dtype=torch.float32, device="cuda")
        asr.asr_restore_int8(want.q, want.power, out[:, 1:cols + 1])
        assert (out[:, 0] == 7).all() and (out[:, cols + 1:] == 7).all()


@pytest.mark.parametrize("rounding", ["rne", "sr"])
def test_checkpoint_of_edges(asr, orc, rounding):
    """Each power's borders, zeros, the smallest and largest numbers, infinities and NaN."""
    import torch
    f32 = torch.finfo(torch.float32)
    tops = [0.0, f32.tiny, 2.0 ** -149, 2.0 ** -130, 2.0 ** -121, 127 * 2.0 ** -127, f32.max, -f32.max, 127.0, 127.5,
            math.nextafter(127.0, 200), 254.0, 255.0, 1e-30, 3.4e38, math.inf, -math.inf, math.nan]
    x = torch.zeros(len(tops), 64)
    x[:, 5] = torch.tensor(tops)
    x[:, 6] = torch.tensor(tops) * 0.37
    x[:, 7] = -torch.tensor(tops) * 0.0039370079
    x[:, 40] = torch.linspace(-1, 1, len(tops))
    bits = ref.words16(len(tops), 64, 9, 2, orc) if rounding == "sr" else None
    q, power, value = ref.checkpoint(x, bits)
    c = asr.checkpoint_int8(x.cuda(), rounding=rounding, step=9, seed=2)
    assert torch.equal(c.power.cpu().long(), power)
    assert torch.equal(c.q.cpu().double(), q)
    got = asr.restore_int8(c).cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(value))
    # next to f32's largest number a value may be nearest to 64 * 2^122 = 2^128, which reads back as infinity
    assert torch.equal(got.nan_to_num(), value.float().double().nan_to_num())


def test_checkpoint_rounds_without_bias(asr):
    """Over 65,536 seeds' worth of bits a stochastic code is the value on average: within five standard deviations of a
    fair draw."""
    import torch
    n = 4096
    x = torch.full((n, 32), 0.3, device="cuda")
    x[:, 0] = 127.0                                # 2^0 a step
    x[:, 1:] += torch.arange(31, device="cuda") / 31
    frac = x[0] - x[0].floor()
    mean = asr.restore_int8(asr.checkpoint_int8(x, rounding="sr", step=1, seed=4)).double().mean(0) - x[0].floor()
    assert ((mean - frac).abs() <= 5 * (frac * (1 - frac) / n).sqrt() + 2.0 ** -16).all()
    assert float(mean[0]) == 0.0


def test_checkpoint_of_shards(asr):
    """Rows made apart, from their own place on, are those of the whole."""
    import torch
    x = make(64, 70, "bf16", 8)
    whole = asr.checkpoint_int8(x, rounding="sr", step=2, seed=1)
    part = asr.checkpoint_int8(x[40:], rounding="sr", step=2, seed=1, base_index=40 * 96)
    assert torch.equal(whole.q[40:], part.q) and torch.equal(whole.power[40:], part.power)
    assert not torch.equal(whole.q, asr.checkpoint_int8(x, rounding="sr", step=3, seed=1).q)


# --------------------------------------------------------------- activation

def slack(x, n, function):
    """Roundings of f and f' in binary32, relative: twenty of their own, the exponential's argument's, relative to u and
    so absolute in it, and the hardware exponential's (2 + 1.16 |u| steps)."""
    u = ref.argument(x[:, :n].double(), function).abs()
    return U * (20 + 10 * u.clamp(max=2.0 ** 20))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (2, 33), (3, 64), (5, 515), (4, 1024), (2, 4097), (40, 224)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("function", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
def test_activation(asr, rows, cols, dtype, function, gated):
    """Forward; backward at the input and at its checkpoint, both roundings; every alignment."""
    import torch
    x = make(rows, cols * (2 if gated else 1), dtype, cols * 7 + rows)
    dy = make(rows, cols, dtype, cols + 1, 1e-3)
    k = slack(x, cols, function)
    y64 = ref.activation(x, function, gated)
    b = x[:, cols:].double().abs() if gated else 1.0
    a = x[:, :cols].double().abs()
    for how in ("plain", "pitched", "odd", "off"):
        y, saved = asr.activation(placed(x, how), function, gated=gated, save="input")
        floor = 2.0 ** -124 * (1 + a) * b               # where e^-|u| is no normal number
        close(y, y64, k * y64.abs() + floor, f"y {how}")
        assert torch.equal(asr.activation(x, function, gated=gated), y)
        for rounding in ("rne", "sr"):
            y8, kept = asr.activation(placed(x, how), function, gated=gated, save="int8", rounding=rounding, step=3, seed=9)
            alone = asr.checkpoint_int8(x, rounding=rounding, step=3, seed=9)
            assert torch.equal(y8, y)
            assert torch.equal(kept.q, alone.q) and torch.equal(kept.power, alone.power)
            for s, at in ((saved, x), (kept, asr.restore_int8(kept, torch.float32))):
                dx = asr.activation_grads(placed(dy, how), s, function, gated=gated)
                want = ref.activation_grads(dy, at, function, gated)
                av, bv = at[:, :cols].double(), at[:, cols:].double().abs() if gated else 1.0
                ks = slack(at, cols, function)
                # f' = s (1 + r t): each term's roundings, t's floor times r
                u = ref.argument(av, function)
                sg = torch.sigmoid(u)
                r = (av * (1 + (3 * 0.044715 * av * av if function == "gelu" else 0))).abs() * 1.6
                g = dy.double().abs()
                da = (ks * sg * (1 + r * (1 - sg)) + 2.0 ** -124 * (1 + r)) * g * bv
                if gated:
                    db = (ks * ref.value(av, function).abs() + 2.0 ** -124 * (1 + av.abs())) * g
                    da = torch.cat((da, db), 1)
                close(dx, want, da, f"dx {how} {rounding}")
                other = placed(torch.zeros_like(dx), how)
                x0 = None if s is kept else s
                asr.asr_activation_grads(dy, x0, other, function, gated=gated, kept=kept if x0 is None else None)
                assert torch.equal(other, dx)


@pytest.mark.parametrize("function", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_activation_of_edges(asr, function, dtype):
    """Large values on both sides, where the exponential leaves its range, and NaN."""
    import torch
    x = torch.tensor([[0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 86.0, -86.0, 100.0, -100.0, 1e4, -1e4, 1e12, -1e12, math.nan,
                       math.inf]]).to(dtype_of(dtype)).cuda()
    y = asr.activation(x, function).double()
    dx = asr.activation_grads(torch.ones_like(x), x, function).double()
    a = x.double()
    assert torch.isnan(y[0, 14]) and torch.isnan(dx[0, 14]) and y[0, 15] == math.inf and dx[0, 15] == 1.0
    fine = slice(0, 14)
    want, slopes = ref.value(a, function)[:, fine], ref.slope(a, function)[:, fine]
    k = slack(x, 16, function)[:, fine]
    close(y[:, fine].to(x.dtype), want, k.clamp(max=1.0) * want.abs() + 1e-33)
    close(dx[:, fine].to(x.dtype), slopes, k.clamp(max=1.0) * slopes.abs() + U * 40 + 1e-33)


def test_activation_gradient_against_differences(asr):
    """Central differences of the 64-bit formula: their own error is 1e-10 of a second difference, and f32's roundings are
    those of `slack`."""
    import torch
    torch.manual_seed(1)
    for function in ("silu", "gelu"):
        x = torch.randn(6, 40, device="cuda") * 2
        c = torch.randn(6, 20, device="cuda")
        dx = asr.activation_grads(c, x, function, gated=True)
        h = 1e-5
        for i, j in ((0, 0), (1, 19), (2, 20), (5, 39), (3, 7)):
            e = torch.zeros_like(x, dtype=torch.float64)
            e[i, j] = h
            up, down = (float((ref.activation(x.double() + s * e, function, True) * c.double()).sum()) for s in (1, -1))
            assert abs(float(dx[i, j]) - (up - down) / (2 * h)) <= 1e-5


# --------------------------------------------------------------------- norm

# a warp's rows, a block's of each size, and those that fit neither
NORM_SHAPES = [(1, 1), (3, 7), (9, 32), (17, 512), (5, 513), (20, 1365), (3, 4096), (4, 4104), (2, 8200), (3, 16384),
               (2, 16390), (3, 40001), (1300, 72), (700, 1032)]
K_SUM = 64          # additions along any path of a row's sum: 16 in a thread (40 where rows do not fit), 5 and 5 across, and
#                     the roundings around them


def norm_bounds(x, w, b, mean, rstd, h):
    """What f32 roundings do to h (before a type's own): the mean's error, sums of |x|, times rstd; and rstd's, relative."""
    dh = K_SUM * U * (rstd * x.double().abs().mean(1, keepdim=True) + h.abs())
    y = (dh + 2 * U * h.abs()) * (1.0 if w is None else w.double().abs()) + (0.0 if b is None else 2 * U * b.double().abs())
    return dh, y


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("centred", [True, False])
def test_norm(asr, rows, cols, dtype, centred):
    import torch
    eps = 1e-5
    x = make(rows, cols, dtype, rows + 3 * cols)
    x = (x.float() + 0.7).to(x.dtype)
    dy = make(rows, cols, dtype, 5 * cols, 1e-3)
    g = torch.Generator().manual_seed(cols)
    other = dtype_of("f32" if (rows + cols) % 2 else "bf16")        # parameters of a type of their own
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(other).cuda()
    b = torch.randn(cols, generator=g).to(other).cuda() if centred else None
    y64, mean, rstd, h = ref.norm(x, w, b, eps, centred)
    dh, dyv = norm_bounds(x, w, b, mean, rstd, h)
    plain = None
    for how in ("plain", "pitched", "odd", "off"):
        y, saved = asr.layer_norm(placed(x, how), w, b, eps=eps, centred=centred, save="input")
        close(y, y64, dyv, f"y {how}")
        close(saved.rstd[:, None], rstd, K_SUM * U * rstd, "rstd")
        if centred:
            close(saved.mean[:, None], mean, K_SUM * U * x.double().abs().mean(1, keepdim=True), "mean")
        else:
            assert saved.mean is None
        assert torch.equal(asr.layer_norm(x, w, b, eps=eps, centred=centred), y)
        rounding = "sr" if how in ("plain", "odd") else "rne"
        y8, saved8 = asr.layer_norm(placed(x, how), w, b, eps=eps, centred=centred, save="int8", rounding=rounding, step=4,
                                    seed=3)
        alone = asr.checkpoint_int8(x, rounding=rounding, step=4, seed=3)
        assert torch.equal(y8, y) and torch.equal(saved8.rstd, saved.rstd)
        assert torch.equal(saved8.input.q, alone.q) and torch.equal(saved8.input.power, alone.power)
        for s, at in ((saved, x), (saved8, asr.restore_int8(saved8.input, torch.float32))):
            dx, dw, db = asr.layer_norm_grads(placed(dy, how), s, w)
            wx, ww, wb = ref.norm_grads(dy, at, w, mean, rstd, centred)
            ha = (at.double() - mean) * rstd
            gg = dy.double() * w.double()
            d = K_SUM * U * (rstd * x.double().abs().mean(1, keepdim=True) + ha.abs())
            along = (gg * ha).abs().mean(1, keepdim=True)
            # each of dx's three terms with the roundings of its sums, h's error in the third twice, rstd's in all
            bound = rstd * (K_SUM * U * (gg.abs() + gg.abs().mean(1, keepdim=True) + 2 * ha.abs() * along) +
                            d * along + ha.abs() * (gg.abs() * d).mean(1, keepdim=True))
            close(dx, wx, bound, f"dx {how}")
            # sums over rows: at most 128 additions along a path (rows a group, groups a warp, warps)
            close(dw, ww, (128 * U * (dy.double() * ha).abs() + dy.double().abs() * d).sum(0), f"dw {how}")
            close(db, wb, 128 * U * dy.double().abs().sum(0), f"db {how}")
            if s is saved and how == "plain":
                plain = (dx, dw, db)
                again = asr.layer_norm_grads(dy, s, w)
                assert all(torch.equal(p, q) for p, q in zip(plain, again))
                only = asr.layer_norm_grads(dy, s, w, need_dx=False, need_dbias=False)
                assert only[0] is None and only[2] is None and torch.equal(only[1], dw)
                only = asr.layer_norm_grads(dy, s, w, need_dweight=False, need_dbias=False)
                assert torch.equal(only[0], dx)


@pytest.mark.parametrize("rows,cols", [(2, 512), (1500, 1024), (3001, 2560), (2100, 4096), (40, 4608)])
def test_norm_gradients_from_codes_without_a_bias(asr, rows, cols):
    """The same gradients whether a bias's is wanted, and however the powers lie; many rows to a block."""
    import torch
    x, dy = make(rows, cols, "bf16", rows), make(rows, cols, "bf16", cols, 1e-3)
    w = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(cols))).to(torch.bfloat16).cuda()
    _, saved = asr.layer_norm(x, w, centred=False, save="int8")
    dx, dw, none = asr.layer_norm_grads(dy, saved, w, need_dbias=False)
    assert none is None
    at, rstd = asr.restore_int8(saved.input, torch.float32), saved.rstd.double()[:, None]
    ha = at.double() * rstd                     # rstd as it is saved: h has a rounding, a product with dy another in its sum
    bound = (128 * U * (dy.double() * ha).abs()).sum(0)
    close(dw, (dy.double() * ha).sum(0), bound, "dw")
    full = asr.layer_norm_grads(dy, saved, w)
    assert torch.equal(full[0], dx)
    close(full[1], (dy.double() * ha).sum(0), bound, "dw with db")
    q, power = saved.input.q, saved.input.power
    groups = cols // 32
    for off, ld in ((0, groups), (1, groups + 4), (4, groups + 1)):
        buf = torch.zeros(off + rows * ld + 8, dtype=torch.uint8, device="cuda")
        p = buf[off:off + rows * ld].view(rows, ld)[:, :groups].copy_(power)
        dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
        asr.asr_layer_norm_grads(dy, None, w, None, saved.rstd, dx2, dw2, None, centred=False, kept=(q, p))
        assert torch.equal(dx2, dx)
        close(dw2, (dy.double() * ha).sum(0), bound, "dw")


@pytest.mark.parametrize("centred", [True, False])
@pytest.mark.parametrize("cols", [40, 1500, 20000])
def test_norm_without_parameters_and_without_rows(asr, centred, cols):
    import torch
    x, dy = make(6, cols, "f32", 1), make(6, cols, "f32", 2)
    ones = torch.ones(cols, device="cuda")
    y, s = asr.layer_norm(x, centred=centred, save="input")
    want, t = asr.layer_norm(x, ones, 0 * ones, centred=centred, save="input")
    assert torch.equal(y, want)
    for p, q in zip(asr.layer_norm_grads(dy, s), asr.layer_norm_grads(dy, t, ones)):
        assert torch.equal(p, q)
    y, s = asr.layer_norm(x[:0], centred=centred, save="input")
    dx, dw, db = asr.layer_norm_grads(dy[:0], s)
    assert y.shape == (0, cols) and dx.shape == (0, cols) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("cols", [64, 2000, 30000])
def test_norm_of_edges(asr, cols):
    """A constant row (no variance but eps's), a large mean (the squares are about it), zeros, infinities, NaN, and the
    neighbours of such rows, which are as they are alone."""
    import torch
    torch.manual_seed(cols)
    x = torch.randn(8, cols, device="cuda")
    x[1] = 3.0
    x[2] += 4096.0
    x[3] = 0.0
    x[4, cols // 2] = math.inf
    x[5, 3] = math.nan
    y, s = asr.layer_norm(x, save="input")
    want, mean, rstd, h = ref.norm(x, None, None, 1e-5, True)
    dh, bound = norm_bounds(x, None, None, mean, rstd, h)
    keep = [0, 1, 2, 3, 6, 7]
    close(y[keep], want[keep], bound[keep])
    assert torch.isnan(y[4]).any() and torch.isnan(y[5]).all()
    dy = torch.randn_like(x)
    dx, _, _ = asr.layer_norm_grads(dy, s)
    for r in keep:
        one, t = asr.layer_norm(x[r:r + 1], save="input")
        assert torch.equal(one, y[r:r + 1])
        assert torch.equal(asr.layer_norm_grads(dy[r:r + 1], t)[0], dx[r:r + 1])
    # in place
    z = x.clone()
    assert asr.asr_layer_norm(z, None, None, z) is z
    assert torch.equal(z[keep], y[keep])


def test_norm_gradient_against_differences(asr):
    import torch
    torch.manual_seed(2)
    for centred in (True, False):
        x, c = torch.randn(3, 50, device="cuda") + 0.5, torch.randn(3, 50, device="cuda")
        w = 1 + 0.2 * torch.randn(50, device="cuda")
        _, s = asr.layer_norm(x, w, None, centred=centred, save="input")
        dx, dw, _ = asr.layer_norm_grads(c, s, w)
        f = lambda a, v: float((ref.norm(a, v, None, 1e-5, centred)[0] * c.double()).sum())  # noqa: E731
        h = 1e-5
        for i, j in ((0, 0), (1, 33), (2, 49)):
            e = torch.zeros_like(x, dtype=torch.float64)
            e[i, j] = h
            assert abs(float(dx[i, j]) - (f(x.double() + e, w) - f(x.double() - e, w)) / (2 * h)) <= 1e-5
            e = torch.zeros_like(w, dtype=torch.float64)
            e[j] = h
            assert abs(float(dw[j]) - (f(x, w.double() + e) - f(x, w.double() - e)) / (2 * h)) <= 1e-5


# ---------------------------------------------------------------- embedding

@pytest.mark.parametrize("tokens,vocab,dim", [(0, 5, 8), (1, 1, 1), (1, 300, 64), (5, 3, 33), (33, 1000, 515), (700, 64, 2050),
                                              (64, 50, 4096)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("index", ["int64", "int32"])
def test_embedding(asr, tokens, vocab, dim, dtype, index):
    import torch
    table = make(vocab, dim, dtype, dim)
    g = torch.Generator().manual_seed(tokens)
    ids = torch.randint(0, vocab, (tokens,), generator=g).to(getattr(torch, index)).cuda()
    for how in ("plain", "pitched", "odd"):
        t = placed(table, how)
        assert torch.equal(asr.embedding(ids, t), table[ids.long()])
        scaled = asr.embedding(ids, t, scale=1.7)
        close(scaled, table[ids.long()].double() * 1.7, 3 * U * 1.7 * table[ids.long()].double().abs())
        other = placed(torch.zeros_like(scaled), how)
        assert torch.equal(asr.asr_embedding(ids, t, other, scale=1.7), scaled)


@pytest.mark.parametrize("index", ["int64", "int32"])
def test_ids_outside_the_table(asr, index):
    """No row: NaN forward, nothing in the gradient, whatever the number."""
    import torch
    vocab, dim = 40, 24
    table = make(vocab, dim, "f32", 1)
    bad = [-1, vocab, vocab + 1, -100, 2 ** 31 - 1, -2 ** 31]
    if index == "int64":
        bad += [2 ** 32, 2 ** 32 + 3, -2 ** 63, 2 ** 63 - 1, -2 ** 32 + 5]
    ids = torch.tensor([3, *bad, 39, 0, 3], dtype=getattr(torch, index), device="cuda")
    y = asr.embedding(ids, table)
    ok = (ids >= 0) & (ids < vocab)
    assert torch.isnan(y[~ok]).all() and torch.equal(y[ok], table[ids[ok].long()])
    dy = make(len(ids), dim, "f32", 2)
    want = ref.embedding_grads(ids, dy, vocab, 1.0)
    close(asr.embedding_grads(ids, dy, vocab), want, 4 * U * want.abs() + 1e-6)
    assert (asr.embedding_grads(ids[1:-3], dy[1:-3], vocab) == 0).all()


def ids_of(kind, tokens, vocab, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    if kind == "same":
        return torch.full((tokens,), vocab // 2)
    if kind == "uniform":
        return torch.randint(0, vocab, (tokens,), generator=g)
    if kind == "few":
        return torch.randint(0, min(3, vocab), (tokens,), generator=g) * (vocab // 3)
    if kind == "ordered":
        return torch.arange(tokens) % vocab
    u = torch.rand(tokens, generator=g, dtype=torch.float64)
    return (torch.exp(u * math.log(vocab)).long() - 1).clamp(0, vocab - 1)


GRADS = [(1, 1, 1), (1, 700, 33), (7, 3, 8), (8, 8, 64), (9, 100, 515), (64, 1001, 40), (300, 17, 2056), (1000, 513, 128),
         (8191, 600, 16), (8192, 70000, 8), (8193, 600, 24), (20000, 130000, 12), (40003, 512, 9), (33000, 5, 40)]


@pytest.mark.parametrize("tokens,vocab,dim", GRADS)
@pytest.mark.parametrize("kind", ["same", "uniform", "few", "ordered", "frequent"])
def test_embedding_grads(asr, tokens, vocab, dim, kind):
    """Every row against its sum in 64 bits, rows without tokens exactly zero, what was there before gone, the same bits
    again, and padding left out."""
    import torch
    for n, (dt, ot, index, scale, padding) in enumerate((("bf16", "bf16", "int64", 1.0, False), ("f32", "f32", "int32", 0.5, True),
                                                         ("bf16", "f32", "int32", 3.0, False), ("f32", "bf16", "int64", 1.0, True))):
        ids = ids_of(kind, tokens, vocab, tokens + n).to(getattr(torch, index)).cuda()
        dy = make(tokens, dim, dt, dim + n)
        pad = int(ids[tokens // 2]) if padding else None
        out = torch.full((vocab, dim), math.nan, dtype=dtype_of(ot), device="cuda")
        how = ("plain", "pitched", "odd", "off")[n]
        asr.asr_embedding_grads(ids, placed(dy, how), out, scale=scale, padding_idx=pad)
        want = ref.embedding_grads(ids, dy, vocab, scale, pad)
        size = ref.embedding_grads(ids, dy.abs(), vocab, scale, pad)
        # additions along a path: a chunk's tokens, then its row's chunks; never more than the row's tokens
        live = ids.long()
        count = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add_(0, live, torch.ones(tokens, dtype=torch.float64, device="cuda"))
        bound = U * (count[:, None] + 2) * size
        close(out, want, bound, f"{kind} {n}")
        assert (out[count == 0] == 0).all()
        if pad is not None:
            assert (out[pad] == 0).all()
        again = torch.empty_like(out)
        asr.asr_embedding_grads(ids, dy, again, scale=scale, padding_idx=pad)
        assert torch.equal(again, out)


def test_embedding_grads_into_unaligned_memory(asr):
    """A table that does not begin on 16 bytes; nothing before or behind it is touched."""
    import torch
    for dt, off in (("bf16", 1), ("f32", 1), ("bf16", 8)):
        vocab, dim, tokens = 130, 72, 50
        buf = torch.full((off + vocab * dim + 40,), 5.0, dtype=dtype_of(dt), device="cuda")
        out = buf[off:off + vocab * dim].view(vocab, dim)
        ids, dy = ids_of("frequent", tokens, vocab, 1).cuda(), make(tokens, dim, dt, 4)
        asr.asr_embedding_grads(ids, dy, out)
        assert torch.equal(out, asr.embedding_grads(ids, dy, vocab))
        assert (buf[:off] == 5).all() and (buf[off + vocab * dim:] == 5).all()


def test_empty_calls(asr):
    import torch
    e = torch.empty(0, 8, device="cuda")
    assert asr.checkpoint_int8(e).q.shape == (0, 8) and asr.restore_int8(asr.checkpoint_int8(e)).shape == (0, 8)
    assert asr.activation(e).shape == (0, 8) and asr.activation_grads(e, e).shape == (0, 8)
    none = torch.empty(4, 0, device="cuda")
    assert asr.layer_norm(none).shape == (4, 0) and asr.activation(none, gated=True).shape == (4, 0)
    assert (asr.embedding_grads(torch.empty(0, dtype=torch.int64, device="cuda"), e, 9) == 0).all()
    assert asr.embedding_grads(torch.empty(0, dtype=torch.int64, device="cuda"), e, 0).shape == (0, 8)
