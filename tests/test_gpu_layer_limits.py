"""The norm, the activation, 8-bit checkpoints and the embedding at the ends of what they take, and where every result
is exact: sums of whole numbers, activations far from zero."""
import pytest

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asr():
    torch_cuda()
    from stochastic_rounding_gb300 import build
    build.build()
    import stochastic_rounding_gb300 as m
    yield m
    assert m.asr_take_device_error() == 0


@pytest.mark.parametrize("cols", [2 ** 23 + 32, 2 ** 23 + 17, 2 ** 24])
@pytest.mark.parametrize("rounding", ["rne", "sr"])
def test_a_gated_input_of_any_width_is_kept(asr, cols, rounding):
    """Both halves together are wider than either: 2^25 columns where the output has 2^24.  Codes are those of the
    input's parts, which end with whole groups, and a backward pass from them is that from the values they stand for."""
    import torch
    g = torch.Generator("cuda").manual_seed(cols)
    x = torch.randn(1, 2 * cols, device="cuda", generator=g).to(torch.bfloat16)
    dy = torch.randn(1, cols, device="cuda", generator=g).to(torch.bfloat16)
    y, kept = asr.activation(x, gated=True, save="int8", rounding=rounding, step=3, seed=5)
    assert torch.equal(y, asr.activation(x, gated=True))
    n = 2 ** 23
    for at in range(0, 2 * cols, n):
        part = asr.checkpoint_int8(x[:, at:at + n], rounding=rounding, base_index=at, step=3, seed=5)
        assert torch.equal(kept.q[:, at:at + n], part.q)
        assert torch.equal(kept.power[:, at // 32:(at + n) // 32], part.power)
    back = asr.restore_int8(kept)
    assert torch.equal(asr.activation_grads(dy, kept, gated=True), asr.activation_grads(dy, back, gated=True))


# ------------------------------------------- sums of whole numbers, which binary32 holds

def whole(shape, most, seed, dtype):
    """Whole numbers from -most to most, every one of them likely."""
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, shape, device="cuda", generator=g).to(dtype)


def tokens_of(kind, tokens, vocab, seed):
    """``runs``: one id for a stretch of 1 to 300 tokens, in the ids' order, so that sorting leaves them in place and rows
    begin and end at any place of a chunk; the others as their names say."""
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    if kind == "same":
        return torch.full((tokens,), vocab // 2, device="cuda")
    if kind == "few":
        return torch.randint(0, min(3, vocab), (tokens,), device="cuda", generator=g) * (vocab // 3)
    if kind == "runs":
        length = torch.randint(1, 301, (tokens,), device="cuda", generator=g)
        return torch.repeat_interleave(torch.arange(tokens, device="cuda"), length)[:tokens] % vocab
    u = torch.rand(tokens, device="cuda", generator=g, dtype=torch.float64)             # frequent
    return (torch.exp(u * torch.log(torch.tensor(float(vocab)))).long() - 1).clamp(0, vocab - 1)


@pytest.mark.parametrize("tokens,vocab,dim", [(700, 90, 33), (8193, 600, 24), (16384, 5000, 8), (16385, 1, 8), (20001, 1, 3),
                                              (20000, 130000, 12), (33000, 5, 40), (40003, 512, 9), (524288, 4000, 16),
                                              (524289, 4000, 7), (600011, 1, 5), (1200000, 9000, 16), (1200001, 40000, 3)])
@pytest.mark.parametrize("kind", ["same", "few", "runs", "frequent"])
def test_embedding_gradients_lose_no_token(asr, tokens, vocab, dim, kind):
    """Up to 1.2 million tokens of at most 4 each: no sum leaves the whole numbers that binary32 holds (2^24), in any order,
    and half of one is exact too.  Beyond 524,288 tokens a block's chunk is more than its 64 keys at hand."""
    import torch
    assert 4 * tokens < 2 ** 24
    ids = tokens_of(kind, tokens, vocab, tokens + dim)
    pad = int(ids[tokens // 3])
    for dt, ot, index, padding in ((torch.bfloat16, torch.float32, torch.int64, None), (torch.float32, torch.bfloat16, torch.int32, pad)):
        dy = whole((tokens, dim), 4, tokens, dt)
        out = torch.full((vocab, dim), float("nan"), dtype=ot, device="cuda")
        asr.asr_embedding_grads(ids.to(index), dy, out, scale=0.5, padding_idx=padding)
        want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double())
        if padding is not None:
            want[padding] = 0
        assert torch.equal(out, (want * 0.5).to(ot))


# rows to lanes, blocks of each size and no block; few rows, and many to a group of sums
@pytest.mark.parametrize("rows,cols", [(200_000, 8), (70_001, 24), (33, 64), (1300, 72), (9001, 512), (1500, 1032), (3001, 2560),
                                       (2100, 4096), (700, 8200), (640, 16384), (70, 16390), (2100, 20000)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("off", [0, 1])
def test_norm_gradients_lose_no_row(asr, rows, cols, dtype, off):
    """The sums over rows with every rstd 1 and every mean 0: of dy, and of dy x, at most 6 a row.  From x and from its codes
    (whole numbers up to 3 are multiples of their step, 2^-5), in memory of either alignment."""
    import torch
    assert 6 * rows < 2 ** 24
    dt = getattr(torch, dtype)

    def placed(t):
        return torch.zeros(t.numel() + off, dtype=dt, device="cuda")[off:].view(rows, cols).copy_(t)
    x, dy = placed(whole((rows, cols), 3, rows, dt)), placed(whole((rows, cols), 2, cols, dt))
    rstd, mean = torch.ones(rows, device="cuda"), torch.zeros(rows, device="cuda")
    kept = asr.checkpoint_int8(x)
    ww, wb = (dy.double() * x.double()).sum(0), dy.double().sum(0)
    for centred in (False, True):
        for codes in (None, (kept.q, kept.power)):
            for bias in (False, True):
                dw = torch.full((cols,), float("nan"), device="cuda")
                db = torch.full((cols,), float("nan"), device="cuda") if bias else None
                dx = torch.empty_like(x)
                asr.asr_layer_norm_grads(dy, None if codes else x, None, mean if centred else None, rstd, dx, dw, db,
                                         centred=centred, kept=codes)
                assert torch.equal(dw.double(), ww), (centred, codes is None, bias)
                assert db is None or torch.equal(db.double(), wb), (centred, codes is None)


# ------------------------------------------------------------ the activation far from zero

U = 2.0 ** -24


@pytest.mark.parametrize("function", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_activation_far_from_zero(asr, function, dtype):
    """An error of the exponential changes s(u) by s(u) s(-u) of it: little where u is large, and nothing where s(-u) is
    lost beside 1.  There f(a) = a and f'(a) = 1, bit for bit.

    Relative to e^-u the exponential is off by at most 9 U |u| (the argument's five roundings, three constants', and the
    product with log2 e) and 4 U of its own; s has two more roundings and f one: 20 U + 10 U |u| s(-u) of f.  f' = s (1 + r
    s(-u)), r = a u': s's error in both terms; s(-u)'s, (20 + 10 |u| s(u)) U of it where it is a product with e^-u (f32), and
    where it is 1 - s (bf16) the exponential's by s s(-u) and four roundings at 1; r and the sum, 8 U.  (r with |a| at most
    128, as s s(-u) is 0 beyond.)"""
    import torch
    import layer_reference as ref
    dt = getattr(torch, dtype)
    g = torch.Generator("cuda").manual_seed(7)
    spread = torch.exp(torch.empty(20000, device="cuda").uniform_(-8, 6, generator=g))
    spread *= torch.randint(0, 2, (20000,), device="cuda", generator=g) * 2 - 1
    far = torch.tensor([30.0, 87.0, 88.5, 100.0, 127.0, 128.0, 129.0, 1e3, 1e4, 1e6, 1e12, 3e38], device="cuda")
    x = torch.cat((spread, far, -far)).to(dt)[None]
    a = x.double()
    u = ref.argument(a, function)
    s, t = torch.sigmoid(u), torch.sigmoid(-u)
    small = a.clamp(-128, 128)
    r = small if function == "silu" else ref.argument(torch.ones_like(a), function) / 1.044715 * small * (1 + 3 * 0.044715 * small ** 2)
    y = asr.activation(x, function)
    dx = asr.activation_grads(torch.ones_like(x), x, function)
    step = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -124                                      # where e^-|u| is no normal number
    un = u.abs().clamp(max=200.0)                           # s(-u) or s(u) is 0 beyond
    f = ref.value(a, function)
    f_bound = (20 + 10 * un * t) * U * f.abs() + tiny * (1 + a.abs().clamp(max=1e3))
    assert ((y.double() - f).abs() <= f_bound + (f.abs() + f_bound) * step).all()
    df = ref.slope(a, function)
    ks = (20 + 10 * un * t) * U
    kt = (4 + (20 + 10 * un) * s * t) * U if dtype == "bfloat16" else (20 + 10 * un * s) * U * t
    df_bound = s * (ks * (1 + r.abs() * t) + r.abs() * (kt + 8 * U * t) + 8 * U) + tiny * (1 + r.abs())
    df_bound = torch.where(u > 25, torch.zeros_like(u), df_bound)
    assert ((dx.double() - df).abs() <= df_bound + (df.abs() + df_bound) * step).all()
    # f32: 1 + e^-u is 1 from u = 17.4 on, and r e^-u is lost beside 1 from 25 on (r at most 45 there, then falling)
    one = u > 25
    assert int(one.sum()) > 1500
    assert torch.equal(y[one], x[one]) and (dx[one] == 1).all()


# ------------------------------------------------------------------ in place

@pytest.mark.parametrize("rows,cols", [(9, 24), (1300, 72), (700, 512), (5, 515), (300, 4096), (40, 4104), (2500, 1032), (3, 16384),
                                       (5, 20001)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_the_norm_in_place(asr, rows, cols, dtype):
    """y may be x, with and without codes, of rows with a gap and of either alignment: the same bits, and nothing written
    between the rows."""
    import torch
    g = torch.Generator("cuda").manual_seed(cols)
    dt = getattr(torch, dtype)
    x = torch.randn(rows, cols, device="cuda", generator=g).to(dt)
    w, b = (torch.randn(cols, device="cuda", generator=g).to(dt) for _ in range(2))
    for centred in (True, False):
        want, saved = asr.layer_norm(x, w, b, centred=centred, save="int8", rounding="sr", step=2, seed=1)
        for off, gap in ((0, 0), (0, 32), (1, 3)):
            buf = torch.full((off + rows * (cols + gap),), 7.0, dtype=dt, device="cuda")
            z = buf[off:].view(rows, cols + gap)[:, :cols]
            for keep in (False, True):
                z.copy_(x)
                q = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
                power = torch.empty(rows, -(-cols // 32), dtype=torch.uint8, device="cuda")
                rstd = torch.empty(rows, device="cuda")
                asr.asr_layer_norm(z, w, b, z, None, rstd, centred=centred, keep=(q, power) if keep else None, rounding="sr",
                                   step=2, seed=1)
                assert torch.equal(z, want) and torch.equal(rstd, saved.rstd)
                assert (buf[:off] == 7).all() and (buf[off:].view(rows, cols + gap)[:, cols:] == 7).all()
                if keep:
                    assert torch.equal(q, saved.input.q) and torch.equal(power, saved.input.power)
