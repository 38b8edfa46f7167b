"""The operators between a layer's 8-bit products in 64 bits, from their definitions, for the tests."""
import math

import numpy as np
import torch


def words16(rows, cols, step, seed, orc, base=0):
    """The 16 random bits of each value of a rows x cols checkpoint, from the oracle's Philox words."""
    across = -(-cols // 32) * 32
    words = orc.philox_fill(rows * across // 8, base // 8, step, 1, seed).reshape(-1, 4)
    halves = np.stack([words & 0xFFFF, words >> 16], 2).reshape(rows, across)[:, :cols]
    return torch.from_numpy(halves.astype(np.int64))


def checkpoint(x, bits=None):
    """(codes, powers as stored, values) of x, row by row of groups of 32, on the CPU in 64 bits."""
    x = x.detach().double().cpu()
    rows, cols = x.shape
    groups = -(-cols // 32)
    wide = torch.zeros(rows, groups * 32, dtype=torch.float64)
    wide[:, :cols] = x
    wide = wide.reshape(rows, groups, 32)
    bad = ~torch.isfinite(wide).all(2)
    clean = torch.where(bad[..., None], torch.zeros_like(wide), wide)
    top = clean.abs().amax(2)
    m, e = torch.frexp(top)
    e = e.long() - torch.where(m * 128 > 127, 6, 7)
    e = torch.where(top == 0, torch.full_like(e, -127), e).clamp(min=-127)
    power_of_two = lambda n: ((n[..., None] + 1023) << 52).view(torch.float64)  # noqa: E731
    y = clean * power_of_two(-e)
    if bits is None:
        q = torch.round(y)
    else:
        r = torch.zeros(rows, groups * 32, dtype=torch.float64)
        r[:, :cols] = bits.double()
        low = torch.floor(y)
        q = low + ((y - low) * 65536 > r.reshape_as(y)).double()
    value = q * power_of_two(e)
    power = torch.where(bad, torch.full_like(e, 255), e + 127)
    value = torch.where(bad[..., None], torch.full_like(value, math.nan), value)
    q = torch.where(bad[..., None], torch.zeros_like(q), q)
    flat = lambda t: t.reshape(rows, groups * 32)[:, :cols]  # noqa: E731
    return flat(q), power, flat(value)


def norm(x, w, b, eps, centred):
    """(y, mean, rstd, h)."""
    x = x.double()
    mean = x.mean(1, keepdim=True) if centred else torch.zeros(x.shape[0], 1, dtype=torch.float64, device=x.device)
    rstd = ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    h = (x - mean) * rstd
    y = h if w is None else h * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean, rstd, h


def norm_grads(dy, x, w, mean, rstd, centred):
    """(dx, dw, db) at x with given mean and rstd."""
    dy, h = dy.double(), (x.double() - mean) * rstd
    g = dy if w is None else dy * w.double()
    dx = g - h * (g * h).mean(1, keepdim=True)
    if centred:
        dx = dx - g.mean(1, keepdim=True)
    return dx * rstd, (dy * h).sum(0), dy.sum(0)


def argument(a, function):
    return a if function == "silu" else math.sqrt(8 / math.pi) * (a + 0.044715 * a ** 3)


def value(a, function):
    a = a.double()
    return a * torch.sigmoid(argument(a, function))


def slope(a, function):
    a = a.double()
    u = argument(a, function)
    du = torch.ones_like(a) if function == "silu" else math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * a * a)
    s, t = torch.sigmoid(u), torch.sigmoid(-u)
    return s + torch.where(t == 0, torch.zeros_like(t), a * du * s * t)


def activation(x, function, gated):
    n = x.shape[1] // 2 if gated else x.shape[1]
    y = value(x[:, :n], function)
    return y * x[:, n:].double() if gated else y


def activation_grads(dy, x, function, gated):
    n = dy.shape[1]
    x, dy = x.double(), dy.double()
    da = dy * slope(x[:, :n], function)
    return torch.cat((da * x[:, n:], dy * value(x[:, :n], function)), 1) if gated else da


def embedding_grads(ids, dy, vocab, scale, padding=None):
    out = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device=dy.device)
    ids = ids.long()
    live = (ids >= 0) & (ids < vocab)
    if padding is not None:
        live &= ids != padding
    return out.index_add_(0, ids[live], dy.double()[live]) * scale
