"""The operators around a weight that is trained in low precision, as cases to be timed and compared.

Four calls, one `kind` each:
  ortho    a stack of gradients orthogonalised by Newton-Schulz products;
  muon     a Muon step: momentum, orthogonalisation, and the decayed update written to bf16 weights by stochastic
           (or nearest) rounding;
  linear   a linear layer's forward product in 8-bit integers: tokens quantised in the call, one scale a token, against a
           weight quantised beforehand, one scale a channel;
  grads    that layer's backward products in 8-bit integers: the input's and the weight's gradient from the output's,
           whose 8-bit form is rounded stochastically.

`run` computes them in elementary torch operations in 32 bits, or, where `own` is true, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
LR, MOMENTUM, WEIGHT_DECAY = 0.02, 0.95, 0.1
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGEST = {"count": 32, "rows": 4096, "cols": 14336, "tokens": 8192}


def listed():
    return [
        # the smallest call: one adapter-sized matrix, where launches count
        {"name": "ortho_small", "kind": "ortho", "count": 1, "rows": 96, "cols": 160, "dtype": "bf16"},
        # the key and value projections of the 1.2B set (16 layers, 8 heads of 64), all in one call
        {"name": "ortho_kv", "kind": "ortho", "count": 32, "rows": 512, "cols": 2048, "dtype": "bf16"},
        # the largest: one feed-forward projection of the 8B set
        {"name": "ortho_ffn_8b", "kind": "ortho", "count": 1, "rows": 4096, "cols": 14336, "dtype": "bf16"},
        # eight of the 1.2B set's square attention projections, a layer group's step
        {"name": "muon_attn", "kind": "muon", "count": 8, "rows": 2048, "cols": 2048, "dtype": "bf16", "rounding": "sr"},
        # two tall feed-forward weights with f32 (accumulated) gradients
        {"name": "muon_ffn_f32", "kind": "muon", "count": 2, "rows": 8192, "cols": 2048, "dtype": "f32", "rounding": "sr"},
        # odd sizes, wide, nearest rounding
        {"name": "muon_odd", "kind": "muon", "count": 3, "rows": 515, "cols": 1365, "dtype": "bf16", "rounding": "rne"},
        # serving, one token: bound by reading the weight
        {"name": "linear_token", "kind": "linear", "tokens": 1, "n": 14336, "k": 4096, "rounding": "rne"},
        # serving, a ragged batch of tokens
        {"name": "linear_batch", "kind": "linear", "tokens": 33, "n": 4096, "k": 14336, "rounding": "rne"},
        # odd sizes in every direction, stochastic rounding of the outputs
        {"name": "linear_odd", "kind": "linear", "tokens": 777, "n": 1001, "k": 2049, "rounding": "sr"},
        # prefill or a training forward pass on the 8B set's feed-forward weight
        {"name": "linear_prefill", "kind": "linear", "tokens": 8192, "n": 14336, "k": 4096, "rounding": "rne"},
        # a backward pass on the 1.2B set's feed-forward weight
        {"name": "grads_ffn", "kind": "grads", "tokens": 4096, "n": 8192, "k": 2048},
        # a small odd backward pass
        {"name": "grads_odd", "kind": "grads", "tokens": 1111, "n": 515, "k": 1365},
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["ortho", "muon", "linear", "grads"])
    if kind in ("ortho", "muon"):
        most = _matrix_flops({"count": 1, "rows": LARGEST["rows"], "cols": LARGEST["cols"]})
        case = {"kind": kind, "count": _between(rng, 1, LARGEST["count"]), "rows": _between(rng, 8, LARGEST["rows"]),
                "cols": _between(rng, 8, LARGEST["cols"]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if rng.random() < 0.5:
            case["rows"], case["cols"] = case["cols"], case["rows"]
        if kind == "muon":
            case["rounding"] = rng.choice(["sr", "rne"])
        while _matrix_flops(case) > most or case["count"] * case["rows"] * case["cols"] > 60e6:
            case["count"] = case["count"] // 2
        return case
    case = {"kind": kind, "tokens": _between(rng, 1, LARGEST["tokens"]), "n": _between(rng, 64, 14336),
            "k": _between(rng, 64, 14336)}
    if kind == "linear":
        case["rounding"] = rng.choice(["rne", "sr"])
    most = 2.0 * 8192 * 14336 * 4096
    while work(case)["flops"] > most:
        case["n"] = max(64, case["n"] // 2 + 1)
        case["tokens"] = max(1, case["tokens"] // 2)
    return case


def _matrix_flops(case):
    """Multiplications and additions of the products: X X' and its square are symmetric, so half of each."""
    m, n = min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    return float(case["count"] * STEPS * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n))


def work(case):
    if case["kind"] in ("ortho", "muon"):
        size = float(case["count"] * case["rows"] * case["cols"])
        grad = 2 if case["dtype"] == "bf16" else 4
        if case["kind"] == "ortho":
            return {"bytes": size * (grad + 2), "flops": _matrix_flops(case)}
        return {"bytes": size * (grad + 2 * 2 + 2 * 4), "flops": _matrix_flops(case)}
    t, n, k = case["tokens"], case["n"], case["k"]
    if case["kind"] == "linear":
        return {"bytes": float(2 * t * k + n * k + 4 * n + 2 * t * n), "flops": 2.0 * t * n * k}
    return {"bytes": float(2 * t * n + 2 * t * k + 2 * n * k + 2 * t * k + 2 * n * k), "flops": 4.0 * t * n * k}


# ------------------------------------------------------------------ inputs


def _gradients(gen, case):
    """Gradients of a weight: noise and a few strong directions, at the size that a trained layer's have."""
    count, rows, cols = case["count"], case["rows"], case["cols"]
    rank = min(8, rows, cols)
    g = torch.randn(count, rows, cols, device="cuda", generator=gen)
    u = torch.randn(count, rows, rank, device="cuda", generator=gen)
    v = torch.randn(count, rank, cols, device="cuda", generator=gen)
    return (1e-3 * (g + 0.5 * (u @ v))).to(DTYPES[case["dtype"]])


def _padded(rows, cols):
    """An int8 matrix whose rows begin a multiple of 16 bytes apart."""
    return torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"case": dict(case), "seed": 1000 + seed, "step": 1 + seed % 1000}
    if case["kind"] in ("ortho", "muon"):
        state["grad"] = _gradients(gen, case)
        if case["kind"] == "muon":
            shape = state["grad"].shape
            state["param"] = (0.02 * torch.randn(shape, device="cuda", generator=gen)).to(torch.bfloat16)
            state["momentum"] = 3e-4 * torch.randn(shape, device="cuda", generator=gen)
        return state
    t, n, k = case["tokens"], case["n"], case["k"]
    weight = (0.02 * torch.randn(n, k, device="cuda", generator=gen)).to(torch.bfloat16)
    x = torch.randn(t, k, device="cuda", generator=gen)
    x = x * (1.0 + 3.0 * (torch.rand(k, device="cuda", generator=gen) < 0.01))     # a few strong channels
    state["x"] = x.to(torch.bfloat16)
    if case["kind"] == "linear":
        scale = weight.float().abs().amax(1) / 127.0
        state["qweight"] = _padded(n, k)
        state["qweight"].copy_(torch.round(weight.float() / scale[:, None]).to(torch.int8))
        state["wscale"] = scale
    else:
        state["weight"] = weight
        state["dy"] = (1e-3 * torch.randn(t, n, device="cuda", generator=gen)).to(torch.bfloat16)
    return state


# ------------------------------------------------------------- plain forms


def _mulhilo(a, b):
    """High and low words of the product of the constant a and the 32-bit words b (held in 64-bit integers)."""
    high = ((a >> 16) * b + (((a & 0xFFFF) * b) >> 16)) >> 16
    return high, (a * b) & 0xFFFFFFFF


def _bits16(shape, step, seed, device):
    """The low 16 bits of each element's Philox4x32-10 word: word (i & 3) at counter (i >> 2, step, 0), key seed."""
    size = math.prod(shape)
    q = torch.arange((size + 3) // 4, dtype=torch.int64, device=device)
    c0, c1, c2, c3 = q & 0xFFFFFFFF, q >> 32, torch.full_like(q, step), torch.zeros_like(q)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(0xD2511F53, c0)
        h1, l1 = _mulhilo(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return (torch.stack((c0, c1, c2, c3), 1).reshape(-1)[:size] & 0xFFFF).reshape(shape)


def _to_bf16(x, rounding, step, seed):
    """Finite f32 values to bf16: 16 random bits added below the kept ones and the sum cut, or to nearest."""
    if rounding == "rne":
        return x.to(torch.bfloat16)
    word = x.contiguous().view(torch.int32).to(torch.int64) & 0xFFFFFFFF
    word = (word + _bits16(x.shape, step, seed, x.device)) >> 16
    return (word << 16).to(torch.int32).view(torch.float32).to(torch.bfloat16)


def _quantise(x, dim, bits=None):
    """8-bit whole numbers (as f32) and scales along `dim`: to nearest, or up with the fraction's probability."""
    top = x.abs().amax(dim, keepdim=True)
    y = x * torch.where(top > 0, 127.0 / top, torch.zeros_like(top))
    if bits is None:
        q = torch.round(y)
    else:
        low = torch.floor(y)
        q = low + ((y - low) * 65536.0 > bits).float()
    return q.clamp(-127.0, 127.0), top / 127.0


def _newton_schulz(g):
    a, b, c = COEFFICIENTS
    tall = g.shape[-2] > g.shape[-1]
    x = g.mT if tall else g
    x = x / x.square().sum((-2, -1), keepdim=True).sqrt().clamp(min=EPS)
    for _ in range(STEPS):
        s = x @ x.mT
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.mT if tall else x


def _plain(state):
    case = state["case"]
    if case["kind"] == "ortho":
        return {"update": _newton_schulz(state["grad"].float()).to(torch.bfloat16).contiguous()}
    if case["kind"] == "muon":
        g, m = state["grad"].float(), state["momentum"]
        m = m + (1.0 - MOMENTUM) * (g - m)
        o = _newton_schulz(g + MOMENTUM * (m - g))
        adjust = 0.2 * math.sqrt(max(case["rows"], case["cols"]))
        p = state["param"].float() * (1.0 - LR * WEIGHT_DECAY) - (LR * adjust) * o
        return {"param": _to_bf16(p, case["rounding"], state["step"], state["seed"]), "momentum": m}
    x = state["x"].float()
    if case["kind"] == "linear":
        q, s = _quantise(x, 1)
        y = (q @ state["qweight"].float().T) * s * state["wscale"]
        return {"y": _to_bf16(y, case["rounding"], state["step"], state["seed"])}
    dy, w = state["dy"].float(), state["weight"].float()
    bits = _bits16(dy.shape, state["step"], state["seed"], dy.device)
    q, s = _quantise(dy, 1, bits)
    v, t = _quantise(w, 0)
    dx = (q @ v) * s * t
    q, s = _quantise(dy, 0, bits)
    v, t = _quantise(x, 0)
    return {"dx": dx.to(torch.bfloat16), "dw": ((q.T @ v) * s.T * t).to(torch.bfloat16)}


def _own(state):
    import stochastic_rounding_gb300 as asr
    case = state["case"]
    if case["kind"] == "ortho":
        update = torch.empty_like(state["grad"], dtype=torch.bfloat16)
        asr.asr_newton_schulz([(state["grad"], update)], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        return {"update": update}
    if case["kind"] == "muon":
        # the step is in place: it goes on copies, so that a pass can be made again
        p, m = state["param"].clone(), state["momentum"].clone()
        asr.asr_muon_sr_multi_tensor([(p, state["grad"], m, 0)], lr=LR, momentum=MOMENTUM, weight_decay=WEIGHT_DECAY,
                                     nesterov=True, steps=STEPS, coefficients=COEFFICIENTS, eps=EPS,
                                     adjust="match_rms_adamw", step=state["step"], seed=state["seed"],
                                     rounding=case["rounding"])
        return {"param": p, "momentum": m}
    if case["kind"] == "linear":
        return {"y": asr.int8_linear(state["x"], state["qweight"], state["wscale"], rounding=case["rounding"],
                                     step=state["step"], seed=state["seed"])}
    dx, dw = asr.int8_linear_grads(state["dy"], state["x"], state["weight"], step=state["step"], seed=state["seed"])
    return {"dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- the same in 64 bits


def _words16(size, step, seed):
    """Philox4x32-10 on unsigned 64-bit arrays, whose products of two 32-bit words are exact."""
    low = np.uint64(0xFFFFFFFF)
    index = np.arange((size + 3) // 4, dtype=np.uint64)
    word = [index & low, index >> np.uint64(32), np.full_like(index, step), np.zeros_like(index)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, r = word[0] * np.uint64(0xD2511F53), word[2] * np.uint64(0xCD9E8D57)
        word = [(r >> np.uint64(32)) ^ word[1] ^ np.uint64(key[0]), r & low,
                (p >> np.uint64(32)) ^ word[3] ^ np.uint64(key[1]), p & low]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    out = np.empty((index.size, 4), dtype=np.int32)
    for j in range(4):
        out[:, j] = (word[j] & np.uint64(0xFFFF)).astype(np.int32)
    return torch.from_numpy(out.reshape(-1)[:size])


def _levels(x, dim, bits=None):
    """(whole numbers, step) of x in 64 bits: x is nearest to number * step, or one of its two neighbours by `bits`."""
    step = x.abs().max(dim, keepdim=True).values / 127
    y = torch.where(step > 0, x / step, torch.zeros_like(x))
    if bits is None:
        return torch.round(y).clamp(-127, 127), step
    low = torch.floor(y)
    return torch.where(y - low > bits.double() / 65536, low + 1, low).clamp(-127, 127), step


def _orthogonal(g):
    out = torch.empty_like(g)
    a, b, c = COEFFICIENTS
    for i in range(g.shape[0]):
        x = g[i]
        x = x / max(float(torch.linalg.matrix_norm(x)), EPS)
        for _ in range(STEPS):
            if x.shape[0] <= x.shape[1]:
                s = torch.mm(x, x.t())
                x = a * x + b * torch.mm(s, x) + c * torch.mm(s, torch.mm(s, x))
            else:
                s = torch.mm(x.t(), x)
                x = a * x + b * torch.mm(x, s) + c * torch.mm(torch.mm(x, s), s)
        out[i] = x
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["kind"] == "ortho":
        return {"update": _orthogonal(state["grad"].double())}
    if case["kind"] == "muon":
        g = state["grad"].double()
        m = MOMENTUM * state["momentum"].double() + (1 - MOMENTUM) * g
        o = _orthogonal(MOMENTUM * m + (1 - MOMENTUM) * g)
        rate = LR * 0.2 * max(case["rows"], case["cols"]) ** 0.5
        return {"param": (1 - LR * WEIGHT_DECAY) * state["param"].double() - rate * o, "momentum": m}
    x = state["x"].double()
    if case["kind"] == "linear":
        q, s = _levels(x, 1)
        return {"y": torch.mm(q * s, (state["qweight"].double() * state["wscale"].double()[:, None]).t())}
    dy, w = state["dy"].double(), state["weight"].double()
    bits = _words16(dy.numel(), state["step"], state["seed"]).to(dy.device).reshape(dy.shape)
    q, s = _levels(dy, 1, bits)
    v, t = _levels(w, 0)
    dx = torch.mm(q * s, v * t)
    q, s = _levels(dy, 0, bits)
    v, t = _levels(x, 0)
    return {"dx": dx, "dw": torch.mm((q * s).t(), v * t)}
