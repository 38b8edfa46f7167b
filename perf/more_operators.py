"""The parts of a layer between its 8-bit products, as cases to be timed and compared.

Four operators, one `kind` each:
  norm        layer norm (or, not centred, the norm by the root mean square): y = (x - mean) rstd w + b, and its backward
              pass with the reduction of the weight's and the bias's gradient;
  act         a layer's activation, x sigmoid(x) ("silu") or the tanh form of gelu, alone or gated (the first half of the
              columns through the function, times the second half), and its backward pass;
  checkpoint  what a layer keeps of its input for the backward pass, in 8 bits: 32 values of a row share a power of two;
              made, and turned back into values;
  embed       rows of a table picked by token and scaled, and the table's gradient, summed by sorted tokens.

A case's `mode` is "forward" (one call), "train" (forward, then backward from what the forward pass read) or "train8" (the
same with the input kept in 8 bits between the two); for embed "forward" or "grads".

`run` computes them in elementary torch operations in 32 bits, or, where `own` is true, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
GROUP = 32                      # values of a row that share a scale
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST_VALUES = 8192 * 14336      # of x or y, and
MOST_TABLE = 128256 * 4096      # of a table


def listed():
    return [
        # serving, one token: where a launch's latency counts
        {"name": "norm_token", "kind": "norm", "mode": "forward", "rows": 1, "cols": 4096, "dtype": "bf16", "centred": True,
         "rounding": "rne"},
        # a training step over the 8B set's width, by the root mean square, the input kept in 8 bits
        {"name": "norm_8b", "kind": "norm", "mode": "train8", "rows": 8192, "cols": 4096, "dtype": "bf16", "centred": False,
         "rounding": "rne"},
        # odd sizes in f32, the input kept as it is
        {"name": "norm_odd", "kind": "norm", "mode": "train", "rows": 777, "cols": 1365, "dtype": "f32", "centred": True,
         "rounding": "rne"},
        # the input of the 8B set's second feed-forward product, kept with stochastic rounding
        {"name": "checkpoint_ffn", "kind": "checkpoint", "rows": 8192, "cols": 14336, "dtype": "bf16", "rounding": "sr"},
        # odd sizes in f32
        {"name": "checkpoint_odd", "kind": "checkpoint", "rows": 1001, "cols": 2049, "dtype": "f32", "rounding": "rne"},
        # serving, a ragged batch of tokens through the 8B set's feed-forward activation
        {"name": "act_batch", "kind": "act", "mode": "forward", "rows": 33, "cols": 14336, "dtype": "bf16", "function": "silu",
         "gated": True, "rounding": "rne"},
        # the largest: a training step of that activation, its input kept in 8 bits, rounded stochastically
        {"name": "act_ffn", "kind": "act", "mode": "train8", "rows": 8192, "cols": 14336, "dtype": "bf16", "function": "silu",
         "gated": True, "rounding": "sr"},
        # odd sizes, gelu, not gated
        {"name": "act_odd", "kind": "act", "mode": "train8", "rows": 1111, "cols": 1365, "dtype": "bf16", "function": "gelu",
         "gated": False, "rounding": "rne"},
        # serving, a ragged batch of tokens
        {"name": "embed_batch", "kind": "embed", "mode": "forward", "tokens": 33, "vocab": 128256, "dim": 4096, "dtype": "bf16",
         "scaled": False, "padded": False, "index": "int64"},
        # a training batch's rows of the 8B set's table, scaled by the root of the width
        {"name": "embed_train", "kind": "embed", "mode": "forward", "tokens": 8192, "vocab": 128256, "dim": 4096,
         "dtype": "bf16", "scaled": True, "padded": False, "index": "int64"},
        # and that table's whole gradient, which an optimizer of this package takes
        {"name": "embed_grads", "kind": "embed", "mode": "grads", "tokens": 8192, "vocab": 128256, "dim": 4096, "dtype": "bf16",
         "scaled": True, "padded": False, "index": "int64"},
        # a small odd table, most rows of it used more than once, the last tokens padding
        {"name": "embed_grads_odd", "kind": "embed", "mode": "grads", "tokens": 2049, "vocab": 1001, "dim": 515, "dtype": "f32",
         "scaled": False, "padded": True, "index": "int32"},
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm", "checkpoint", "act", "embed"])
    case = {"kind": kind, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if kind == "embed":
        case.update(mode=rng.choice(["forward", "grads"]), tokens=_between(rng, 1, 16384), vocab=_between(rng, 16, 128256),
                    dim=_between(rng, 16, 8192), scaled=rng.random() < 0.5, padded=rng.random() < 0.5,
                    index=rng.choice(["int64", "int32"]))
        while case["vocab"] * case["dim"] * (2 if case["dtype"] == "f32" else 1) > MOST_TABLE:
            case["vocab"] = case["vocab"] // 2 + 1
        return case
    case.update(rows=_between(rng, 1, 16384), cols=_between(rng, 16, 16384), rounding=rng.choice(["sr", "rne"]))
    if kind == "norm":
        case.update(mode=rng.choice(["forward", "train", "train8"]), centred=rng.random() < 0.5)
    if kind == "act":
        case.update(mode=rng.choice(["forward", "train", "train8"]), function=rng.choice(["silu", "gelu"]),
                    gated=rng.random() < 0.5)
    while case["rows"] * case["cols"] * (2 if case["dtype"] == "f32" else 1) > MOST_VALUES:
        case["rows"] = case["rows"] // 2 + 1
    return case


def _kept_bytes(rows, cols):
    return rows * (cols + (cols + GROUP - 1) // GROUP)


def work(case):
    """Each input read and each output written once; what is kept in 8 bits is an output of the forward pass and an input of
    the backward pass."""
    size = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "embed":
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        index = 8 if case["index"] == "int64" else 4
        if case["mode"] == "forward":
            return {"bytes": float(t * index + size * (min(t, v) * d + t * d)), "flops": float(t * d)}
        return {"bytes": float(t * index + size * (t * d + v * d)), "flops": float(2 * t * d)}
    rows, cols = case["rows"], case["cols"]
    if case["kind"] == "checkpoint":
        return {"bytes": float(2 * (size * rows * cols + _kept_bytes(rows, cols))), "flops": float(4 * rows * cols)}
    if case["kind"] == "norm":
        x, params = size * rows * cols, size * cols * (2 if case["centred"] else 1)
        total, flops = 2 * x + params, 8 * rows * cols
        if case["mode"] != "forward":
            total += 2 * x + size * cols + params + (x if case["mode"] == "train" else 2 * _kept_bytes(rows, cols))
            flops += 14 * rows * cols
        return {"bytes": float(total), "flops": float(flops)}
    y = size * rows * cols
    width = cols * (2 if case["gated"] else 1)
    x = size * rows * width
    total, flops = x + y, 8 * rows * cols
    if case["mode"] != "forward":
        total += y + x + (x if case["mode"] == "train" else 2 * _kept_bytes(rows, width))
        flops += 16 * rows * cols
    return {"bytes": float(total), "flops": float(flops)}


# ------------------------------------------------------------------ inputs


def _values(gen, rows, cols, dtype):
    """A layer's values: noise, a few strong channels, channels with an offset, tokens of several sizes."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    x *= 1.0 + 9.0 * (torch.rand(cols, device="cuda", generator=gen) < 0.01)
    x += 0.2 * torch.randn(cols, device="cuda", generator=gen)
    x *= 0.5 + torch.rand(rows, 1, device="cuda", generator=gen)
    return x.to(DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    state = {"case": dict(case), "seed": 1000 + seed, "step": 1 + seed % 1000}
    if case["kind"] == "embed":
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        # the k-th token of a language comes with a frequency of about 1 / k
        ids = torch.exp(torch.rand(t, device="cuda", generator=gen, dtype=torch.float64) * math.log(v)).long().clamp(1, v) - 1
        if case["padded"]:
            ids[t - t // 8:] = v - 1
        state["ids"] = ids.to(torch.int64 if case["index"] == "int64" else torch.int32)
        state["padding"] = v - 1 if case["padded"] else None
        state["scale"] = math.sqrt(d) if case["scaled"] else 1.0
        if case["mode"] == "forward":
            state["table"] = (0.02 * torch.randn(v, d, device="cuda", generator=gen)).to(dtype)
        else:
            state["dy"] = (1e-3 * torch.randn(t, d, device="cuda", generator=gen)).to(dtype)
        return state
    rows, cols = case["rows"], case["cols"]
    width = 2 * cols if case["kind"] == "act" and case["gated"] else cols
    state["x"] = _values(gen, rows, width, case["dtype"])
    if case["kind"] == "norm":
        state["weight"] = (1.0 + 0.1 * torch.randn(cols, device="cuda", generator=gen)).to(dtype)
        state["bias"] = (0.1 * torch.randn(cols, device="cuda", generator=gen)).to(dtype) if case["centred"] else None
    if case["kind"] != "checkpoint" and case["mode"] != "forward":
        state["dy"] = (1e-3 * torch.randn(rows, cols, device="cuda", generator=gen)).to(dtype)
    return state


# ------------------------------------------------------------- plain forms


def _mulhilo(a, b):
    """High and low words of the product of the constant a and the 32-bit words b (held in 64-bit integers)."""
    high = ((a >> 16) * b + (((a & 0xFFFF) * b) >> 16)) >> 16
    return high, (a * b) & 0xFFFFFFFF


def _kept_bits(rows, groups, step, seed, device):
    """Sixteen random bits for every value of whole groups: eight values to a Philox4x32-10 counter (i >> 3, step, 1), i the
    value's place in rows of whole groups; word (i >> 1) & 3, the low half where i is even."""
    q = torch.arange(rows * groups * GROUP // 8, dtype=torch.int64, device=device)
    c0, c1, c2, c3 = q & 0xFFFFFFFF, q >> 32, torch.full_like(q, step), torch.ones_like(q)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(0xD2511F53, c0)
        h1, l1 = _mulhilo(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack((c0, c1, c2, c3), 1)
    return torch.stack((words & 0xFFFF, words >> 16), 2).to(torch.int32).reshape(rows, groups, GROUP)


def _kept(x, rounding, step, seed):
    """The values that x's 8-bit form stands for, in f32: whole numbers of at most 127 times a power of two for every 32."""
    rows, cols = x.shape
    groups = (cols + GROUP - 1) // GROUP
    v = torch.zeros(rows, groups * GROUP, device=x.device)
    v[:, :cols] = x
    v = v.reshape(rows, groups, GROUP)
    # the least power of two whose 127-fold is no less than the largest: by its bits, 127 = 2^6 * 1.984375
    top = v.abs().amax(2, keepdim=True).view(torch.int32)
    power = (((top + 0x1FFFF) >> 23) - 6).clamp(min=0)
    y = v * ((254 - power) << 23).view(torch.float32)
    if rounding == "rne":
        q = torch.round(y)
    else:
        q = torch.floor(y)
        q += (y - q) * 65536.0 > _kept_bits(rows, groups, step, seed, x.device)
    q *= torch.where(power > 0, power << 23, torch.full_like(power, 0x400000)).view(torch.float32)
    return q.reshape(rows, groups * GROUP)[:, :cols]


def _norm(state):
    case, x, w = state["case"], state["x"].float(), state["weight"].float()
    mean = x.mean(1, keepdim=True) if case["centred"] else torch.zeros(x.shape[0], 1, device=x.device)
    rstd = 1.0 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + EPS)
    y = (x - mean) * rstd * w
    if state["bias"] is not None:
        y = y + state["bias"].float()
    dtype = state["x"].dtype
    out = {"y": y.to(dtype)}
    if case["mode"] == "forward":
        return out
    if case["mode"] == "train8":
        x = _kept(x, case["rounding"], state["step"], state["seed"])
    hat, dy = (x - mean) * rstd, state["dy"].float()
    g = dy * w
    dx = g - hat * (g * hat).mean(1, keepdim=True)
    if case["centred"]:
        dx = dx - g.mean(1, keepdim=True)
        out["dbias"] = dy.sum(0).to(dtype)
    out["dx"] = (dx * rstd).to(dtype)
    out["dweight"] = (dy * hat).sum(0).to(dtype)
    return out


def _sigmoid(u):
    t = torch.exp(-u.abs())
    return torch.where(u >= 0, torch.ones_like(t), t) / (1.0 + t)


def _argument(a, function):
    """Both functions are a sigmoid(u): u, and its derivative by a."""
    if function == "silu":
        return a, torch.ones_like(a)
    c = 2.0 * math.sqrt(2.0 / math.pi)
    return c * (a + 0.044715 * a * a * a), c * (1.0 + 0.134145 * a * a)


def _act(state):
    case, x, cols = state["case"], state["x"].float(), state["case"]["cols"]
    a = x[:, :cols]
    y = a * _sigmoid(_argument(a, case["function"])[0])
    if case["gated"]:
        y = y * x[:, cols:]
    dtype = state["x"].dtype
    out = {"y": y.to(dtype)}
    if case["mode"] == "forward":
        return out
    if case["mode"] == "train8":
        x = _kept(x, case["rounding"], state["step"], state["seed"])
        a = x[:, :cols]
    dy = state["dy"].float()
    u, slope = _argument(a, case["function"])
    s = _sigmoid(u)
    da = dy * s * (1.0 + a * slope * _sigmoid(-u))
    if case["gated"]:
        da = torch.cat((da * x[:, cols:], dy * a * s), 1)
    out["dx"] = da.to(dtype)
    return out


def _embed(state):
    case, ids = state["case"], state["ids"].long()
    scale = torch.tensor(state["scale"], dtype=torch.float32, device=ids.device)
    if case["mode"] == "forward":
        return {"y": (state["table"][ids].float() * scale).to(state["table"].dtype)}
    dy, (t, d) = state["dy"].float(), state["dy"].shape
    if state["padding"] is not None:
        dy = torch.where((ids == state["padding"])[:, None], torch.zeros_like(dy), dy)
    # tokens sorted; the rows of one token are added up in 64 bits by running sums, block by block of the columns
    order = torch.argsort(ids, stable=True)
    rows, count = torch.unique_consecutive(ids[order], return_counts=True)
    ends = torch.cumsum(count, 0) - 1
    out = torch.zeros(case["vocab"], d, dtype=state["dy"].dtype, device=ids.device)
    for c in range(0, d, 1024):
        total = torch.cumsum(dy[order, c:c + 1024].double(), 0)[ends]
        total[1:] -= total[:-1].clone()
        out[rows, c:c + 1024] = (total.float() * scale).to(out.dtype)
    if state["padding"] is not None:
        out[state["padding"]] = 0
    return {"dtable": out}


def _plain(state):
    kind = state["case"]["kind"]
    if kind == "norm":
        return _norm(state)
    if kind == "act":
        return _act(state)
    if kind == "embed":
        return _embed(state)
    return {"kept": _kept(state["x"].float(), state["case"]["rounding"], state["step"], state["seed"]).to(state["x"].dtype)}


def _own(state):
    import stochastic_rounding_gb300 as asr
    case = state["case"]
    key = {"rounding": case.get("rounding"), "step": state["step"], "seed": state["seed"]}
    if case["kind"] == "embed":
        if case["mode"] == "forward":
            return {"y": asr.embedding(state["ids"], state["table"], scale=state["scale"])}
        return {"dtable": asr.embedding_grads(state["ids"], state["dy"], case["vocab"], scale=state["scale"],
                                              padding_idx=state["padding"])}
    if case["kind"] == "checkpoint":
        return {"kept": asr.restore_int8(asr.checkpoint_int8(state["x"], **key))}
    if case["kind"] == "norm":
        x, w, b = state["x"], state["weight"], state["bias"]
        if case["mode"] == "forward":
            return {"y": asr.layer_norm(x, w, b, eps=EPS, centred=case["centred"])}
        if case["mode"] == "train":
            y, saved = asr.layer_norm(x, w, b, eps=EPS, centred=case["centred"], save="input")
        else:
            y, saved = asr.layer_norm(x, w, b, eps=EPS, centred=case["centred"], save="int8", **key)
        dx, dw, db = asr.layer_norm_grads(state["dy"], saved, w, need_dbias=b is not None)
        out = {"y": y, "dx": dx, "dweight": dw}
        if b is not None:
            out["dbias"] = db
        return out
    x, function, gated = state["x"], case["function"], case["gated"]
    if case["mode"] == "forward":
        return {"y": asr.activation(x, function, gated=gated)}
    if case["mode"] == "train":
        y, saved = asr.activation(x, function, gated=gated, save="input")
    else:
        y, saved = asr.activation(x, function, gated=gated, save="int8", **key)
    return {"y": y, "dx": asr.activation_grads(state["dy"], saved, function, gated=gated)}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- the same in 64 bits


def _halves(count, step, seed):
    """Philox4x32-10 on unsigned 64-bit arrays, whose products of two 32-bit words are exact: the eight halves of each of
    `count` counters' outputs in order, from low to high."""
    low = np.uint64(0xFFFFFFFF)
    index = np.arange(count, dtype=np.uint64)
    word = [index & low, index >> np.uint64(32), np.full_like(index, step), np.full_like(index, 1)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, r = word[0] * np.uint64(0xD2511F53), word[2] * np.uint64(0xCD9E8D57)
        word = [(r >> np.uint64(32)) ^ word[1] ^ np.uint64(key[0]), r & low,
                (p >> np.uint64(32)) ^ word[3] ^ np.uint64(key[1]), p & low]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    out = np.empty((count, 4), dtype="<u4")
    for j in range(4):
        out[:, j] = word[j].astype(np.uint32)
    return torch.from_numpy(out.view("<u2").astype(np.int32).reshape(-1))


def _stands_for(x, case, state):
    """What x (64 bits) is kept as, group by group of columns: a whole number times the least power of two, at least
    2^-127, that leaves none above 127."""
    rows, cols = x.shape
    across = -(-cols // GROUP)
    bits = None
    if case["rounding"] == "sr":
        bits = _halves(rows * across * GROUP // 8, state["step"], state["seed"]).to(x.device).reshape(rows, across, GROUP)
    whole = torch.nn.functional.pad(x, (0, across * GROUP - cols)).reshape(rows, across, GROUP)
    part, exponent = torch.frexp(whole.abs().max(2, keepdim=True).values)
    exponent = torch.where(part * 128 > 127, exponent - 6, exponent - 7)
    exponent = torch.where(part == 0, torch.full_like(exponent, -127), exponent).clamp(min=-127)
    scale = ((exponent.long() + 1023) << 52).view(torch.float64)        # 2^exponent itself: pow need not give it
    number = whole / scale
    if bits is None:
        number = torch.round(number)
    else:
        below = torch.floor(number)
        number = torch.where(number - below > bits.double() / 65536, below + 1, below)
    return (number * scale).reshape(rows, -1)[:, :cols]


def _exact_norm(case, state):
    x, w, n = state["x"].double(), state["weight"].double(), case["cols"]
    shift = torch.sum(x, 1, keepdim=True) / n if case["centred"] else 0.0
    inverse = torch.rsqrt(torch.sum((x - shift) ** 2, 1, keepdim=True) / n + EPS)
    y = (x - shift) * inverse * w
    out = {"y": y if state["bias"] is None else y + state["bias"].double()}
    if case["mode"] == "forward":
        return out
    if case["mode"] == "train8":
        x = _stands_for(x, case, state)
    hat = (x - shift) * inverse
    dy = state["dy"].double()
    back = dy * w
    along = torch.sum(back * hat, 1, keepdim=True) / n
    if case["centred"]:
        out["dbias"] = torch.sum(dy, 0)
        out["dx"] = inverse * (back - torch.sum(back, 1, keepdim=True) / n - hat * along)
    else:
        out["dx"] = inverse * (back - hat * along)
    out["dweight"] = torch.sum(dy * hat, 0)
    return out


def _value_and_slope(a, function):
    if function == "silu":
        s = torch.sigmoid(a)
        return a * s, s + a * s * (1 - s)
    k = (2 / math.pi) ** 0.5
    h = torch.tanh(k * (a + 0.044715 * a ** 3))
    # 1 + h loses its digits far below zero, where the exponential has them
    half = torch.sigmoid(2 * k * (a + 0.044715 * a ** 3))
    return a * half, half + 0.5 * a * (1 - h * h) * k * (1 + 3 * 0.044715 * a * a)


def _exact_act(case, state):
    x, n = state["x"].double(), case["cols"]
    y, _ = _value_and_slope(x[:, :n], case["function"])
    out = {"y": y * x[:, n:] if case["gated"] else y}
    if case["mode"] == "forward":
        return out
    if case["mode"] == "train8":
        x = _stands_for(x, case, state)
    value, slope = _value_and_slope(x[:, :n], case["function"])
    dy = state["dy"].double()
    if not case["gated"]:
        out["dx"] = dy * slope
    else:
        out["dx"] = torch.empty_like(x)
        out["dx"][:, :n] = dy * slope * x[:, n:]
        out["dx"][:, n:] = dy * value
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["kind"] == "norm":
        return _exact_norm(case, state)
    if case["kind"] == "act":
        return _exact_act(case, state)
    if case["kind"] == "checkpoint":
        return {"kept": _stands_for(state["x"].double(), case, state)}
    ids = state["ids"].long()
    if case["mode"] == "forward":
        return {"y": torch.index_select(state["table"].double(), 0, ids) * state["scale"]}
    if state["padding"] is not None:
        live = torch.nonzero(ids != state["padding"])[:, 0]
    else:
        live = torch.arange(ids.numel(), device=ids.device)
    out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device=ids.device)
    return {"dtable": out.index_add_(0, ids[live], state["dy"][live].double()).mul_(state["scale"])}
