"""Operators on matrix parameters, as measured work.

Orthogonalisation of matrices by a Newton-Schulz iteration ("ortho"), the optimizer step that takes it of its momentum
("muon"), MXFP4 quantisation along rows and columns with the values read back ("quant"), and the MXFP4 matrix product:
a layer's output for tokens that arrive in 16 bits ("linear"), and its training step ("train": output, the inputs'
gradient and the weights').

MXFP4 is e2m1 codes, two per byte, with one power-of-two scale (e8m0) per 32 consecutive elements of a row.
"""

import math
import random

import torch

own = False

MASK = 0xFFFFFFFF
BLOCK = 32
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
COEFS = (3.4445, -4.7750, 2.0315)  # the iteration's polynomial: steep at 0, within about 0.3 of 1 over most of [0, 1]
STEPS = 5
EPS = 1e-7
HP = dict(lr=4e-4, beta=0.95, weight_decay=0.1)
LOSS_SCALE = 1024.0  # of fp16 gradients


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one small matrix (a router's or an adapter's): all latency
        dict(name="ortho 32x48", op="ortho", layout="one", rows=32, cols=48, grad="bf16", out="bf16"),
        # 24 matrices of odd and ragged sizes, as a model with adapters and heads of many widths has them
        dict(name="ortho 24 ragged", op="ortho", layout="ragged", n=24, most=1500, grad="f16", out="f16"),
        # one large square matrix, an attention output's, from an fp32 momentum
        dict(name="ortho 4096x4096", op="ortho", layout="one", rows=4096, cols=4096, grad="f32", out="bf16"),
        # the four matrices of a d=64 layer: the smallest step
        dict(name="muon layer d64", op="muon", layout="layer", d=64, grad="bf16", copy="bf16", clip=True, nesterov=True),
        # a layer's 32 experts, fp32 gradients (kept from the reduce)
        dict(name="muon 32 experts", op="muon", layout="experts", n=32, rows=1408, cols=512, grad="f32", copy="bf16",
             clip=False, nesterov=True),
        # the four matrices of a d=4096 layer, the largest step here
        dict(name="muon layer d4096", op="muon", layout="layer", d=4096, grad="bf16", copy="bf16", clip=True, nesterov=True),
        # one token's activations: the smallest quantisation
        dict(name="quant 1x4096", op="quant", rows=1, cols=4096, x="bf16", values="bf16", both=False, stochastic=False),
        # gradients of a layer's output for an odd number of tokens, rounded stochastically, for both products of backward
        dict(name="quant 5003x2730 both", op="quant", rows=5003, cols=2730, x="bf16", values="f32", both=True, stochastic=True),
        # fp32 weights into the two forms that forward and backward read
        dict(name="quant 8192x8192 both", op="quant", rows=8192, cols=8192, x="f32", values="bf16", both=True, stochastic=False),
        # one token through a layer, as generation runs it
        dict(name="linear 1 token", op="linear", tokens=1, n=8192, k=4096, x="bf16", out="bf16"),
        # a prompt of an odd length through a layer of odd width
        dict(name="linear 777 tokens", op="linear", tokens=777, n=5000, k=2120, x="f16", out="f16"),
        # forward and backward of a layer over 8192 tokens, the weights' gradient in fp32
        dict(name="train 8192 tokens", op="train", tokens=8192, n=8192, k=4096, x="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("ortho", "muon", "muon", "quant", "linear", "linear", "train"))
    while True:
        case = dict(op=op)
        if op in ("ortho", "muon"):
            case["layout"] = rng.choice(("one", "layer", "experts", "ragged"))
            if case["layout"] == "one":
                case["rows"], case["cols"] = _log(rng, 1, 8192), _log(rng, 1, 8192)
            elif case["layout"] == "layer":
                case["d"] = _log(rng, 16, 4096)
            elif case["layout"] == "experts":
                case["n"], case["rows"], case["cols"] = _log(rng, 2, 64), _log(rng, 32, 2048), _log(rng, 32, 2048)
            else:
                case["n"], case["most"] = _log(rng, 2, 64), _log(rng, 16, 2048)
            case["grad"] = rng.choice(("bf16", "bf16", "f32", "f16"))
            if op == "ortho":
                case["out"] = rng.choice(("bf16", "f16"))
            else:
                case["copy"] = rng.choice(("bf16", "bf16", "none", "f16"))
                case["clip"], case["nesterov"] = rng.random() < 0.5, rng.random() < 0.75
        elif op == "quant":
            case.update(rows=_log(rng, 1, 16384), cols=_log(rng, 1, 16384), x=rng.choice(("bf16", "f32", "f16")),
                        values=rng.choice(("bf16", "f32")), both=rng.random() < 0.5, stochastic=rng.random() < 0.5)
        else:
            case.update(tokens=_log(rng, 1, 8192), n=_log(rng, 16, 16384), k=_log(rng, 16, 16384),
                        x=rng.choice(("bf16", "f16")), out=rng.choice(("bf16", "f16", "f32")))
        w = work(case)
        if w["flops"] <= (1.2e13 if op in ("ortho", "muon") else 1.6e12) and w["bytes"] <= 1.6e9:
            return case


def _shapes(case):
    """(rows, cols) of every matrix of a case."""
    kind = case["layout"]
    if kind == "one":
        return [(case["rows"], case["cols"])]
    if kind == "layer":  # qkv, attention output, the two MLP matrices
        d = case["d"]
        return [(3 * d, d), (d, d), (4 * d, d), (d, 4 * d)]
    if kind == "experts":
        return [(case["rows"], case["cols"])] * case["n"]
    sizes = random.Random(case["n"] * 31 + case["most"])  # ragged: log-uniform sides
    side = lambda: max(1, int(math.exp(sizes.random() * math.log(case["most"]))))  # noqa: E731
    return [(side(), side()) for _ in range(case["n"])]


def _runs(case):
    """(matrices, rows, cols) of every run of matrices of one shape."""
    runs = []
    for r, c in _shapes(case):
        if runs and runs[-1][1:] == [r, c]:
            runs[-1][0] += 1
        else:
            runs.append([1, r, c])
    return runs


def _dense(parts):
    """The runs' matrices back to back in one buffer."""
    return torch.cat([p.reshape(-1) for p in parts])


def _partition(parts):
    """The same with every matrix at a multiple of 32 elements, and zeros between."""
    flat = (p.flatten(1) for p in parts)
    return torch.cat([torch.nn.functional.pad(p, (0, -p.shape[1] % BLOCK)).reshape(-1) for p in flat])


def _bytes(name):
    return 4 if name == "f32" else 0 if name == "none" else 2


def _mx4_bytes(rows, cols):
    """Codes and scales."""
    return rows * -(-cols // BLOCK) * (BLOCK // 2 + 1)


def work(case):
    op = case["op"]
    if op in ("ortho", "muon"):
        shapes = _shapes(case)
        n = sum(r * c for r, c in shapes)
        flops = 0
        for r, c in shapes:  # X X^T and its square are symmetric: half of each
            m, k = min(r, c), max(r, c)
            flops += STEPS * (m * m * k + m * m * m + 2 * m * m * k)
        if op == "ortho":
            return {"bytes": (_bytes(case["grad"]) + _bytes(case["out"])) * n, "flops": flops}
        return {"bytes": (_bytes(case["grad"]) + 16 + _bytes(case["copy"])) * n, "flops": flops + 10 * n}
    if op == "quant":
        r, c = case["rows"], case["cols"]
        n, forms = r * c, 2 if case["both"] else 1
        held = _mx4_bytes(r, c) + (_mx4_bytes(c, r) if case["both"] else 0)
        return {"bytes": _bytes(case["x"]) * n + 2 * held + forms * _bytes(case["values"]) * n, "flops": 4 * forms * n}
    t, n, k = case["tokens"], case["n"], case["k"]
    if op == "linear":
        return {"bytes": _bytes(case["x"]) * t * k + _mx4_bytes(n, k) + _bytes(case["out"]) * t * n, "flops": 2 * t * n * k}
    read = _bytes(case["x"]) * (t * k + t * n) + _mx4_bytes(n, k) + _mx4_bytes(k, n)
    return {"bytes": read + _bytes(case["out"]) * (t * n + t * k) + 4 * n * k, "flops": 6 * t * n * k}


# ---------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    st = dict(case=case, seed=(seed * 2654435761 + 12345) % (1 << 63))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    op = case["op"]
    if op in ("ortho", "muon"):
        scale = LOSS_SCALE if case["grad"] == "f16" else 1.0
        grad, master, momentum = [], [], []
        for count, r, c in _runs(case):
            # noise, and the few directions that most of a batch's gradient lies in; some rows see no token
            seen = (torch.rand(count, r, 1, generator=gen, device=dev) >= 1 / 16).float()
            rank = max(1, min(r, c) // 64)
            common = torch.bmm(normal(count, r, rank), normal(count, rank, c)).mul_(2e-3)
            grad.append(((normal(count, r, c).mul_(1e-3) + common) * seen * scale).to(DTYPE[case["grad"]]))
            if op == "muon":
                master.append(normal(count, r, c).mul_(0.02))
                momentum.append((normal(count, r, c).mul_(2e-4) + common.mul_(0.5)) * seen)
        st["grad"] = _dense(grad)
        if op == "muon":
            st["master"], st["momentum"] = _dense(master), _partition(momentum)
            if case["copy"] != "none":
                st["copy"] = st["master"].to(DTYPE[case["copy"]])
            st["found"] = torch.zeros(1, dtype=torch.int32, device=dev)
            st["coef"] = None
            if case["clip"] or scale != 1.0:  # what unscaling and clipping to a global norm multiply the gradients by
                clip = 0.25 + 0.5 * torch.rand(1, generator=gen, device=dev, dtype=torch.float64) if case["clip"] else 1.0
                st["coef"] = torch.ones(1, dtype=torch.float64, device=dev) * clip / scale
        if own:
            import sharded_flatparameter_pack_amd as fp

            shapes = _shapes(case)
            views = lambda t: [x.view(s) for x, s in zip(t.split([r * c for r, c in shapes]), shapes)]  # noqa: E731
            if op == "ortho":
                st["out"] = torch.empty_like(st["grad"], dtype=DTYPE[case["out"]])
                st["plan"] = fp.Muon(views(st["grad"]), updates=views(st["out"]))
                st["workspace"] = st["plan"].new_workspace()
            else:
                copies = views(st["copy"]) if "copy" in st else None
                st["plan"] = fp.Muon(views(st["grad"]), views(st["master"]), copies)
                st["step"] = st["plan"].stepper(st["momentum"], st["plan"].new_workspace(), **HP, nesterov=case["nesterov"],
                                                found_inf=st["found"], grad_coef=st["coef"])
        return st
    if op == "quant":
        # entries of very different rows and columns, with a few outliers
        r, c = case["rows"], case["cols"]
        x = normal(r, c) * torch.exp(normal(r, 1)) * torch.exp(0.5 * normal(1, c))
        x *= 1 + 15 * (torch.rand(r, c, generator=gen, device=dev) < 1e-3)
        st["x"] = (x * 0.02).to(DTYPE[case["x"]])
        return st
    t, n, k = case["tokens"], case["n"], case["k"]
    st["x"] = (normal(t, k) * torch.exp(0.5 * normal(1, k))).to(DTYPE[case["x"]])
    w = normal(n, k).mul_(0.02)
    if op == "train":
        st["dy"] = normal(t, n).mul_(1e-3).to(DTYPE[case["x"]])
    if own:
        import sharded_flatparameter_pack_amd as fp

        st["w"] = fp.mx4_quantize(w, transposed=op == "train")
    else:
        st["w"] = _values(w, None)
        st["w_t"] = _values(w.t(), None).t() if op == "train" else None
    return st


# ---------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if op == "ortho":
        if own:
            st["plan"].orthogonalize(st["workspace"])
            return st["out"]
        return _dense([_ortho(g.float()) for g in _matrices(st["case"], st["grad"])]).to(DTYPE[st["case"]["out"]])
    if op == "muon":
        if own:
            st["step"]()
        else:
            _muon(st)
        return {k: st[k] for k in ("master", "momentum", "copy") if k in st}
    st["seed"] += 1
    if op == "quant":
        return _own_quant(st) if own else _quant(st)
    if op == "linear":
        return _own_linear(st) if own else _linear(st)
    return _own_train(st) if own else _train(st)


def _matrices(case, flat, padded=False):
    """A [matrices, rows, cols] view of every run."""
    got, at = [], 0
    for count, r, c in _runs(case):
        room = r * c + (-(r * c) % BLOCK if padded else 0)
        got.append(flat[at:at + count * room].view(count, room)[:, :r * c].view(count, r, c))
        at += count * room
    return got


def _ortho(u):
    x = u / (u.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    turned = x.shape[1] > x.shape[2]
    if turned:
        x = x.transpose(1, 2)
    a, b, c = COEFS
    for _ in range(STEPS):
        g = x @ x.transpose(1, 2)
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.transpose(1, 2) if turned else x


def _muon(st):
    case, beta = st["case"], HP["beta"]
    kept = st["found"] == 0
    master, momentum = [], []
    runs = (_matrices(case, st["grad"]), _matrices(case, st["master"]), _matrices(case, st["momentum"], True))
    for g, w, m in zip(*runs):
        g = g.float()
        if st["coef"] is not None:
            g = g * st["coef"].float()
        m = beta * m + (1 - beta) * g
        u = (1 - beta) * g + beta * m if case["nesterov"] else m
        rate = HP["lr"] * 0.2 * math.sqrt(max(g.shape[1:]))
        master.append(w * (1 - HP["lr"] * HP["weight_decay"]) - rate * _ortho(u))
        momentum.append(m)
    st["master"] = torch.where(kept, _dense(master), st["master"])
    st["momentum"] = torch.where(kept, _partition(momentum), st["momentum"])
    if "copy" in st:
        st["copy"] = st["master"].to(st["copy"].dtype)


# MXFP4 in the plain form: everything up to the rounding is exact in 32 bits, the rounding's own sum is taken in 64.
def _power(e):
    """2^e of whole numbers -149 <= e <= 127, in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _values(x, dither):
    """What MXFP4 of the rows of x stands for, in fp32: rounded to nearest even, or stochastically with 16 bits of dither.

    The scale puts the block's largest value on the grid's top, 4 to 6, after rounding to e2m1's precision (stochastic: so
    that it is at most 6 before); a block that is not finite, or whose scale passes fp32's range, reads as NaN.
    """
    r, c = x.shape
    pad = -c % BLOCK
    y = torch.nn.functional.pad(x.float(), (0, pad)).reshape(-1, BLOCK)
    bits = y.view(torch.int32) & 0x7FFFFFFF
    top = (bits.amax(1).long() + ((1 << 21) if dither is None else (1 << 22) - 1)) >> 23
    byte = (top - 2).clamp(min=0)
    scale = _power(byte - 127)[:, None]
    a = y.abs().double() / scale
    q = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    if dither is None:
        v = torch.round(a / q)
    else:
        v = torch.floor(a / q + torch.nn.functional.pad(dither, (0, pad)).reshape(-1, BLOCK).double() / 65536)
    v = torch.copysign(v * q * scale, y.double())
    v = torch.where((top >= 255)[:, None], torch.full_like(v, math.nan), v)
    return v.float().view(r, c + pad)[:, :c]


def _key(seed):
    z = (seed * 0x9E3779B97F4A7C15) % (1 << 64)
    z ^= z >> 32
    z = (z * 0xD6E8FEB86659FD93) % (1 << 64)
    return (z ^ (z >> 32)) & MASK


def _dither(rows, cols, seed, device):
    """16 bits for the rows' form and 16 for the columns', of every element."""
    x = ((torch.arange(rows * cols, device=device).view(rows, cols) * 0x9E3779B1) & MASK) ^ _key(seed)
    x ^= x >> 16
    x = (x * 0x6A09E667) & MASK
    x ^= x >> 15
    x = (x * 0xBB67AE85) & MASK
    return x >> 16, x & 0xFFFF


def _quant(st):
    case, x = st["case"], st["x"]
    d, dt = _dither(*x.shape, st["seed"], x.device) if case["stochastic"] else (None, None)
    got = {"values": _values(x, d).to(DTYPE[case["values"]])}
    if case["both"]:
        got["values_t"] = _values(x.t(), None if dt is None else dt.t()).to(DTYPE[case["values"]])
    return got


def _own_quant(st):
    import sharded_flatparameter_pack_amd as fp

    case, x = st["case"], st["x"]
    held = fp.mx4_quantize(x, transposed=case["both"], seed=st["seed"] if case["stochastic"] else None)
    got = {"values": fp.mx4_dequantize(held[0], held[1], x.shape[1], dtype=DTYPE[case["values"]])}
    if case["both"]:
        got["values_t"] = fp.mx4_dequantize(held[2], held[3], x.shape[0], dtype=DTYPE[case["values"]])
    return got


def _linear(st):
    return (_values(st["x"], None) @ st["w"].t()).to(DTYPE[st["case"]["out"]])


def _own_linear(st):
    import sharded_flatparameter_pack_amd as fp

    return fp.mx4_matmul(fp.mx4_quantize(st["x"]), st["w"], dtype=DTYPE[st["case"]["out"]])


def _train(st):
    x, dy, out = st["x"], st["dy"], DTYPE[st["case"]["out"]]
    d, dt = _dither(*dy.shape, st["seed"], dy.device)
    return {"y": (_values(x, None) @ st["w"].t()).to(out),
            "dx": (_values(dy, d) @ st["w_t"]).to(out),
            "dw": _values(dy.t(), dt.t()) @ _values(x.t(), None).t()}


def _own_train(st):
    import sharded_flatparameter_pack_amd as fp

    out = DTYPE[st["case"]["out"]]
    x = fp.mx4_quantize(st["x"], transposed=True)
    y = fp.mx4_matmul(x[:2], st["w"][:2], dtype=out)
    dy = fp.mx4_quantize(st["dy"], transposed=True, seed=st["seed"])
    return {"y": y, "dx": fp.mx4_matmul(dy[:2], st["w"][2:], dtype=out),
            "dw": fp.mx4_matmul(dy[2:], x[2:], dtype=torch.float32)}


# ---------------------------------------------------------------------- in 64 bits, from the definition
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "ortho":
        return torch.cat([_polar(g.double()).reshape(-1) for run in _matrices(case, st["grad"]) for g in run])
    if op == "muon":
        at, new = 0, {"master": [], "momentum": torch.zeros_like(st["momentum"], dtype=torch.float64)}
        place = 0
        for r, c in _shapes(case):
            g, w = (st[k][at:at + r * c].view(r, c).double() for k in ("grad", "master"))
            m = st["momentum"][place:place + r * c].view(r, c).double()
            if st["coef"] is not None:
                g = g * st["coef"]
            m = m + (1 - HP["beta"]) * (g - m)
            u = g + HP["beta"] * (m - g) if case["nesterov"] else m
            step = HP["weight_decay"] * w + 0.2 * max(r, c) ** 0.5 * _polar(u)
            new["master"].append((w - HP["lr"] * step).reshape(-1))
            new["momentum"][place:place + r * c] = m.reshape(-1)
            at, place = at + r * c, place + -(-r * c // BLOCK) * BLOCK
        new["master"] = torch.cat(new["master"])
        if "copy" in st:
            new["copy"] = new["master"]
        return new
    s = st["seed"] + 1
    if op == "quant":
        x = st["x"].double()
        d, dt = _dither(*x.shape, s, x.device) if case["stochastic"] else (None, None)
        got = {"values": _grid(x, d)}
        if case["both"]:
            got["values_t"] = _grid(x.t(), None if dt is None else dt.t())
        return got
    x, w = st["x"].double(), st["w"].double()
    y = _grid(x, None) @ w.t()
    if op == "linear":
        return y
    dy = st["dy"].double()
    d, dt = _dither(*dy.shape, s, dy.device)
    return {"y": y, "dx": _grid(dy, d) @ st["w_t"].double(), "dw": _grid(dy.t(), dt.t()) @ _grid(x.t(), None).t()}


def _polar(u):
    """The iteration on the smaller side's products: X <- X (a I + b X^T X + c (X^T X)^2) for a tall X."""
    x = u if u.shape[0] >= u.shape[1] else u.t()
    x = x / (torch.linalg.vector_norm(x) + EPS)
    for _ in range(STEPS):
        g = x.t() @ x
        p = COEFS[1] * g + COEFS[2] * torch.mm(g, g)
        p.diagonal().add_(COEFS[0])
        x = x @ p
    return x if u.shape[0] >= u.shape[1] else x.t()


LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _grid(x, u):
    """MXFP4 on the values: the level at or below each, and the next one where the distance (or the dither) says so."""
    r, c = x.shape
    out = torch.empty(r, c, dtype=torch.float64, device=x.device)
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    rows = max(1, (1 << 24) // max(1, c))
    for at in range(0, r, rows):
        a = x[at:at + rows]
        a = torch.nn.functional.pad(a, (0, -c % BLOCK)).reshape(-1, BLOCK)
        mantissa, exponent = torch.frexp(a.abs().amax(1))
        up = mantissa >= 0.875 if u is None else mantissa > 0.75
        k = (exponent - 3 + up.int()).clamp(min=-127)
        k = torch.where(mantissa == 0, torch.full_like(k, -127), k)
        scale = (k.long() + 1023).bitwise_left_shift(52).view(torch.float64)[:, None]
        y = a.abs() / scale
        low = (torch.searchsorted(levels, y, right=True) - 1).clamp(max=6)
        step = levels[low + 1] - levels[low]
        share = (y - levels[low]) / step
        if u is None:
            more = (share > 0.5) | ((share == 0.5) & (low % 2 == 1))
        else:
            d = torch.nn.functional.pad(u[at:at + rows], (0, -c % BLOCK)).reshape(-1, BLOCK).double()
            more = share + d / 65536 >= 1
        v = torch.copysign(levels[low + more.long()] * scale, a)
        out[at:at + rows] = v.reshape(-1, c + -c % BLOCK)[:, :c]
    return out
