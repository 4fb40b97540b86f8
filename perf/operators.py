"""The optimizer step over many separate tensors, as measured work.

Operators: AdamW over many tensors with fp32 moments ("adamw") and with MXFP8 moments ("adamw8"), the sum of
squares and overflow check of many gradients ("grad_norm"), and the conversion of moments between fp32 and MXFP8
("quantize", "dequantize").

A rank's tensors are views of one dense buffer each for the gradients, the fp32 weights and their low-precision
copies, as the dim-0 layout of a parameter group has them; the moments sit in one partition where every tensor starts
at a multiple of 32 elements.  MXFP8 is e4m3 codes with one power-of-two scale (e8m0) per 32 consecutive elements.
"""

import math
import random

import torch

own = False

MASK = 0xFFFFFFFF
BLOCK = 32
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)
WEIGHT_DECAY = (0.01, 0.0)  # matrices, and the tensors that are not decayed (biases, norm weights)
GRAD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
COPY = {"none": None, "bf16": torch.bfloat16, "f16": torch.float16}
LOSS_SCALE = 1024.0  # of fp16 gradients


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # three (4, 2) weights: the smallest group, all latency
        dict(name="step of three 4x2", op="adamw", layout="three", grad="f32", copy="none", clip=False),
        # one rank of eight: its rows of a d=1024 Transformer layer, clipped
        dict(name="step layer d1024", op="adamw", layout="layer", d=1024, world=8, grad="bf16", copy="bf16", clip=True),
        # one rank of sixteen: a 611M model in 25 MiB buckets, fp32 gradients (kept from the reduce)
        dict(name="step 611M buckets", op="adamw", layout="buckets", total=611_000_000, world=16, grad="f32",
             copy="bf16", clip=True),
        # three (4, 2) weights with 8-bit moments
        dict(name="step8 of three 4x2", op="adamw8", layout="three", grad="bf16", copy="bf16", clip=False),
        # the d=1024 layer's slice with 8-bit moments
        dict(name="step8 layer d1024", op="adamw8", layout="layer", d=1024, world=8, grad="bf16", copy="bf16", clip=True),
        # one rank of 64: pieces of 10 000 ragged tensors at any alignment, fp16 gradients under a loss scale
        dict(name="step8 10k ragged", op="adamw8", layout="ragged", n=10_000, largest=4_194_304, world=64, grad="f16",
             copy="f16", clip=False),
        # one rank of eight: its rows of a d=12288 layer, the largest step here
        dict(name="step8 layer d12288", op="adamw8", layout="layer", d=12288, world=8, grad="bf16", copy="bf16", clip=True),
        # the norm of three tiny gradients
        dict(name="norm of three 4x2", op="grad_norm", layout="three", grad="f32"),
        # the norm of 10 000 ragged pieces
        dict(name="norm 10k ragged", op="grad_norm", layout="ragged", n=10_000, largest=4_194_304, world=64, grad="bf16"),
        # the norm before clipping the d=12288 layer's slice
        dict(name="norm layer d12288", op="grad_norm", layout="layer", d=12288, world=8, grad="bf16"),
        # a layer's first moments into 8 bits (a checkpoint in fp32 loaded into an 8-bit run)
        dict(name="quantize layer d1024", op="quantize", layout="layer", d=1024, world=8, root=False),
        # a 611M model's second moments out of 8 bits (a checkpoint written in fp32)
        dict(name="dequantize 611M", op="dequantize", layout="buckets", total=611_000_000, world=16, root=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("adamw", "adamw8", "adamw8", "grad_norm", "quantize", "dequantize"))
    most = 100_000_000 if op == "adamw" else 200_000_000
    while True:
        case = dict(op=op, layout=rng.choice(("layer", "buckets", "ragged")), world=_log(rng, 1, 64))
        if case["layout"] == "layer":
            case["d"] = _log(rng, 16, 12288)
        elif case["layout"] == "buckets":
            case["total"] = _log(rng, 1, 700_000_000)
        else:
            case["n"], case["largest"] = _log(rng, 1, 10_000), _log(rng, 1, 4_194_304)
        if sum(n for n, _ in _tensors(case)) <= most:
            break
    if op in ("quantize", "dequantize"):
        case["root"] = rng.random() < 0.5
        return case
    case["grad"] = rng.choice(("bf16", "bf16", "f32", "f16"))
    if op != "grad_norm":
        case["copy"] = rng.choice(("bf16", "bf16", "none", "f16"))
        case["clip"] = rng.random() < 0.5
    return case


def _tensors(case):
    """(elements, parameter group) of every tensor that the rank holds."""
    kind = case["layout"]
    if kind == "three":
        return [(8, 0)] * 3
    if kind == "layer":  # qkv, attention output, the two MLP matrices, their biases, two LayerNorms: first rows of each
        d, world = case["d"], case["world"]
        shapes = [(3 * d, d), (3 * d, 1), (d, d), (d, 1), (4 * d, d), (4 * d, 1), (d, 4 * d), (d, 1)] + [(d, 1)] * 4
        return [(-(-rows // world) * cols, int(cols == 1)) for rows, cols in shapes]
    if kind == "buckets":  # 25 MiB of bf16 each
        bucket, left, got = 13_107_200, case["total"], []
        while left > 0:
            got.append((-(-min(bucket, left) // case["world"]), 0))
            left -= bucket
        return got
    sizes = random.Random(case["n"] * 31 + case["largest"])  # ragged: log-uniform sizes
    top = math.log(case["largest"])
    return [(-(-max(1, int(math.exp(sizes.random() * top))) // case["world"]), int(i % 3 == 2)) for i in range(case["n"])]


def _room(n):
    return -(-n // BLOCK) * BLOCK


def work(case):
    sizes = [n for n, _ in _tensors(case)]
    n, blocks = sum(sizes), sum(_room(x) // BLOCK for x in sizes)
    op = case["op"]
    if op in ("quantize", "dequantize"):
        return {"bytes": 5 * n + blocks, "flops": 4 * n}
    g = 4 if case["grad"] == "f32" else 2
    if op == "grad_norm":
        return {"bytes": g * n, "flops": 2 * n}
    weights = g + 8 + (0 if case["copy"] == "none" else 2)
    return {"bytes": (weights + 16) * n if op == "adamw" else (weights + 4) * n + 4 * blocks, "flops": 20 * n}


# ---------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    tensors = _tensors(case)
    sizes = [n for n, _ in tensors]
    n, room = sum(sizes), sum(_room(x) for x in sizes)
    st = dict(case=case, n=n, room=room, t=100, seed=(seed * 2654435761 + 12345) % (1 << 63))

    def normal(count, sigma):
        return torch.randn(count, generator=gen, device=dev).mul_(sigma)

    live = torch.rand(-(-n // 64), generator=gen, device=dev) >= 1 / 16  # the others: rows that no token has reached
    live = live.repeat_interleave(64)[:n]

    # where each dense element sits in the partition (None: at the same place)
    st["at"] = None
    if room != n:
        gap = torch.tensor([_room(x) - x for x in sizes], device=dev)
        gap = gap.cumsum(0) - gap
        st["at"] = torch.arange(n, device=dev) + gap.repeat_interleave(torch.tensor(sizes, device=dev), output_size=n)

    def placed(x):
        if st["at"] is None:
            return x
        p = torch.zeros(room, device=dev)
        p[st["at"]] = x
        return p

    def first():
        return normal(n, 1e-4) * live

    def second():
        return normal(n, 1e-3).square_() * live

    op = case["op"]
    if op in ("quantize", "dequantize"):
        x = placed(second() if case["root"] else first())
        if op == "quantize":
            st["x"] = x
            st["codes"] = torch.zeros(room, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
            st["scales"] = torch.zeros(room // BLOCK, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu)
        else:
            st["codes"], st["scales"] = _quantized(x.double().sqrt().float() if case["root"] else x, None, case["root"])
            st["x"] = torch.zeros(room, device=dev)
        return st

    scale = LOSS_SCALE if case["grad"] == "f16" else 1.0
    grad = (normal(n, 1e-3) * live * scale).to(GRAD[case["grad"]])
    st["grad"] = grad
    dense = [grad]
    if op == "grad_norm":
        st["found"] = torch.zeros(1, dtype=torch.int32, device=dev)
        st["sq"] = torch.zeros(1, dtype=torch.float64, device=dev)
    else:
        st["master"] = normal(n, 0.02)
        dense.append(st["master"])
        if case["copy"] != "none":
            st["copy"] = st["master"].to(COPY[case["copy"]])
            dense.append(st["copy"])
        group = torch.tensor([k for _, k in tensors], device=dev)
        decay = torch.tensor([1.0 - HP["lr"] * w for w in WEIGHT_DECAY], dtype=torch.float64, device=dev)
        st["decay"] = decay[group].repeat_interleave(torch.tensor(sizes, device=dev), output_size=n).float()
        st["found"] = torch.zeros(1, dtype=torch.int32, device=dev)
        st["coef"] = None
        if case["clip"] or scale != 1.0:  # what unscaling and clipping to a global norm multiply the gradients by
            clip = 0.25 + 0.5 * torch.rand(1, generator=gen, device=dev, dtype=torch.float64) if case["clip"] else 1.0
            st["coef"] = torch.ones(1, dtype=torch.float64, device=dev) * clip / scale
        if op == "adamw":
            st["moments"] = [placed(first()), placed(second())]
        else:
            st["moments"] = [*_quantized(placed(first()), None, False), *_quantized(placed(second()).sqrt(), None, True)]

    if own:
        import sharded_flatparameter_pack_amd as fp

        views = [d.split(sizes) for d in dense]
        if op == "grad_norm":
            st["plan"] = fp.Params(views[0])
            st["workspace"] = st["plan"].new_workspace()
        else:
            st["plan"] = fp.Params(views[0], views[1], views[2] if len(views) > 2 else None, groups=[k for _, k in tensors])
            st["step"] = st["plan"].stepper(st["moments"], **HP, weight_decay=WEIGHT_DECAY, found_inf=st["found"],
                                            grad_coef=st["coef"])
    return st


# ---------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if op == "grad_norm":
        return _own_norm(st) if own else _norm(st)
    if op == "quantize":
        if own:
            import sharded_flatparameter_pack_amd as fp
            fp.mx8_quantize(st["x"], st["codes"], st["scales"], root=st["case"]["root"])
            return {"codes": st["codes"], "scales": st["scales"]}
        x = st["x"].double().sqrt().float() if st["case"]["root"] else st["x"]
        codes, scales = _quantized(x, None, st["case"]["root"])
        return {"codes": codes, "scales": scales}
    if op == "dequantize":
        if own:
            import sharded_flatparameter_pack_amd as fp
            return fp.mx8_dequantize(st["codes"], st["scales"], st["x"], root=st["case"]["root"])
        x = _values(st["codes"], st["scales"])
        return x.square().float() if st["case"]["root"] else x.float()
    st["t"] += 1
    st["seed"] += 1
    if own:
        if op == "adamw":
            st["step"](st["t"])
        else:
            st["step"](st["t"], seed=st["seed"])
    elif op == "adamw":
        _adamw(st)
    else:
        _adamw8(st)
    names = ("exp_avg", "exp_avg_sq") if op == "adamw" else ("exp_avg", "exp_avg_scale", "root", "root_scale")
    got = dict(zip(names, st["moments"]), master=st["master"])
    if "copy" in st:
        got["copy"] = st["copy"]
    return got


def _own_norm(st):
    st["found"].zero_()
    st["plan"].grad_norm(st["sq"], st["workspace"], found_inf=st["found"])
    return {"found_inf": st["found"], "sq_norm": st["sq"]}


def _norm(st):
    # in 64 bits: a sum of 10^8 squares loses what matters in 32
    g = st["grad"]
    return {"found_inf": (~torch.isfinite(g)).any().to(torch.int32).reshape(1), "sq_norm": g.double().square().sum().reshape(1)}


def _taken(st, p):
    return p if st["at"] is None else p[st["at"]]


def _put(st, p, x):
    if st["at"] is None:
        return x
    p = p.clone()
    p[st["at"]] = x
    return p


def _update(st, m, v, kept):
    """The weights and their copy from the dense moments; an overflow leaves the weights."""
    t = st["t"]
    root = (v / (1 - HP["beta2"] ** t)).sqrt()
    theta = st["master"] * st["decay"] - HP["lr"] / (1 - HP["beta1"] ** t) * m / (root + HP["eps"])
    st["master"] = torch.where(kept, theta.float(), st["master"])
    if "copy" in st:
        st["copy"] = st["master"].to(st["copy"].dtype)


def _adamw(st):
    kept = st["found"] == 0
    g = st["grad"].float()
    if st["coef"] is not None:
        g = g * st["coef"].float()
    m0, v0 = (_taken(st, p) for p in st["moments"])
    m = HP["beta1"] * m0 + (1 - HP["beta1"]) * g
    v = HP["beta2"] * v0 + (1 - HP["beta2"]) * g * g
    _update(st, m, v, kept)
    st["moments"] = [_put(st, p, torch.where(kept, x, x0)) for p, x, x0 in zip(st["moments"], (m, v), (m0, v0))]


def _power(e):
    """2^e of whole numbers -1022 <= e <= 1023, in 64 bits."""
    return ((e + 1023) << 52).view(torch.float64)


def _values(codes, scales):
    """What MXFP8 stands for, in 64 bits."""
    return (codes.view(-1, BLOCK).double() * scales.double()[:, None]).reshape(-1)


def _quantized(x, dither, root):
    """MXFP8 of an fp32 partition: rounded stochastically with 16 bits of dither per element, or to nearest even.

    The scale puts the block's largest value, rounded to e4m3's precision, at 2^7; a block that is not finite gets the
    scale NaN.  A root that is not zero does not round to zero.  Codes are next to borders: whole-number work.
    """
    bits = x.view(torch.int32).long() & MASK
    size = bits & 0x7FFFFFFF
    top = (size.view(-1, BLOCK).amax(1) + (1 << 19)) >> 23
    byte = torch.where(top >= 255, torch.full_like(top, 255), (top - 7).clamp(min=0))
    y = x.abs().double().view(-1, BLOCK) * _power(7 - torch.where(top >= 255, torch.zeros_like(byte), byte))[:, None]
    y = y.float().view(-1).view(torch.int32).long()  # fp32 bits of |x| / scale * 2^-120: e4m3's exponent bias is 7
    if dither is None:
        code = (y + 0x7FFFF + ((y >> 20) & 1)) >> 20
    else:
        code = (y + (dither << 4)) >> 20
    if root:
        code = torch.where((code == 0) & (size > 0), torch.ones_like(code), code)
    else:
        code = code | ((bits >> 31) << 7)
    code = torch.where((byte == 255).repeat_interleave(BLOCK), torch.zeros_like(code), code)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), byte.to(torch.uint8).view(torch.float8_e8m0fnu)


def _key(seed):
    z = (seed * 0x9E3779B97F4A7C15) % (1 << 64)
    z ^= z >> 32
    z = (z * 0xD6E8FEB86659FD93) % (1 << 64)
    return (z ^ (z >> 32)) & MASK


def _dither(room, seed, device):
    """16 bits for the first moment and 16 for the root, of every element of the partition."""
    x = ((torch.arange(room, device=device) * 0x9E3779B1) & MASK) ^ _key(seed)
    x ^= x >> 16
    x = (x * 0x6A09E667) & MASK
    x ^= x >> 15
    x = (x * 0xBB67AE85) & MASK
    return x >> 16, x & 0xFFFF


def _adamw8(st):
    # the moments in 64 bits: where they fall next to a border of the rounding, 32 would give another code
    kept = st["found"] == 0
    g = st["grad"].double()
    if st["coef"] is not None:
        g = g * st["coef"]
    cm, sm, cr, sr = st["moments"]
    m = HP["beta1"] * _taken(st, _values(cm, sm)) + (1 - HP["beta1"]) * g
    v = HP["beta2"] * _taken(st, _values(cr, sr)).square() + (1 - HP["beta2"]) * g * g
    _update(st, m.float(), v, kept)
    zero = torch.zeros(st["room"], device=g.device)
    dm, dr = _dither(st["room"], st["seed"], g.device)
    new = [*_quantized(_put(st, zero, m.float()), dm, False), *_quantized(_put(st, zero, v.sqrt().float()), dr, True)]
    st["moments"] = [torch.where(kept, x.view(torch.uint8), x0.view(torch.uint8)).view(x.dtype)
                     for x, x0 in zip(new, st["moments"])]


# ---------------------------------------------------------------------- in 64 bits, from the definition
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "grad_norm":
        parts = [x.double() for x in st["grad"].split(1 << 20)]
        bad = any(bool(torch.isnan(p).any() | torch.isinf(p).any()) for p in parts)
        return {"found_inf": int(bad), "sq_norm": torch.tensor([math.fsum(float(p @ p) for p in parts)], dtype=torch.float64)}
    if op == "quantize":
        codes, scales = _grid(st["x"].double().sqrt().float() if case["root"] else st["x"], None, case["root"])
        return {"codes": codes, "scales": scales}
    if op == "dequantize":
        x = st["codes"].double() * st["scales"].double().repeat_interleave(BLOCK)
        return x * x if case["root"] else x
    t, seed2 = st["t"] + 1, st["seed"] + 1
    g = st["grad"].double() * (1.0 if st["coef"] is None else st["coef"])
    if op == "adamw":
        m0, v0 = (p.double() for p in st["moments"])
    else:
        cm, sm, cr, sr = st["moments"]
        m0 = cm.double() * sm.double().repeat_interleave(BLOCK)
        v0 = (cr.double() * sr.double().repeat_interleave(BLOCK)) ** 2
    at = st["at"] if st["at"] is not None else slice(None)
    m, v = m0.clone(), v0.clone()
    m[at] = HP["beta1"] * m0[at] + (1 - HP["beta1"]) * g
    v[at] = HP["beta2"] * v0[at] + (1 - HP["beta2"]) * g ** 2
    bias1, bias2 = 1 - HP["beta1"] ** t, 1 - HP["beta2"] ** t
    step = HP["lr"] * (m[at] / bias1) / (torch.sqrt(v[at] / bias2) + HP["eps"])
    group = torch.tensor([k for _, k in _tensors(case)], device=g.device)
    decay = torch.tensor([1.0 - HP["lr"] * w for w in WEIGHT_DECAY], dtype=torch.float64, device=g.device)[group]
    decay = decay.repeat_interleave(torch.tensor([k for k, _ in _tensors(case)], device=g.device))
    theta = st["master"].double() * decay - step
    got = {"master": theta}
    if case["copy"] != "none":
        got["copy"] = theta
    if op == "adamw":
        got.update(exp_avg=m, exp_avg_sq=v)
    else:
        dm, dr = _dither(st["room"], seed2, g.device)
        got["exp_avg"], got["exp_avg_scale"] = _grid(m.float(), dm / 65536, False)
        got["root"], got["root_scale"] = _grid(v.sqrt().float(), dr / 65536, True)
    return got


def _grid(x, u, root):
    """MXFP8 on the values: each e4m3 interval's width q, and the value at it down (with u in [0, 1) added) or nearest."""
    a = x.double().abs().view(-1, BLOCK)
    big = a.amax(1)
    mantissa, exponent = torch.frexp(big)
    k = torch.where(big > 0, exponent - 1 + (mantissa >= 31 / 32).int() - 7, torch.full_like(exponent, -127)).clamp(min=-127)
    y = torch.ldexp(a, -k[:, None]).reshape(-1)
    q = torch.ldexp(torch.ones_like(y), (torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    z = torch.round(y / q) if u is None else torch.floor(y / q + u)
    z = z * q
    if root:
        z = torch.where((y > 0) & (z == 0), torch.full_like(z, 2.0 ** -9), z)
    return torch.copysign(z, x.double()), torch.ldexp(torch.ones_like(big), k)
