"""The step over many separate tensors and MXFP8, in numpy and 64 bits.

Tolerances.  A value that the kernels compute in fp64 and round once to fp32
is off by at most half a step, 2^-24 of it (2^-150 below the normal range),
plus the fp64 operations' own error, a few 2^-53 of the terms: `near` takes
2^-24 of the value and 2^-48 of the largest term.  A code may differ from the
reference's only where the value is that close to a border between two codes,
so a code is right if it is the code of the value moved by a relative 2^-40
either way or of the value itself.

With 8-bit moments a weight's change is evaluated in fp32 and added once.  Its
roundings, relative to the change: of r', the root's bias correction, eps, the
denominator, m', their quotient, the step size, lr * weight_decay, its product
and the sum, each at most 2^-24, and of the hardware's reciprocal, at most
2^-23: 12 * 2^-24 in all, below 2^-20.  `near` takes 2^-20 of `change` for it.
"""

import numpy as np

BLOCK = 32
U32, U64 = np.uint32, np.uint64


def decode(codes, scales):
    """fp64 values of e4m3 codes (uint8) and e8m0 scales, whole blocks or a last part."""
    c = codes.astype(np.int64)
    e, f = (c >> 3) & 15, c & 7
    x = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e.astype(float) - 10))
    x = np.where(c & 127 == 127, np.nan, x) * np.where(c & 128, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(float) - 127))
    return x * np.repeat(s, BLOCK)[:x.size]


def blocks(x):
    room = -(-x.size // BLOCK) * BLOCK
    return np.concatenate([x, np.zeros(room - x.size, x.dtype)]).reshape(-1, BLOCK)


def scale_bytes(x):
    """Scale byte of every block of fp32 values."""
    x = x.astype(np.float32)
    top = (blocks(x.view(U32) & U32(0x7FFFFFFF)).max(1).astype(np.int64) + (1 << 19)) >> 23
    return np.where(top >= 255, 255, np.maximum(top - 7, 0)).astype(np.uint8)


def encode(x, scales, dither=None, root=False):
    """Codes of fp32 values under given scale bytes: q the width of e4m3's
    interval at y = |x| / scale, q floor(y / q + dither / 2^16), or y rounded to
    the nearest multiple of q (ties to even)."""
    x = x.astype(np.float32)
    b = np.repeat(scales, BLOCK)[:x.size].astype(np.int64)
    y = np.where(b == 255, 0.0, np.ldexp(np.abs(np.where(b == 255, 0, x)).astype(np.float64), 127 - b))
    q = np.exp2(np.maximum(np.frexp(y)[1] - 1, -6).astype(float) - 3)
    v = q * (np.rint(y / q) if dither is None else np.floor(y / q + dither / 65536.0))
    e = np.where(v > 0, np.frexp(v)[1] - 1, -7)
    code = np.where(e < -6, v * 512, (e + 7) * 8 + np.ldexp(v, 3 - e) - 8).astype(np.int64)
    if root:
        code = np.where((code == 0) & (y > 0), 1, code)
    else:
        code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(b == 255, 0, code).astype(np.uint8)


def dither(index, seed):
    """(first moment's, root's) 16 bits for partition elements `index`."""
    z = (int(seed) * 0x9E3779B97F4A7C15) % (1 << 64)
    z ^= z >> 32
    z = (z * 0xD6E8FEB86659FD93) % (1 << 64)
    key = (z ^ (z >> 32)) & 0xFFFFFFFF
    x = ((index.astype(np.int64) & 0xFFFFFFFF).astype(U32) * U32(0x9E3779B1)) ^ U32(key)
    x = x ^ (x >> U32(16))
    x = x * U32(0x6A09E667)
    x = x ^ (x >> U32(15))
    x = x * U32(0xBB67AE85)
    return x >> U32(16), x & U32(0xFFFF)


def adamw(g, th, m, v, hp, t, coef=1.0):
    """fp64 (weights, first moment, second moment) of one step, the size of the
    terms that the weights are the sum of, and that of their change."""
    g = g.astype(np.float64) * coef
    m = hp["beta1"] * m.astype(np.float64) + (1 - hp["beta1"]) * g
    v = hp["beta2"] * v.astype(np.float64) + (1 - hp["beta2"]) * g * g
    step = hp["lr"] * (m / (1 - hp["beta1"] ** t)) / (np.sqrt(v / (1 - hp["beta2"] ** t)) + hp["eps"])
    th = th.astype(np.float64)
    decay = hp["lr"] * hp["weight_decay"] * th
    return th - decay - step, m, v, np.abs(th) + np.abs(step), np.abs(decay) + np.abs(step)


def near(got, want, terms=None, what="", change=0.0):
    """`got` (fp32) is the fp64 `want` rounded once (see above)."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    terms = np.abs(want) if terms is None else terms
    fine = np.isfinite(want) & (np.abs(want) < 3.4e38)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: other NaNs"
    err = np.abs(got[fine] - want[fine])
    tol = 2.0 ** -24 * np.abs(want[fine]) + 2.0 ** -48 * terms[fine] + 2.0 ** -150
    tol = tol + 2.0 ** -20 * np.broadcast_to(change, want.shape)[fine]
    if (err > tol).any():
        i = int(np.argmax(err - tol))
        raise AssertionError(f"{what}: {int((err > tol).sum())} of {err.size} off; got {got[fine][i]!r} "
                             f"want {want[fine][i]!r}, over by {err[i] / tol[i]:.3g}")


def check_mx8(codes, scales, value, seed_dither=None, root=False, what=""):
    """Codes and scale bytes of one tensor are those of the fp64 `value`."""
    with np.errstate(all="ignore"):
        near_by = [(value * f).astype(np.float32) for f in (1.0, 1 - 2.0 ** -40, 1 + 2.0 ** -40)]
    tops = [scale_bytes(x) for x in near_by]
    ok = np.zeros(scales.size, bool)
    for s in tops:
        ok |= scales == s
    assert ok.all(), f"{what}: {int((~ok).sum())} scale bytes of {ok.size}, first block {int(np.argmin(ok))}"
    ok = np.zeros(codes.size, bool)
    for x in near_by:
        ok |= codes == encode(x, scales, seed_dither, root)
    if not ok.all():
        i = int(np.argmin(ok))
        raise AssertionError(f"{what}: {int((~ok).sum())} codes of {ok.size}, first {i}: got {codes[i]} for {value[i]!r} "
                             f"under scale {scales[i // BLOCK]}, want {encode(near_by[0], scales, seed_dither, root)[i]}")
