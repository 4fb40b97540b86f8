"""Plain references of the operators on matrices, in 64 bits: MXFP4 from its
definition (numpy, value by value), the Newton-Schulz iteration and the step
that takes it (torch on the CPU)."""

import numpy as np
import torch

BLOCK, PAD = 32, 256
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
COEFS = (3.4445, -4.7750, 2.0315)
M32 = 0xFFFFFFFF


def padded(n):
    return -(-n // PAD) * PAD


def key_of(seed):
    z = (seed * 0x9E3779B97F4A7C15) % (1 << 64)
    z ^= z >> 32
    z = (z * 0xD6E8FEB86659FD93) % (1 << 64)
    return (z ^ (z >> 32)) & M32


def hashes(index, seed):
    """The hash of elements' indices: 32 bits."""
    x = (np.asarray(index).astype(np.uint64) * np.uint64(0x9E3779B1) & np.uint64(M32)) ^ np.uint64(key_of(seed))
    x ^= x >> np.uint64(16)
    x = x * np.uint64(0x6A09E667) & np.uint64(M32)
    x ^= x >> np.uint64(15)
    return x * np.uint64(0xBB67AE85) & np.uint64(M32)


def dither(rows, cols, seed):
    return hashes(np.arange(rows * cols, dtype=np.uint64), seed).reshape(rows, cols)


def quantize(x, d=None):
    """(codes [rows, P / 2], scales [rows, P / 32]) of fp32 values along their rows; d: 16 bits of dither per element, or
    None for rounding to nearest even."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    P = padded(cols)
    nib = np.zeros((rows, P), np.uint8)
    scales = np.zeros((rows, P // BLOCK), np.uint8)
    for b in range(-(-cols // BLOCK)):
        at = slice(b * BLOCK, min(cols, (b + 1) * BLOCK))
        v = x[:, at]
        bits = (np.ascontiguousarray(v).view(np.uint32) & 0x7FFFFFFF).astype(np.int64).max(1)
        f = (bits + ((1 << 21) if d is None else (1 << 22) - 1)) >> 23
        s = np.where(f >= 255, 255, np.maximum(f - 2, 0))
        scales[:, b] = s
        with np.errstate(invalid="ignore", over="ignore"):
            y = np.abs(v.astype(np.float64)) * np.exp2((127 - s).astype(np.float64))[:, None]
            q = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))
            z = np.rint(y / q) if d is None else np.floor(y / q + d[:, at].astype(np.float64) / 65536)
            z = np.where(s[:, None] == 255, 0.0, z * q)
        code = np.searchsorted(LEVELS, z).astype(np.uint8)
        assert (LEVELS[np.minimum(code, 7)] == z).all()
        sign = (np.ascontiguousarray(v).view(np.uint32) >> 31).astype(np.uint8)
        nib[:, at] = np.where(s[:, None] == 255, 0, code | (sign << 3))
    return nib[:, 0::2] | (nib[:, 1::2] << 4), scales


def values(codes, scales, cols):
    """What codes and scales stand for, in 64 bits."""
    nib = np.empty((codes.shape[0], codes.shape[1] * 2), np.uint8)
    nib[:, 0::2], nib[:, 1::2] = codes & 15, codes >> 4
    v = LEVELS[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v * np.repeat(s, BLOCK, axis=1))[:, :cols]


def orthogonalize(u, steps=5, coefs=COEFS, eps=1e-7):
    """The iteration in 64 bits, on a torch matrix."""
    x = u.double()
    x = x / (x.norm() + eps)
    rows = [coefs] * steps if not hasattr(coefs[0], "__len__") else coefs
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    for a, b, c in rows:
        g = x @ x.t()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.t() if tall else x


def adjust_of(shape, adjust):
    r, c = shape
    return {"rms": 0.2 * max(r, c) ** 0.5, "shape": max(1.0, r / c) ** 0.5, None: 1.0}[adjust]


def muon(g, m, w, *, lr, beta, weight_decay, nesterov, adjust="rms", coef=1.0, **kw):
    """(momentum rounded to fp32, weights in 64 bits, the orthogonalised matrix) of one step."""
    g = g.double() * coef
    m32 = (beta * m.double() + (1 - beta) * g).float()
    u = (1 - beta) * g + beta * m32.double() if nesterov else m32
    x = orthogonalize(u, **kw)
    return m32, (1 - lr * weight_decay) * w.double() - lr * adjust_of(g.shape, adjust) * x, x
