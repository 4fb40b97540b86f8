"""What the header says of MXFP8 moments, checked with the numpy reference, and
plans that the binding refuses before it asks a GPU."""

import os
import re

import numpy as np
import pytest

import params_ref as ref
from conftest import ROOT

HEADER = open(os.path.join(ROOT, "include", "flatparam.h")).read()
HEADER = re.sub(r"\s+", " ", re.sub(r"\n \* ?", " ", HEADER))
CODES = np.arange(0, 127, dtype=np.uint8)


def test_the_range_whose_squares_are_fp32():
    """Every root in the range that the header states comes back from its square
    in fp32; just outside, some do not."""
    lo, hi = map(int, re.search(r"2\^(-\d+) <= r < 2\^(\d+)", HEADER).groups())
    seen = []
    with np.errstate(over="ignore", under="ignore"):
        for b in range(255):
            r = ref.decode(CODES, np.full(4, b, np.uint8))
            v = r.astype(np.float32) * r.astype(np.float32)
            back = np.sqrt(v.astype(np.float64)).astype(np.float32)
            seen += list(zip(r, back == r))
    assert all(ok for r, ok in seen if r == 0 or 2.0 ** lo <= r < 2.0 ** hi)
    assert any(not ok for r, ok in seen if 2.0 ** (lo - 1) < r < 2.0 ** lo)
    assert not any(ok for r, ok in seen if 2.0 ** hi <= r < 2.0 ** (hi + 1))


def test_values_that_come_back():
    """Quantization gives back what it gave, and what a step's rounding gave
    unless a block's largest value went up to 256 units: its scale doubles and
    values below 2^-13 of that value may move by their last bit."""
    assert "2^-13 of" in HEADER
    r = np.random.default_rng(0)
    n = 32 * 4096
    x = (r.uniform(200, 247.99, (4096, 32)) * np.exp2(-r.integers(0, 18, (4096, 32)))).astype(np.float32)
    x[:, 0] = r.uniform(125, 247.99, 4096)
    x = x.reshape(-1) * np.where(r.random(n) < 0.5, np.float32(-1), np.float32(1))
    s = ref.scale_bytes(x)
    for d in (None, r.integers(0, 65536, n).astype(np.uint32)):
        y = ref.decode(ref.encode(x, s, d), s)
        s2 = ref.scale_bytes(y)
        z = ref.decode(ref.encode(y.astype(np.float32), s2), s2)
        top = np.repeat(np.abs(y).reshape(-1, 32).max(1), 32)
        went = top == 256
        assert np.array_equal(z[~went], y[~went])
        if d is None:
            assert not went.any()
            continue
        assert went.any() and (z != y)[went].any()
        moved = went & (z != y)
        assert (np.abs(y[moved]) < 2.0 ** -13 * 256).all() and (np.abs(z - y)[moved] == 2.0 ** -9).all()


def test_the_dithers_mean():
    """Over all dithers a value comes out low by less than 2^-16 of a code's
    width, 2^-17 on average."""
    assert "2^-17 of" in HEADER
    r = np.random.default_rng(1)
    d = np.arange(65536, dtype=np.uint32)
    s = np.full(2048, 127, np.uint8)
    low = []
    for y in np.concatenate([r.uniform(16, 32, 100), r.uniform(2.0 ** -7, 2.0 ** -6, 100)]).astype(np.float32):
        q = 2.0 if y >= 16 else 2.0 ** -9
        got = ref.decode(ref.encode(np.full(65536, y, np.float32), s, d), s).mean()
        low.append((float(y) - got) / q)
    assert 0 <= min(low) and max(low) < 2.0 ** -16
    assert abs(np.mean(low) - 2.0 ** -17) < 0.2 * 2.0 ** -17  # sigma of the mean: 2^-16 / sqrt(12 * 200)


def test_one_seed_for_every_step_sticks():
    """Why every step needs a seed of its own: decaying without gradients, nearly
    every root stays where it is under a repeated dither, and none under new ones."""
    assert "with one seed nearly every moment that changes by less than a code's width a step stays where it is" in HEADER
    n = 4096
    i = np.arange(n)
    first = np.full(n, 200.0, np.float32)
    for seed_of, stuck in ((lambda t: 1, True), (lambda t: t, False)):
        s = ref.scale_bytes(first)
        x = ref.decode(ref.encode(first, s, ref.dither(i, 1)[1], root=True), s)
        start = x.copy()
        for t in range(2, 402):
            y = (x * np.sqrt(0.999)).astype(np.float32)
            s = ref.scale_bytes(y)
            x = ref.decode(ref.encode(y, s, ref.dither(i, seed_of(t))[1], root=True), s)
        assert ((x == start).mean() > 0.95) == stuck
        assert (abs(x.mean() / start.mean() - 0.999 ** 200) < 0.01) != stuck


@pytest.mark.parametrize("top", [1.9375, 1.96, 2 - 2.0 ** -23])
def test_blocks_that_round_past_fp32(top):
    """They have no scale under which the rounded value is an fp32."""
    assert "1.9375 * 2^127" in HEADER
    x = np.zeros(32, np.float32)
    x[5] = top * 2.0 ** 127
    assert np.isfinite(x).all() and ref.scale_bytes(x)[0] == 255
    y = ref.decode(ref.encode(x, np.array([248], np.uint8)), np.array([248], np.uint8))
    assert y[5] == 2.0 ** 128  # not an fp32


@pytest.mark.parametrize("grads", [[None], [None, None]])
def test_a_gradient_that_is_not_there(fp, grads):
    with pytest.raises(TypeError, match=r"grads\[0\] is None"):
        fp.Params(grads)


@pytest.mark.parametrize("groups", [[16], [-1], [1 << 32], [(1 << 32) + 1]])
def test_group_numbers_out_of_range(fp, groups):
    """Also those whose low 32 bits are a group's."""
    import torch
    with pytest.raises(ValueError, match="group"):
        fp.Params([torch.zeros(4)], groups=groups)
