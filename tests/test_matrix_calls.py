"""Calls of fp_mx4_* that have nothing to do, and what the header says of MXFP4's roundings, without a GPU."""

import os
import re

import numpy as np
import pytest

import matrix_ref as ref
from conftest import ROOT

HEADER = open(os.path.join(ROOT, "include", "flatparam.h")).read()
HEADER = re.sub(r"\s+", " ", re.sub(r"\n \* ?", " ", HEADER))
F32 = 0
RANGE = -2


@pytest.mark.parametrize("want,kw", [
    (0, dict(m=0)), (0, dict(n=0, pitch=0)), (0, dict(m=0, n=0, pitch=0)),
    (RANGE, dict(m=0, k=-1)), (RANGE, dict(m=0, k=(1 << 22) + 1)), (RANGE, dict(m=-1)),
])
def test_an_output_without_elements_and_no_contraction(fp, want, kw):
    a = {**dict(m=8, n=16, k=0, pitch=16), **kw}
    assert fp.lib().fp_mx4_matmul(a["m"], a["n"], a["k"], None, None, None, None, F32, None, a["pitch"], 0, None) == want


def low_by(y, d):
    """How far below each of up to 31 values their stochastic rounding comes out on average over the dithers d, under a scale of 1."""
    row = np.concatenate([[6.0], y]).astype(np.float32)
    codes, scales = ref.quantize(np.repeat(row[None], len(d), 0), np.repeat(d[:, None], len(row), 1))
    assert (scales[:, 0] == 127).all()
    return (row.astype(np.float64) - ref.values(codes, scales, len(row)).mean(0))[1:]


def test_the_stochastic_rounding_is_low_by_less_than_the_header_says():
    assert "low by less than 2^-16 of q, by 2^-17 of it on average" in HEADER
    r = np.random.default_rng(2)
    d = np.arange(65536, dtype=np.uint64)
    low = np.concatenate([low_by(r.uniform(lo, hi, 31), d) / q for lo, hi, q in ((0, 2, 0.5), (2, 4, 1.0), (4, 6, 2.0))])
    assert 0 <= low.min() and low.max() < 2.0 ** -16
    assert abs(low.mean() - 2.0 ** -17) < 0.25 * 2.0 ** -17  # sigma of the mean: 2^-16 / sqrt(12 * 93), 0.06 of it
    tiny = np.float32(0.4 * 2.0 ** -16)
    assert low_by([tiny], d)[0] == tiny  # below 2^-16 of q: never up


def test_one_seed_for_every_call_does_not_average_out():
    """Over calls with one seed an element stays where its dither put it; over new seeds its mean is the value: 400 draws of
    0 or 0.5 for 0.2, within 5 of their standard deviations."""
    assert "with one seed an element is rounded the same way every time" in HEADER
    x = np.full((1, 64), 0.2, np.float32)
    x[0, ::32] = 6.0
    rounded = lambda seed: ref.values(*ref.quantize(x, ref.dither(1, 64, seed) >> np.uint64(16)), 64)[0, 1::32]  # noqa: E731
    same, new = np.array([rounded(7) for _ in range(400)]), np.array([rounded(t) for t in range(400)])
    assert (same == same[0]).all() and (np.abs(same.mean(0) - 0.2) >= 0.19).all()
    assert (np.abs(new.mean(0) - 0.2) <= 5 * 0.5 * (0.4 * 0.6 / 400) ** 0.5).all()
