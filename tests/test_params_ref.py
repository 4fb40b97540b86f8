"""The numpy reference of the step over separate tensors, pinned on the CPU:
e4m3 against torch's type, the rounding rules by their definitions, and
planted mistakes that the checks must catch."""

import numpy as np
import pytest
import torch

import params_ref as ref


def test_decode_is_torchs_e4m3_and_e8m0():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    got = ref.decode(codes, np.full(8, 127, np.uint8))
    np.testing.assert_array_equal(got, want)
    one = np.full(256 * 32, 0x38, np.uint8)  # code of 1.0
    want = torch.from_numpy(codes).view(torch.float8_e8m0fnu).double().numpy()
    np.testing.assert_array_equal(ref.decode(one, codes)[::32], want)


def test_nearest_is_torchs_rounding_under_the_blocks_scale():
    r = np.random.default_rng(0)
    x = (r.standard_normal(1 << 14) * np.exp2(r.integers(-30, 30, 1 << 14).repeat(1))).astype(np.float32)
    s = ref.scale_bytes(x)
    y = (x.astype(np.float64) / np.repeat(2.0 ** (s.astype(float) - 127), 32)).astype(np.float32)
    assert np.abs(y).reshape(-1, 32).max(1).min() >= 124 and np.abs(y).max() < 248
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.encode(x, s), want)


def test_nearest_keeps_what_mx8_holds():
    r = np.random.default_rng(1)
    x = r.standard_normal(1 << 12).astype(np.float32)
    s = ref.scale_bytes(x)
    c = ref.encode(x, s)
    x2 = ref.decode(c, s).astype(np.float32)
    np.testing.assert_array_equal(ref.scale_bytes(x2), s)
    np.testing.assert_array_equal(ref.encode(x2, s), c)


def test_stochastic_rounding_by_its_definition():
    """A value a share u of the way between two codes rounds up for just that
    share of the dithers, in the normal and the subnormal range."""
    d = np.arange(65536, dtype=np.uint32)
    for v, lo, hi in ((200.0, 192.0, 208.0), (9.25, 9.0, 10.0), (0.011, 5 * 2.0 ** -9, 6 * 2.0 ** -9), (0.0005, 0.0, 2.0 ** -9)):
        s = np.full(65536 // 32, 127, np.uint8)
        got = ref.decode(ref.encode(np.full(65536, v, np.float32), s, d), s)
        assert set(np.unique(got)) <= {lo, hi}
        assert abs((got == hi).mean() - (v - lo) / (hi - lo)) <= 2.0 ** -16
        assert ref.decode(ref.encode(np.full(32, v, np.float32), s[:1], d[:32], root=True), s[:1]).min() > 0


@pytest.mark.parametrize("top,byte", [(0.0, 0), (2.0 ** -149, 0), (2.0 ** -119, 1), (1.0, 120), (1.9374, 120),
                                      (1.9375, 121), (3.0e38, 247), (3.4e38, 255), (np.inf, 255), (np.nan, 255)])
def test_scale_byte(top, byte):
    x = np.zeros(32, np.float32)
    x[17] = top
    assert ref.scale_bytes(x)[0] == byte


def test_dithers_of_steps_are_even_and_unrelated():
    i = np.arange(1 << 14)
    d = np.stack([np.stack(ref.dither(i, t)).astype(np.float64) / 65536 - 0.5 for t in range(1, 65)])  # [T, 2, N]
    # sums of K independent terms of variance 1/12 (1/144 for products): six sigma
    K = d[:, 0].size
    for k in range(2):
        assert abs(d[:, k].mean()) < 6 / np.sqrt(12 * K)
        assert abs((d[1:, k] * d[:-1, k]).mean()) < 6 / (12 * np.sqrt(K))
        assert abs((d[:, k, 1:] * d[:, k, :-1]).mean()) < 6 / (12 * np.sqrt(K))
    assert abs((d[:, 0] * d[:, 1]).mean()) < 6 / (12 * np.sqrt(K))


@pytest.mark.parametrize("plant", ["nearest", "other element", "other half", "no sign", "scale"])
def test_the_checks_catch_planted_mistakes(plant):
    r = np.random.default_rng(2)
    n = 1000
    x = r.standard_normal(n)
    dm, dr = ref.dither(np.arange(n), 5)
    s = ref.scale_bytes(x)
    c = ref.encode(x, s, dm)
    ref.check_mx8(c, s, x, dm)
    if plant == "nearest":
        c = ref.encode(x, s)
    elif plant == "other element":
        c = ref.encode(x, s, np.roll(dm, 1))
    elif plant == "other half":
        c = ref.encode(x, s, dr)
    elif plant == "no sign":
        c = c & 0x7F
    else:
        s = s + 1
        c = ref.encode(x, s, dm)
    with pytest.raises(AssertionError):
        ref.check_mx8(c, s, x, dm)


def test_near_catches_a_second_rounding():
    r = np.random.default_rng(3)
    x = r.standard_normal(4096)
    ref.near(x.astype(np.float32), x)
    with pytest.raises(AssertionError):
        ref.near((x * (1 + 2.0 ** -24)).astype(np.float32), x)
