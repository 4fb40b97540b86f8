"""Calls of fp_mx4_* that have nothing to do, and what the header says of MXFP4's roundings, without a GPU."""

import pytest

F32 = 0
RANGE = -2


@pytest.mark.parametrize("want,kw", [
    (0, dict(m=0)), (0, dict(n=0, pitch=0)), (0, dict(m=0, n=0, pitch=0)),
    (RANGE, dict(m=0, k=-1)), (RANGE, dict(m=0, k=(1 << 22) + 1)), (RANGE, dict(m=-1)),
])
def test_an_output_without_elements_and_no_contraction(fp, want, kw):
    a = {**dict(m=8, n=16, k=0, pitch=16), **kw}
    assert fp.lib().fp_mx4_matmul(a["m"], a["n"], a["k"], None, None, None, None, F32, None, a["pitch"], 0, None) == want
