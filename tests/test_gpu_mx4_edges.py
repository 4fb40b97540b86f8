"""MXFP4 products at the ends of what they take, on the GPU: no contraction at all."""

import pytest
import torch

from gpu_common import dev

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ no contraction
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_a_layer_without_tokens(fp, dtype):
    """No rows in, none out; the weights' gradient is the empty sum: zeros, or what it is added to."""
    n, k = 37, 70
    qw = fp.mx4_quantize(torch.randn(n, k, device=dev()), transposed=True)
    qx = fp.mx4_quantize(torch.zeros(0, k, device=dev()), transposed=True)
    qd = fp.mx4_quantize(torch.zeros(0, n, device=dev()), transposed=True, seed=3)
    assert fp.mx4_matmul(qx[:2], qw[:2]).shape == (0, n)
    assert fp.mx4_matmul(qd[:2], qw[2:]).shape == (0, k)
    dw = fp.mx4_matmul(qd[2:], qx[2:], dtype=DT[dtype])
    assert dw.shape == (n, k) and dw.dtype == DT[dtype] and bool((dw == 0).all())
    whole = torch.full((n, k + 9), 5.0, dtype=DT[dtype], device=dev())
    out = whole[:, 4:4 + k]
    assert fp.mx4_matmul(qd[2:], qx[2:], out, accumulate=True) is out
    assert bool((whole == 5).all())
    before = whole._version
    out[3, 3] = float("nan")
    fp.mx4_matmul(qd[2:], qx[2:], out)
    assert whole._version > before + 1
    assert bool((out == 0).all()) and bool((whole[:, :4] == 5).all()) and bool((whole[:, 4 + k:] == 5).all())


def test_no_contraction_and_no_output(fp):
    q = fp.mx4_empty(0, 0, dev())
    assert fp.mx4_matmul(q, q).shape == (0, 0)
    assert fp.mx4_matmul(fp.mx4_empty(5, 0, dev()), q).shape == (5, 0)


def test_refusals_without_contraction(fp):
    a, b = fp.mx4_empty(5, 0, dev()), fp.mx4_empty(6, 0, dev())
    with pytest.raises(ValueError, match="shape"):
        fp.mx4_matmul(a, b, torch.zeros(5, 7, device=dev()))
    with pytest.raises(TypeError):
        fp.mx4_matmul(a, b, dtype=torch.float64)
    with pytest.raises(ValueError, match="contiguous"):
        fp.mx4_matmul(a, b, torch.zeros(6, 5, device=dev()).t())
    with pytest.raises(ValueError, match="device"):
        fp.mx4_matmul(a, b, torch.zeros(5, 6))
