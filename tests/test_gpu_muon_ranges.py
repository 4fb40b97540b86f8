"""Coefficients and eps at the ends of what the orthogonalisation takes, on the GPU."""

import pytest
import torch

import matrix_ref as ref
from gpu_common import dev, say

pytestmark = pytest.mark.gpu

OFF = 4e-3  # as in test_gpu_muon.py
SHAPES = [(3, 100), (100, 3), (40, 70)]
LARGE = (700, 600)


def plan_of(fp, grads):
    out = [torch.full(g.shape, 9.0, device=dev()) for g in grads]
    return fp.Muon([g.to(dev()) for g in grads], updates=out), out


@pytest.mark.parametrize("beside", [False, True])
@pytest.mark.parametrize("c", [1e-17, -1e-17, 1e-30, 1e-300, 0.0])
def test_a_polynomial_whose_highest_coefficient_is_next_to_nothing(fp, c, beside):
    """50 x - 49 x^3 + c x^5 is largest, 19.4, at 0.58, and 1 at 1: the scale of the next X goes by the former."""
    grads = [torch.randn(s, generator=torch.Generator().manual_seed(i)) for i, s in enumerate(SHAPES + ([LARGE] if beside else []))]
    coefs = [(50.0, -49.0, c), (1.0, 0.0, 0.0)]
    plan, out = plan_of(fp, grads)
    plan.orthogonalize(plan.new_workspace(), steps=2, coefs=coefs)
    for g, x in zip(grads, out):
        say("coefficients", c, tuple(g.shape))
        want = ref.orthogonalize(g, 2, coefs)
        # 3 rows have singular values of about 0.58, where x loses 49 x^2 = 16 of its 50 to the products, whose operands are
        # rounded by 2^-12 four times: 2 * 16 / 34 * 2^-12 = 2.3e-4, less elsewhere
        assert float((x.cpu().double() - want).norm() / want.norm()) <= OFF


@pytest.mark.parametrize("beside", [False, True])
def test_the_smallest_eps(fp, beside):
    """Zeros stay zeros under the smallest normal eps; smaller ones, whose reciprocal fp64 does not hold, are refused."""
    grads = [torch.zeros(s) for s in SHAPES] + [torch.randn(20, 30, generator=torch.Generator().manual_seed(1))]
    if beside:
        grads += [torch.zeros(LARGE), torch.randn(LARGE, generator=torch.Generator().manual_seed(2))]
    plan, out = plan_of(fp, grads)
    ws = plan.new_workspace()
    plan.orthogonalize(ws, eps=2.3e-308)
    for g, x in zip(grads, out):
        if not bool(g.any()):
            assert bool((x == 0).all())
        else:
            want = ref.orthogonalize(g, eps=2.3e-308)
            assert float((x.cpu().double() - want).norm() / want.norm()) <= OFF
    for eps in (1e-310, 5e-324, 0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(fp._lib.FlatParamError, match="eps"):
            plan.orthogonalize(ws, eps=eps)
