"""The step over many separate tensors and MXFP8 on the GPU, at the ends of
their ranges: against the numpy reference (params_ref.py)."""

import math

import numpy as np
import pytest
import torch

import params_ref as ref
from gpu_common import dev, say
from test_gpu_params import HPS, SIZES, Case, columns, run

pytestmark = pytest.mark.gpu

# The weights are evaluated in fp64 and rounded once.  The largest error before
# that rounding is the quotient's: a hardware reciprocal within 2^-23 of its
# value and one Newton step, which squares that, to 2^-46 of the change; the
# root's is below 1.5 * 2^-46, the other operations' 2^-53 each: 2^-44 in all.
# The first moment's two terms may cancel: its roundings, two here and three in
# the reference, are 2^-53 each of the terms, not of their sum: 2^-50 in all.
ONCE, TERMS = 2.0 ** -24, 2.0 ** -30  # `near` takes 2^-20 of its last argument


def check_weights(case, before, t, what, hps=None):
    after = case.host()
    for i, s, d, o in case.tensors():
        if s:
            p, b = slice(o, o + s), slice(o // 32, o // 32 + -(-s // 32))
            old = before["moments"]
            g, w, hp = before["grad"][d], before["master"][d], (hps or case.hps)[case.groups[i]]
            m, v = ref.decode(old[0][p], old[1][b]), ref.decode(old[2][p], old[3][b]) ** 2
            th, _, _, terms, change = ref.adamw(g, w, m, v, hp, t)
            apart = ref.adamw(np.abs(g), w, np.abs(m), v, hp, t)[4]  # the change if its terms added up
            ref.near(after["master"][d], th, terms, f"{what} tensor {i} of {s}", change * ONCE + apart * TERMS)


@pytest.mark.parametrize("grad", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("zero", [False, True])
def test_weights_with_8_bit_moments_are_rounded_once(fp, grad, zero):
    """As those with fp32 moments; weights of zero (biases) show it most."""
    say("rounded once", grad, zero)
    for sizes in SIZES:
        case = Case(fp, SIZES[sizes], grad, "bf16", 8, 1, seed=11)
        if zero:
            case.master.zero_()
        for t in (1, 2, 50):
            before = case.host()
            run(case, t, seed=t)
            check_weights(case, before, t, f"{sizes} step {t}")


@pytest.mark.parametrize("eps", [1e-8, 0.0])
@pytest.mark.parametrize("e", [-140, -133, -127, -124, -120, -60, 60, 110, 119, 122, 124, 126])
def test_changes_at_all_magnitudes(fp, e, eps):
    """Gradients and roots of 2^e to 2^(e + 1), at the first step, where the
    root's bias correction is largest, and at a later one."""
    say("magnitude", e, eps)
    for t in (1, 100):
        case = Case(fp, [1000, 33], grad="f32", copy=None, bits=8, warm=False, groups=False)
        r = np.random.default_rng(e + 1000 + t)
        g = np.ldexp(r.uniform(1, 2, case.n) * r.choice([-1, 1], case.n), e).astype(np.float32)
        case.grad.copy_(torch.from_numpy(g).to(dev()))
        case.master[::2] = 0.0
        if t > 1:
            x = torch.from_numpy(np.ldexp(r.uniform(1, 1.9, case.plan.partition), e).astype(np.float32)).to(dev())
            fp.mx8_quantize(x, case.moments[2], case.moments[3])
        case.hps = [dict(HPS[0], eps=eps)]
        before = case.host()
        run(case, t, seed=t)
        check_weights(case, before, t, f"2^{e} step {t}", [dict(HPS[0], eps=max(eps, 2.0 ** -126))])
        case.hps = [dict(HPS[0], eps=max(eps, 2.0 ** -126))]
        case.check(before, t, t, what=f"2^{e} step {t}")
