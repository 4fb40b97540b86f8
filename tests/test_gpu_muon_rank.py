"""The orthogonalisation of matrices of low rank, as the gradients of few tokens are, on the GPU against 64 bits.

How far it may be off, relative and in the 2-norm.  Let X have rank k, X_h its fp16 form and E = X - X_h, and D + R = B.
A step in the directions that X has is off as tests/test_gpu_muon.py counts it, by 1.9e-3 in all.  What those directions do not hold
grows by a = 3.44 in every step.  B times anything lies in the columns of X, and the roundings of A and of R act on X from the
left, so neither leaves the rank but by products of two roundings (2^-24 times 3.44^4 = 140: 1e-5); nor do the 20 bits of X
between the steps count (2^-21 * 140 = 7e-5).  Where D multiplies X_h that is all.  In the last two steps it multiplies X, which
adds D E, by which later steps multiply 3.44 at most, then 1: with |D| <= |B| <= 2.8 and E's root mean square of 2^-12 of X
that is 2.8 * 2^-12 * (3.44^2 + 1)^(1/2) = 2.4e-3.  Together (1.9^2 + 2.4^2)^(1/2) = 3.1e-3; the header says:
"""

import pytest
import torch

import matrix_ref as ref
from gpu_common import dev, say

pytestmark = pytest.mark.gpu

OFF = 4e-3
HP = dict(lr=0.01, beta=0.9, weight_decay=0.1, nesterov=True)


def low_rank(r, c, rank, seed, rows=None):
    """A product of normal factors; rows: the smaller side's rows (columns) beyond so many are zero."""
    gen = torch.Generator().manual_seed(seed)
    a, b = torch.randn(r, rank, generator=gen), torch.randn(rank, c, generator=gen)
    if rows is not None:
        if r <= c:
            a[rows:] = 0
        else:
            b[:, rows:] = 0
    return a @ b * 1e-3


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


SHAPES = [(2, 512), (512, 2), (4, 64), (64, 8), (16, 1024), (32, 48), (48, 32), (64, 64), (100, 128), (128, 128)]
LARGE = (700, 600)  # beside it small matrices go through the launches of large ones


@pytest.mark.parametrize("beside", [False, True])
@pytest.mark.parametrize("rank", [1, 2, 4])
def test_low_rank(fp, rank, beside):
    shapes = SHAPES + ([LARGE] if beside else [])
    grads = [low_rank(r, c, rank, 10 * i + rank) for i, (r, c) in enumerate(shapes)]
    out = [torch.empty(s, device=dev()) for s in shapes]
    plan = fp.Muon([g.to(dev()) for g in grads], updates=out)
    assert (plan.workspace_bytes > 0) == beside
    plan.orthogonalize(plan.new_workspace())
    off = {}
    for s, g, x in zip(shapes, grads, out):
        off[s] = rel(x.cpu(), ref.orthogonalize(g))
        say("rank", rank, s, off[s])
    assert all(v <= OFF for v in off.values()), off


@pytest.mark.parametrize("shape", [(300, 300), (512, 1408), (1408, 512), (2048, 2048), (64, 30000)])
@pytest.mark.parametrize("rank", [1, 2])
def test_few_rows_of_large_matrices(fp, shape, rank):
    """A gradient that has only a few rows, of rank 1 or 2."""
    g = low_rank(*shape, rank, 5, rows=3 * rank)
    x = torch.empty(shape, device=dev())
    plan = fp.Muon([g.to(dev())], updates=[x])
    plan.orthogonalize(plan.new_workspace())
    off = rel(x, ref.orthogonalize(g.to(dev())))
    say("few rows", rank, shape, off)
    assert off <= OFF


@pytest.mark.parametrize("beside", [False, True])
def test_steps_on_the_gradients_of_one_token(fp, beside):
    """The momentum of two such gradients has rank 2."""
    shapes = [(2, 512), (8, 64), (32, 48), (64, 64)] + ([LARGE] if beside else [])
    grads = [low_rank(r, c, 1, i).to(dev()) for i, (r, c) in enumerate(shapes)]
    master = [low_rank(r, c, 4, 50 + i).to(dev()) for i, (r, c) in enumerate(shapes)]
    plan = fp.Muon(grads, master)
    mom, ws = plan.new_momentum(), plan.new_workspace()
    for t in range(2):
        for i, g in enumerate(grads):
            g.copy_(low_rank(*shapes[i], 1, 100 * t + i))
        ms = [plan.tensor_slice(mom, i).cpu().view(s) for i, s in enumerate(shapes)]
        before = [w.cpu().clone() for w in master]
        plan.step(mom, ws, **HP)
        for i, s in enumerate(shapes):
            say("step", t, s)
            _, w, x = ref.muon(grads[i].cpu(), ms[i], before[i], **HP)
            rate = HP["lr"] * ref.adjust_of(s, "rms")
            assert float((master[i].cpu().double() - w).norm()) <= OFF * rate * float(x.norm()) + 2.0 ** -24 * float(w.norm())


def test_a_slower_iteration_of_many_steps(fp):
    """Ten steps of 15/8, -10/8, 3/8: a direction near 0 grows by 1.875 a step, 540 in all."""
    for shape in ((2, 512), (64, 64), (700, 600)):
        g = low_rank(*shape, 1, 3, rows=2)
        x = torch.empty(shape, device=dev())
        plan = fp.Muon([g.to(dev())], updates=[x])
        plan.orthogonalize(plan.new_workspace(), steps=10, coefs=(1.875, -1.25, 0.375))
        off = rel(x.cpu(), ref.orthogonalize(g, 10, (1.875, -1.25, 0.375)))
        say("ten steps", shape, off)
        # |B| <= 1.05, and the two last factors are 1.875^2 and 1.875 (4 is what the rule allows): less than above
        assert off <= OFF


def few_values():
    gen = torch.Generator().manual_seed(9)
    sign = lambda r, c: torch.sign(torch.randn(r, c, generator=gen))  # noqa: E731
    one = torch.zeros(20, 30)
    one[7] = torch.randn(30, generator=gen)
    return [torch.eye(m, 64) for m in (1, 3, 8, 32, 43, 64)] + [torch.ones(m, n) for m, n in ((3, 3), (16, 64), (38, 38), (48, 64), (128, 100))] \
        + [sign(m, n) for m, n in ((3, 3), (3, 64), (64, 4), (40, 50))] + [sign(24, 3) @ sign(3, 16), torch.diag(torch.randn(4, generator=gen)), one]


@pytest.mark.parametrize("beside", [False, True])
def test_matrices_of_few_values(fp, beside):
    """Elements that are all rounded alike: nothing averages out.  With S the singular values s, a relative rounding d of X's
    elements moves a s + b s^3 + c s^5 by (2 b s^3 + 4 c s^5) d through A and (b s^3 + c s^5) d in the product, one of A by (b s^3 +
    2 c s^5) d, one of R by (b s^3 + c s^5) d, and the polynomial's derivative carries this on.  With d's root mean square,
    2^-11 / 3^(1/2), over five steps that comes to 1.4e-2 of s at most, for s from 0 to 1; twice that: """
    grads = few_values() + ([low_rank(*LARGE, 1, 2)] if beside else [])
    out = [torch.empty(g.shape, device=dev()) for g in grads]
    plan = fp.Muon([g.to(dev()) for g in grads], updates=out)
    plan.orthogonalize(plan.new_workspace())
    for i, (g, x) in enumerate(zip(grads, out)):
        off = rel(x.cpu(), ref.orthogonalize(g))
        say("few values", i, tuple(g.shape), off)
        assert off <= 2.8e-2


def test_a_matrix_alone_and_beside_others(fp):
    """Another plan's kernels give another result within the iteration's error; a plan over the same sizes gives the same bits."""
    shapes = [(40, 70), (128, 128), (30, 5000), (16, 4096), (300, 310)]

    def run(more):
        grads = [torch.randn(s, generator=torch.Generator().manual_seed(i)).to(dev()) for i, s in enumerate(shapes + more)]
        out = [torch.empty(s, device=dev()) for s in shapes + more]
        plan = fp.Muon(grads, updates=out)
        plan.orthogonalize(plan.new_workspace())
        return out[:len(shapes)]

    first, again, other = run([(20, 30)]), run([(20, 30)]), run([(1200, 1100)] * 20)
    for i, s in enumerate(shapes):
        g = torch.randn(s, generator=torch.Generator().manual_seed(i))
        alone = torch.empty(s, device=dev())
        one = fp.Muon([g.to(dev())], updates=[alone])
        one.orthogonalize(one.new_workspace())
        want = ref.orthogonalize(g)
        assert torch.equal(first[i], again[i])
        for x in (first[i], other[i], alone):
            assert rel(x.cpu(), want) <= OFF
        say("alone and beside others", s, rel(first[i], alone.double()), rel(other[i], alone.double()))
