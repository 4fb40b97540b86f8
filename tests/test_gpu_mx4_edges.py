"""MXFP4 products at the ends of what they take, on the GPU: no contraction at all, scales at the ends of their range, many steps
on the large tiles with every output, and a layer's gradients against differences."""

import numpy as np
import pytest
import torch

import matrix_ref as ref
from gpu_common import dev, say

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


# ------------------------------------------------------------------ products
def to_dev(form):
    return [torch.from_numpy(t).to(dev()) for t in form]


def reference(qa, qb, k):
    """The product and the sum of its terms' sizes, in 64 bits."""
    va, vb = torch.from_numpy(ref.values(*qa, k)), torch.from_numpy(ref.values(*qb, k))
    return va @ vb.t(), va.abs() @ vb.abs().t()


@pytest.mark.parametrize("m,n,k", [(5, 100, 8192), (20, 100, 8192), (70, 80, 8192), (1501, 1699, 1024)])
def test_scales_of_the_whole_range(fp, m, n, k):
    """Blocks under scales from 2^-127 to 2^127, the other operand's under the opposite ones, so that every product is of a
    middle size."""
    rng = np.random.default_rng(m)
    base = np.linspace(0, 254, k // 32).round().astype(np.int64)
    base[:4], base[-4:] = (0, 1, 2, 3), (251, 252, 253, 254)
    rng.shuffle(base)

    def form(rows, at):
        codes = rng.integers(0, 256, (rows, k // 2)).astype(np.uint8)
        return codes, np.clip(at + rng.integers(-3, 4, (rows, k // 32)), 0, 254).astype(np.uint8)

    qa, qb = form(m, base), form(n, 254 - base)
    assert {0, 254} <= set(qa[1].ravel()) and {0, 254} <= set(qb[1].ravel())
    want, size = reference(qa, qb, k)
    got = fp.mx4_matmul(to_dev(qa), to_dev(qb), dtype=torch.float32).cpu().double()
    assert bool(((got - want).abs() <= k * 2.0 ** -24 * size).all())


def test_lengths_that_pad_alike(fp):
    """300 and 400 elements are both padded to 512: what the shorter rows lack counts as zeros."""
    gen = torch.Generator().manual_seed(4)
    a, b = torch.randn(20, 300, generator=gen), torch.randn(30, 400, generator=gen)
    got = fp.mx4_matmul(fp.mx4_quantize(a.to(dev())), fp.mx4_quantize(b.to(dev())), dtype=torch.float32)
    longer = torch.cat([a, torch.zeros(20, 100)], 1)
    assert torch.equal(got, fp.mx4_matmul(fp.mx4_quantize(longer.to(dev())), fp.mx4_quantize(b.to(dev())), dtype=torch.float32))


LARGE = {}


def large(m, n, k):
    """Operands and their product, made once per shape; elements small enough for fp16 sums."""
    if (m, n, k) not in LARGE:
        LARGE.clear()
        rng = np.random.default_rng(k)
        q = [ref.quantize((rng.standard_normal((r, k)) * np.exp(0.3 * rng.standard_normal((r, 1)))).astype(np.float32)) for r in (m, n)]
        LARGE[m, n, k] = [to_dev(f) for f in q], *reference(*q, k)
    return LARGE[m, n, k]


@pytest.mark.parametrize("m,n,k", [(1501, 1699, 777), (3901, 4203, 777)])  # on 128- and 256-wide tiles
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_many_steps_on_large_tiles(fp, m, n, k, dtype, accumulate):
    (a, b), want, size = large(m, n, k)
    say("product", m, n, k, dtype, accumulate)
    whole = torch.full((m, n + 9), 5.0, dtype=DT[dtype], device=dev())
    out = whole[:, 4:4 + n]
    if accumulate:
        old = (torch.randn(m, n, generator=torch.Generator().manual_seed(7)) * 20).to(DT[dtype])
        out.copy_(old.to(dev()))
        want, size = want + old.double(), size + old.double().abs()
    fp.mx4_matmul(a, b, out, accumulate=accumulate)
    assert bool((want.abs() < 60000).all())
    # the sum's terms, one rounding of the output, and fp16's smallest step
    bound = (k + 1) * 2.0 ** -24 * size + torch.finfo(DT[dtype]).eps / 2 * 1.01 * want.abs() + (2.0 ** -25 if dtype == "f16" else 0.0)
    bad = (out.cpu().double() - want).abs() > bound
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())
    assert bool((whole[:, :4] == 5).all()) and bool((whole[:, 4 + n:] == 5).all())


# ------------------------------------------------------------------ gradients
@pytest.mark.parametrize("t,n,k", [(1, 40, 70), (37, 300, 130), (260, 64, 257), (700, 1100, 900)])
def test_gradients_are_the_forwards_differences(fp, t, n, k):
    """The loss sum(dy (x w^T)) through the forward product at x + d and x - d, and at w + d and w - d.  Elements are whole numbers
    up to 3, which every block's scale holds (1, 2 and 3 are 2, 4 and 6 halves), so that quantisation, to nearest or
    stochastically, changes nothing; sums are whole numbers below 2^24.  So the differences are the gradients' products
    with d, exactly, and far from 0 (a gradient of zeros or of another sign would show)."""
    gen = torch.Generator().manual_seed(t + n)
    pick = lambda r, c: (torch.randint(1, 3, (r, c), generator=gen) * (2 * torch.randint(0, 2, (r, c), generator=gen) - 1)).float()  # noqa: E731
    x, w, dy = pick(t, k), pick(n, k), pick(t, n)
    dev_x, dev_w, dev_dy = x.to(dev()), w.to(dev()), dy.to(dev())
    qx, qw = fp.mx4_quantize(dev_x, transposed=True), fp.mx4_quantize(dev_w, transposed=True)
    qd = fp.mx4_quantize(dev_dy, transposed=True, seed=11)
    dx = fp.mx4_matmul(qd[:2], qw[2:], dtype=torch.float32)
    dw = torch.zeros(n, k, device=dev())
    fp.mx4_matmul(qd[2:], qx[2:], dw, accumulate=True)

    def loss(a, b):
        y = fp.mx4_matmul(fp.mx4_quantize(a), fp.mx4_quantize(b), dtype=torch.float32)
        return float((y.double() * dev_dy.double()).sum())

    for name, g, move in (("x", dx, lambda d: loss(dev_x + d, dev_w) - loss(dev_x - d, dev_w)),
                          ("w", dw, lambda d: loss(dev_x, dev_w + d) - loss(dev_x, dev_w - d))):
        one = torch.zeros_like(g)
        for d in (torch.sign(g), one):  # towards the gradient, and one element alone
            if d is one:
                at = int(g.abs().argmax())
                d.view(-1)[at] = 1.0
            exact = float((g.double() * d.double()).sum())
            got = move(d) / 2
            assert got == exact and abs(exact) >= 1, (name, got, exact)
    assert torch.equal(dx.cpu().double(), dy.double() @ w.double()) and torch.equal(dw.cpu().double(), dy.double().t() @ x.double())
