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


@pytest.mark.parametrize("e", [-149, -146, -140, -136, -130, -127, -126, -123, -120, -119, -118])
def test_mx8_under_the_smallest_scales(fp, e):
    """Blocks whose largest value is 2^e to 2^(e + 1), subnormal ones and those
    under the scale byte 0 among them, both signs and zeros."""
    say("mx8 small", e)
    r = np.random.default_rng(e + 1000)
    n = 32 * 40 + 7
    x = np.ldexp(r.uniform(1, 2, n), e) * np.exp2(-r.integers(0, 12, n)) * r.choice([-1.0, 0.0, 1.0], n)
    x[::32] = np.ldexp(r.uniform(1, 2, x[::32].size), e)
    x = x.astype(np.float32)
    c, s = fp.mx8_quantize(torch.from_numpy(x).to(dev()))
    c, s = (t.view(torch.uint8).cpu().numpy() for t in (c, s))
    ref.check_mx8(c, s, x.astype(np.float64), what=f"2^{e}")
    assert s.max() <= max(0, e + 1 + 127 - 7) and (e >= -120 or not s.any())
    out = fp.mx8_dequantize(torch.from_numpy(c).to(dev()), torch.from_numpy(s).to(dev()))
    np.testing.assert_array_equal(out.cpu().numpy(), ref.decode(c, s).astype(np.float32))


@pytest.mark.parametrize("e", range(-137, -119))
def test_steps_under_the_smallest_scales(fp, e):
    """Moments that the step rounds stochastically under scale bytes 0 to 9, and
    roots that it raises there."""
    say("step small", e)
    case = Case(fp, [32 * 50 + 3, 40], grad="f32", copy=None, bits=8, warm=False)
    r = np.random.default_rng(e + 1000)
    g = np.ldexp(r.uniform(1, 2, case.n), e) * np.exp2(-r.integers(0, 14, case.n)) * r.choice([-1.0, 0.0, 1.0], case.n)
    case.grad.copy_(torch.from_numpy(g.astype(np.float32)).to(dev()))
    for t in (1, 2, 3):
        before = case.host()
        run(case, t, seed=t)
        case.check(before, t, t, what=f"2^{e} step {t}")
    assert int(case.moments[1].max()) <= 9 and int(case.moments[3].max()) <= 9


@pytest.mark.parametrize("top,finite", [(1.9374, True), (1.9375, False), (1.9999, False)])
def test_blocks_at_fp32s_end(fp, top, finite):
    """A block whose largest value rounds past fp32's range reads as NaN, by the
    conversion and by the step; one just below keeps its values."""
    say("fp32's end", top)
    x = np.full(64, 2.0 ** 125, np.float32)
    x[3] = -top * 2.0 ** 127
    t = torch.from_numpy(x).to(dev())
    c, s = fp.mx8_quantize(t)
    y = fp.mx8_dequantize(c, s)
    assert bool(torch.isnan(y[:32]).all()) != finite and bool(torch.isfinite(y[:32]).all()) == finite
    assert torch.equal(y[32:], t[32:])
    w = torch.zeros(64, device=dev())
    plan = fp.Params([t], [w])
    mom = plan.new_moments(8)
    plan.step(mom, step=1, seed=1, **dict(HPS[0], beta1=0.0))
    assert int(mom[1].view(torch.uint8)[0]) == (247 if finite else 255) and int(mom[1].view(torch.uint8)[1]) < 255
    assert bool(torch.isfinite(w).all())


def roots(seed, lo, hi):
    """fp32 roots whose non-zero MXFP8 values lie in [2^lo, 2^hi]."""
    r = np.random.default_rng(seed)
    x = np.exp2(r.uniform(lo, hi, (64, 1)) - r.uniform(0, 20, (64, 32)))
    x = np.where(r.random(x.shape) < 0.1, 0.0, np.maximum(x, 2.0 ** lo))
    return x.reshape(-1).astype(np.float32)


@pytest.mark.parametrize("lo,hi", [(-71, -50), (-30, 0), (20, 63.9)])
def test_second_moments_come_back_as_fp32(fp, lo, hi):
    say("second moments", lo, hi)
    c, s = fp.mx8_quantize(torch.from_numpy(roots(1, lo, hi)).to(dev()))
    r = ref.decode(*(x.view(torch.uint8).cpu().numpy() for x in (c, s)))
    assert r[r > 0].min() >= 2.0 ** -71 and r.max() < 2.0 ** 64
    v = fp.mx8_dequantize(c, s, root=True)
    np.testing.assert_array_equal(v.cpu().numpy(), r * r)
    c2, s2 = fp.mx8_quantize(v, root=True)
    assert torch.equal(c2.view(torch.uint8), c.view(torch.uint8)) and torch.equal(s2.view(torch.uint8), s.view(torch.uint8))


@pytest.mark.parametrize("lo,hi", [(-149, -120), (-100, -72), (64, 90), (100, 127.9), (-149, 127.9)])
def test_roots_come_back_at_every_magnitude(fp, lo, hi):
    """Where a second moment would leave fp32's range, its root does not."""
    say("roots", lo, hi)
    c, s = fp.mx8_quantize(torch.from_numpy(roots(2, lo, hi)).to(dev()))
    r = fp.mx8_dequantize(c, s)
    c2, s2 = fp.mx8_quantize(r)
    assert torch.equal(c2.view(torch.uint8), c.view(torch.uint8)) and torch.equal(s2.view(torch.uint8), s.view(torch.uint8))
    with np.errstate(over="ignore", under="ignore"):
        want = np.square(r.cpu().numpy())
    np.testing.assert_array_equal(fp.mx8_dequantize(c, s, root=True).cpu().numpy(), want)


@pytest.mark.parametrize("sigma", [1e-30, 1e-3, 1e25])
def test_a_checkpoint_in_fp32(fp, sigma):
    """Moments of an 8-bit run as fp32, cut for three ranks, joined and taken back
    into 8 bits, where the second moments themselves have left fp32's range too."""
    say("checkpoint", sigma)
    case = Case(fp, [4096, 96], grad="f32", copy=None, bits=8, warm=False, grad_sigma=sigma)
    for t in range(1, 5):
        run(case, t, seed=t)
    P = case.plan.partition
    for codes, scales in (case.moments[:2], case.moments[2:]):
        x = fp.mx8_dequantize(codes, scales)
        cut = fp.ReshardPlan(P, 1, 3).reshard([x])
        back = fp.ReshardPlan(P, 3, 1).reshard(list(cut.split(cut.numel() // 3)))[:P]
        c, s = fp.mx8_quantize(back)
        y = fp.mx8_dequantize(c, s)
        top = ref.decode(codes.cpu().numpy() & 0x7F, np.full(P // 32, 127, np.uint8)).reshape(-1, 32).max(1)
        same = torch.from_numpy(np.repeat(top < 256, 32)).to(dev())
        assert torch.equal(y[same], x[same]) and bool(same.float().mean() > 0.8) and bool((x != 0).any())
        lost = (x != y) & (x.abs() >= 2.0 ** -13 * x.abs().view(-1, 32).amax(1).repeat_interleave(32))
        assert not bool(lost.any())


def test_backward_through_stepped_weights_raises(fp):
    """As after a torch optimizer: autograd sees that a weight or a copy that it
    kept for a backward pass has changed."""
    say("versions")
    for bits in (32, 8):
        flat = torch.randn(96, device=dev())
        weights = [torch.nn.Parameter(torch.randn(64, device=dev())), torch.nn.Parameter(flat[:32].view(4, 8)), flat[32:]]
        copies = [w.detach().bfloat16() for w in weights]
        x = [torch.randn_like(w, requires_grad=True) for w in weights]
        plan = fp.Params([torch.ones_like(w) for w in weights], weights, copies)
        mom = plan.new_moments(bits)
        sq, ws = torch.zeros(1, dtype=torch.float64, device=dev()), plan.new_workspace()
        for kept in weights + copies:
            y = [x[i].to(kept.dtype) * kept for i in range(3) if x[i].shape == kept.shape][0].sum()
            plan.grad_norm(sq, ws)
            y.backward(retain_graph=True)
            plan.step(mom, step=1, seed=1 if bits == 8 else None, **HPS[0])
            with pytest.raises(RuntimeError, match="inplace"):
                y.backward()
        with torch.inference_mode():
            w = torch.zeros(8, device=dev())
            fp.Params([torch.ones_like(w)], [w]).step([torch.zeros(32, device=dev()) for _ in range(2)], step=1, **HPS[0])
        assert bool((w < 0).all())


def test_a_refused_rate_does_not_stay(fp):
    say("refused rate")
    w = [torch.ones(64, device=dev()) for _ in range(2)]
    g = torch.randn(64, device=dev())
    steps = []
    for x in w:
        plan = fp.Params([g], [x])
        steps.append(plan.stepper(plan.new_moments(), **HPS[0]))
    for bad in (math.nan, math.inf):
        with pytest.raises(fp.FlatParamError, match="finite"):
            steps[0](1, lr=bad)
    steps[0](1)
    steps[1](1)
    assert torch.equal(w[0], w[1]) and not torch.equal(w[0], torch.ones_like(w[0]))
    steps[0](2, lr=0.5)   # one that is taken stays
    steps[0](3)
    steps[1](2, lr=0.5)
    steps[1](3, lr=0.5)
    assert torch.equal(w[0], w[1])


def test_a_gradient_that_is_not_there(fp):
    say("no gradient")
    t = [torch.zeros(8, device=dev()) for _ in range(4)]
    for grads, master, copies, match in (([t[0], None], t[2:], None, r"grads\[1\] is None"),
                                         (t[:2], [t[2], None], None, r"master\[1\] is None"),
                                         (t[:2], t[2:], [None, None], r"copies\[0\] is None")):
        with pytest.raises(TypeError, match=match):
            fp.Params(grads, master, copies)
    plan = fp.Params(t[:2], t[2:])
    with pytest.raises(TypeError, match=r"grads\[1\] is None"):
        plan.set_grads([t[0], None])


@pytest.mark.parametrize("copy", ["bf16", "f16", None])
@pytest.mark.parametrize("bits,first", [(8, 3_000_000), (32, 4_000_000)])
def test_larger_plans(fp, bits, first, copy):
    """Plans of the sizes at which waves take whole tiles (8-bit moments) and at
    which fewer workgroups are resident (fp32 moments), with every kind of copy."""
    say("larger", bits, copy)
    for shift in (0, 1):
        case = Case(fp, [first, 5, 70_001, 512, 0, 515, 3], "bf16" if copy != "f16" else "f16", copy, bits, shift, seed=3)
        for t in (1, 7):
            before = case.host()
            run(case, t, seed=t)
            case.check(before, t, t, what=f"{copy} {bits} bits shift {shift} step {t}")
