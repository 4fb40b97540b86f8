"""The optimizer step over many separate tensors on the GPU against the numpy
reference (params_ref.py, which derives the tolerances)."""

import math
import os

import numpy as np
import pytest
import torch

import params_ref as ref
from conftest import ROOT
from gpu_common import dev, norm_rel_tol, say

pytestmark = pytest.mark.gpu

HPS = [dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01),
       dict(lr=3e-4, beta1=0.8, beta2=0.95, eps=1e-6, weight_decay=0.0)]
GRAD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {
    "one": [1],
    "small": [8, 0, 1, 31, 32, 33, 3, 0, 64],
    "edges": [1023, 1024, 1025, 4, 2047, 4097, 5],
    "ragged": [100_003, 1, 17, 65_536, 12_345, 40],
}


def columns(hps):
    return {k: [h[k] for h in hps] for k in hps[0]}


class Case:
    """Tensors of `sizes` as views of dense buffers with canaries around each
    buffer; `shift` elements off the buffers' alignment."""

    def __init__(self, fp, sizes, grad="bf16", copy="bf16", bits=32, shift=0, seed=0, groups=True, grad_sigma=1e-3,
                 warm=True):
        r = np.random.default_rng(seed)
        self.sizes, self.n, self.bits = sizes, sum(sizes), bits
        g = torch.Generator().manual_seed(seed)

        def buf(x, fill):
            pad = torch.full((64,), fill, dtype=x.dtype)
            whole = torch.cat([pad[:16 + shift], x, pad]).to(dev())
            return whole, whole[16 + shift:16 + shift + x.numel()]

        n = self.n
        live = torch.rand(n, generator=g) > 0.2
        grads = (torch.randn(n, generator=g) * grad_sigma * live).to(GRAD[grad])
        master = torch.randn(n, generator=g) * 0.02
        self.whole = {}
        self.whole["grad"], self.grad = buf(grads, 7.0)
        self.whole["master"], self.master = buf(master, 7.0)
        self.copy = None
        if copy:
            self.whole["copy"], self.copy = buf(torch.full((n,), 5.0).to(GRAD[copy]), 7.0)
        self.groups = [i % 2 for i in range(len(sizes))] if groups else [0] * len(sizes)
        self.plan = fp.Params(self.grad.split(sizes), self.master.split(sizes),
                              self.copy.split(sizes) if copy else None, groups=self.groups)
        P = self.plan.partition
        assert P == sum(-(-s // 32) * 32 for s in sizes)
        assert self.plan.offsets == [sum(-(-s // 32) * 32 for s in sizes[:i]) for i in range(len(sizes))]
        # the gaps of the partition hold a pattern that has to stay
        self.at = np.concatenate([np.arange(o, o + s) for o, s in zip(self.plan.offsets, sizes)]).astype(np.int64)
        m = np.full(P, 0.5, np.float32)
        v = np.full(P, 0.25, np.float32)
        keep = live.numpy() & warm
        m[self.at] = r.standard_normal(n).astype(np.float32) * 1e-4 * keep
        v[self.at] = np.square(r.standard_normal(n).astype(np.float32) * 1e-3) * keep
        if bits == 32:
            host = [m, v]
        else:
            host = []
            for x, root in ((m, False), (np.sqrt(v.astype(np.float64)).astype(np.float32), True)):
                real = np.zeros_like(x)
                real[self.at] = x[self.at]
                s = ref.scale_bytes(real)
                c = np.full(P, 0x5A, np.uint8)
                c[self.at] = ref.encode(real, s, root=root)[self.at]
                host += [c, s]
        self.moments = [torch.from_numpy(x).to(dev()) for x in host]
        self.hps = HPS[:self.plan.n_groups]

    def host(self):
        f = lambda t: t.detach().float().cpu().numpy()  # noqa: E731
        return dict(grad=f(self.grad), master=f(self.master), moments=[x.cpu().numpy().copy() for x in self.moments])

    def tensors(self):
        at = 0
        for i, s in enumerate(self.sizes):
            yield i, s, slice(at, at + s), self.plan.offsets[i]
            at += s

    def check(self, before, t, seed=None, coef=1.0, skipped=False, what=""):
        """The step from `before` gave what is there now."""
        after = self.host()
        for i, s, d, o in self.tensors():
            if s == 0:
                continue
            hp = self.hps[self.groups[i]]
            where = f"{what} tensor {i} of {s}"
            if skipped:
                np.testing.assert_array_equal(after["master"][d], before["master"][d], err_msg=where)
                continue
            p, b = slice(o, o + s), slice(o // 32, o // 32 + -(-s // 32))
            old = before["moments"]
            if self.bits == 32:
                m0, v0 = old[0][p], old[1][p]
            else:
                m0 = ref.decode(old[0][p], old[1][b])
                v0 = ref.decode(old[2][p], old[3][b]) ** 2
            th, m, v, terms, change = ref.adamw(before["grad"][d], before["master"][d], m0, v0, hp, t, coef)
            ref.near(after["master"][d], th, terms, where + " weights", change if self.bits == 8 else 0.0)
            new = after["moments"]
            if self.bits == 32:
                g = np.abs(before["grad"][d].astype(np.float64) * coef)
                ref.near(new[0][p], m, np.abs(m0) + g, where + " first moment")
                ref.near(new[1][p], v, None, where + " second moment")
            else:
                dm, dr = ref.dither(np.arange(o, o + s), seed)
                ref.check_mx8(new[0][p], new[1][b], m, dm, what=where + " first moment")
                ref.check_mx8(new[2][p], new[3][b], np.sqrt(v), dr, root=True, what=where + " root")
        if skipped:
            for x, y in zip(after["moments"], before["moments"]):
                np.testing.assert_array_equal(x, y, err_msg=what)
        gap = np.ones(self.plan.partition, bool)
        gap[self.at] = False
        for x, y in zip(after["moments"], before["moments"]):
            if x.size == gap.size:
                np.testing.assert_array_equal(x[gap], y[gap], err_msg=what + " gaps of the partition")
        if self.copy is not None:
            assert torch.equal(self.copy, self.master.to(self.copy.dtype)), what + " copies"
        for k, w in self.whole.items():
            edge = torch.cat([w[:w.numel() - 64 - self.n], w[-64:]])
            assert (edge == 7.0).all(), f"{what}: written past {k}"


def run(case, t, seed, **kw):
    case.plan.step(case.moments, step=t, seed=seed if case.bits == 8 else None, **columns(case.hps), **kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad,copy", [("bf16", "bf16"), ("f32", None), ("f16", "f16"), ("f32", "bf16"), ("bf16", None)])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_steps(fp, sizes, grad, copy, bits):
    for shift in (0, 1, 3):
        say("step", sizes, grad, copy, bits, "shift", shift)
        case = Case(fp, SIZES[sizes], grad, copy, bits, shift, seed=shift)
        for t in (1, 2, 50):
            before = case.host()
            run(case, t, seed=1000 + t)
            case.check(before, t, 1000 + t, what=f"{sizes} {grad} {copy} {bits} bits shift {shift} step {t}")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("flag", [0, 1, 2, 3])
def test_overflow_skips(fp, bits, flag):
    say("skip", bits, flag)
    case = Case(fp, SIZES["edges"] + SIZES["small"], bits=bits, shift=1)
    case.grad[5] = math.inf
    found = torch.tensor([flag], dtype=torch.int32, device=dev())
    coef = torch.tensor([0.125], dtype=torch.float64, device=dev())
    if flag == 0:
        case.grad[5] = 0.25
    before = case.host()
    run(case, 3, 17, found_inf=found, grad_coef=coef)
    case.check(before, 3, 17, coef=0.125, skipped=flag != 0, what=f"flag {flag}")
    assert int(found) == flag


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sigma", [1e-30, 1e-20, 1e-12, 1.0, 1e15])
def test_far_magnitudes(fp, bits, sigma):
    """Gradients whose squares leave fp32's range: 8-bit moments keep the root."""
    say("magnitude", bits, sigma)
    if bits == 32 and sigma in (1e-30, 1e-20):
        sigma = 1e-15
    case = Case(fp, [1000, 33], grad="f32", copy=None, bits=bits, grad_sigma=sigma, warm=False)
    for t in (1, 2):
        before = case.host()
        run(case, t, seed=t)
        case.check(before, t, t, what=f"sigma {sigma} step {t}")
    if bits == 8:
        root = case.moments[2].cpu().numpy()[case.at]
        m = case.moments[0].cpu().numpy()[case.at] & 0x7F
        assert not ((m > 0) & (root == 0)).any(), "a moment without a root"


@pytest.mark.parametrize("grad", list(GRAD))
@pytest.mark.parametrize("room", [4_000_000, 46_000_000])
def test_large_plans_step_small_tensors_alike(fp, room, grad):
    """Plans split their work by their size (below 3, up to 46 million elements,
    above): the tensors in front of a large one come out bit for bit as in a
    small plan."""
    sizes = SIZES["edges"] + SIZES["small"] + SIZES["ragged"] + [3, 515, 256, 300]
    say("large plan", room, grad)
    small = Case(fp, sizes, grad=grad, copy="f16", bits=8, shift=1)
    before = small.host()
    run(small, 5, seed=5)
    small.check(before, 5, 5, what="small plan")
    n = room - small.plan.partition + 1
    twin = Case(fp, sizes, grad=grad, copy="f16", bits=8, shift=1)
    big = [torch.zeros(n, dtype=t.dtype, device=dev()) for t in (twin.grad, twin.master, twin.copy)]
    big[0][-70:] = 0.5
    plan = fp.Params([*twin.grad.split(sizes), big[0]], [*twin.master.split(sizes), big[1]],
                     [*twin.copy.split(sizes), big[2]], groups=twin.groups + [0])
    P = twin.plan.partition
    assert plan.partition >= room and plan.offsets[:-1] == twin.plan.offsets and plan.offsets[-1] == P
    mom = [x.view(torch.uint8) for x in plan.new_moments(8)]
    for x, y in zip(mom, twin.moments):
        x[:y.numel()] = y
    plan.step(mom, step=5, seed=5, **columns(small.hps))
    torch.cuda.synchronize()
    assert torch.equal(twin.master, small.master) and torch.equal(twin.copy, small.copy)
    for x, y in zip(mom, small.moments):
        assert torch.equal(x[:y.numel()], y)
    # the large tensor's last elements, up to a last part of a quad
    o, g = P + n - 70, np.full(70, 0.5, np.float32)
    th, m, v, terms, change = ref.adamw(g, np.zeros(70, np.float32), np.zeros(70), np.zeros(70), HPS[0], 5)
    ref.near(big[1][-70:].cpu().numpy(), th, terms, "last weights", change)
    assert not big[1][:-70].any() and torch.equal(big[2], big[1].half())
    first = -(-o // 32) * 32                                  # the first whole block of them
    k = P + n - first
    dm, dr = ref.dither(np.arange(first, first + k), 5)
    b = slice(first // 32, first // 32 + -(-k // 32))
    ref.check_mx8(mom[0][first:P + n].cpu().numpy(), mom[1][b].cpu().numpy(), m[-k:], dm, what="last first moments")
    ref.check_mx8(mom[2][first:P + n].cpu().numpy(), mom[3][b].cpu().numpy(), np.sqrt(v[-k:]), dr, root=True, what="last roots")


def test_zero_gradients_leave_zero_moments(fp):
    say("zero gradients")
    for bits in (32, 8):
        case = Case(fp, [1000], bits=bits, warm=False, grad_sigma=0.0)
        before = case.host()
        run(case, 1, seed=1)
        case.check(before, 1, 1, what="zeros")
        for k, x in enumerate(case.moments):
            x = x.cpu().numpy()
            if bits == 8 and k % 2:
                assert (x == 0).all()
            elif bits == 8:  # zeros of either sign
                assert (x[case.at] & 0x7F == 0).all()
            else:
                assert (x[case.at] == 0).all()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_gradient_that_is_not_finite_without_a_flag(fp, bad):
    """8-bit moments: its block reads as NaN, the others are as they would be."""
    say("not finite", bad)
    case = Case(fp, [200, 40], grad="bf16", copy="bf16", bits=8)
    case.grad[70] = bad
    before = case.host()
    run(case, 2, seed=9)
    m, ms, r, rs = (x.cpu().numpy() for x in case.moments)
    assert ms[2] == 255 and rs[2] == 255 and (m[64:96] == 0).all() and (r[64:96] == 0).all()
    assert np.isnan(ref.decode(m, ms)[64:96]).all()
    assert (np.delete(ms, 2) != 255).all() and (np.delete(rs, 2) != 255).all()
    assert bool(torch.isnan(case.master[70])) and int(torch.isnan(case.master).sum()) == 1
    other = Case(fp, [200, 40], grad="bf16", copy="bf16", bits=8)
    run(other, 2, seed=9)
    keep = np.ones(case.plan.partition, bool)
    keep[64:96] = False
    np.testing.assert_array_equal(m[keep], other.moments[0].cpu().numpy()[keep])
    np.testing.assert_array_equal(r[keep], other.moments[2].cpu().numpy()[keep])
    # the next step on the block: still NaN, its neighbours live
    case.grad[70] = 0.5
    run(case, 3, seed=10)
    assert int(torch.isnan(case.master).sum()) == 32


def test_stochastic_rounding_lets_moments_decay(fp):
    """Without gradients r falls by sqrt(beta2) a step in the mean, though every
    step is below half a code.  64 Ki elements of one value, 400 steps: r has
    decayed to exp(-0.2002) of its value.  A rounding's variance is at most
    q delta (q a code's width, delta the step's change), summed over the steps
    at most q (1 - exp(-0.2)) r with q <= r / 8 of the largest value: the
    mean's deviation is below sqrt(0.023 / 65536) = 6e-4, six of them 0.0036."""
    say("decay")
    n = 1 << 16
    g = torch.zeros(n, device=dev())
    w = torch.ones(n, device=dev())
    plan = fp.Params([g], [w])
    mom = plan.new_moments(8)
    fp.mx8_quantize(torch.full((n,), 1e-4, device=dev()), mom[0], mom[1])
    fp.mx8_quantize(torch.full((n,), 1.0, device=dev()), mom[2], mom[3], root=True)
    step = plan.stepper(mom, lr=0.0, beta1=0.999, beta2=0.999, eps=1e-8, weight_decay=0.0)
    m0, r0 = (float(fp.mx8_dequantize(mom[k], mom[k + 1]).mean()) for k in (0, 2))
    for t in range(1, 401):
        step(t, seed=t)
    m, r = (float(fp.mx8_dequantize(mom[k], mom[k + 1]).double().mean()) for k in (0, 2))
    assert abs(r / r0 - 0.999 ** 200) < 0.0036
    # m decays twice as fast: sqrt(0.041 / 65536) * 6
    assert abs(m / m0 - 0.999 ** 400) < 0.0048


@pytest.mark.parametrize("grad", list(GRAD))
@pytest.mark.parametrize("sizes", list(SIZES))
def test_norm(fp, sizes, grad):
    for shift in (0, 1):
        say("norm", sizes, grad, shift)
        case = Case(fp, SIZES[sizes], grad=grad, shift=shift, grad_sigma=0.5)
        sq = torch.full((1,), -1.0, dtype=torch.float64, device=dev())
        ws = case.plan.new_workspace()
        found = torch.zeros(1, dtype=torch.int32, device=dev())
        want = float(np.square(case.host()["grad"].astype(np.float64)).sum())
        first = None
        for _ in range(3):
            case.plan.grad_norm(sq, ws, found)
            assert abs(float(sq) - want) <= norm_rel_tol(case.n) * want
            first = float(sq) if first is None else first
            assert float(sq) == first and int(found) == 0
        case.plan.grad_norm(sq, ws)  # no flag wanted
        for i, s, d, _ in case.tensors():
            for at in {d.start, d.stop - 1, (d.start + d.stop) // 2} if s else ():
                for bad in (math.inf, -math.inf, math.nan):
                    old = case.grad[at].clone()
                    case.grad[at] = bad
                    found.fill_(2)
                    case.plan.grad_norm(sq, ws, found)
                    assert int(found) == 3 and not math.isfinite(float(sq)), f"tensor {i} element {at - d.start}"
                    case.grad[at] = old
        found.fill_(2)
        case.plan.grad_norm(sq, ws, found)
        assert int(found) == 2 and float(sq) == first


def test_norm_of_many_workgroups_again_and_again(fp):
    """Gradients doubled from call to call, the calls back to back on one
    workspace: doubling is exact, so every sum is four times the one before,
    bit for bit; a partial sum of an earlier call would show."""
    say("norm again and again")
    sizes = [6_000_000, 3, 1_000_001, 70_000]
    g = torch.randn(sum(sizes), device=dev()) * 1e-3
    plan = fp.Params(g.split(sizes))
    ws = plan.new_workspace()
    found = torch.zeros(1, dtype=torch.int32, device=dev())
    sq = torch.zeros(40, dtype=torch.float64, device=dev())
    for k in range(40):
        plan.grad_norm(sq[k:k + 1], ws, found)
        g.mul_(2.0)
    sq = sq.cpu().numpy()
    want = float((g.double() * 2.0 ** -40).square().sum())
    assert abs(sq[0] - want) <= norm_rel_tol(g.numel()) * want
    np.testing.assert_array_equal(sq, sq[0] * 4.0 ** np.arange(40))
    assert int(found) == 0


def test_norm_only_plan_and_empty_tensors(fp):
    say("empty")
    g = [torch.empty(0, device=dev()), torch.empty(0, device=dev())]
    plan = fp.Params(g)
    sq = torch.full((1,), -1.0, dtype=torch.float64, device=dev())
    plan.grad_norm(sq, plan.new_workspace())
    assert float(sq) == 0.0 and plan.partition == 0
    plan = fp.Params([torch.full((3,), 2.0, device=dev()), g[0]])
    plan.grad_norm(sq, plan.new_workspace())
    assert float(sq) == 12.0
    with pytest.raises(fp.FlatParamError, match="no master"):
        plan.step(plan.new_moments(), step=1, **HPS[0])
    plan = fp.Params(g, [torch.empty(0, device=dev()) for _ in g])
    plan.step(plan.new_moments(), step=1, **HPS[0])
    plan.step(plan.new_moments(8), step=1, seed=0, **HPS[0])


def test_shared_gradients(fp):
    """One gradient for two tensors (read only), and gradients that overlap."""
    say("shared gradients")
    g = torch.randn(1000, device=dev())
    w = [torch.ones(600, device=dev()) for _ in range(3)]
    plan = fp.Params([g[:600], g[:600], g[400:]], w)
    plan.step(plan.new_moments(), step=1, **HPS[0])
    assert torch.equal(w[0], w[1]) and torch.equal(w[0][400:], w[2][:200]) and not torch.equal(w[0], w[2])


def test_bf16_as_bits(fp):
    """bf16 gradients and copies in 16-bit integer tensors, as elsewhere here."""
    say("bits")
    g = (torch.randn(1000, device=dev()) * 1e-3).bfloat16()
    w = [torch.ones(1000, device=dev()) for _ in range(2)]
    c = [torch.zeros(1000, dtype=d, device=dev()) for d in (torch.bfloat16, torch.int16)]
    for x, k in ((g, 0), (g.view(torch.int16), 1)):
        plan = fp.Params([x], [w[k]], [c[k]])
        plan.step(plan.new_moments(8), step=1, seed=1, **HPS[0])
    assert torch.equal(w[0], w[1]) and torch.equal(c[0].view(torch.int16), c[1]) and not torch.equal(w[0], torch.ones_like(w[0]))
    with pytest.raises(TypeError):
        fp.Params([g], [w[0]], [w[1]])


def test_new_gradients(fp):
    say("set_grads")
    for bits in (32, 8):
        case = Case(fp, SIZES["edges"], bits=bits, grad="f32")
        a, b = Case(fp, SIZES["edges"], grad="f32", seed=5), Case(fp, SIZES["edges"], grad="f32", seed=6)
        for t, other in ((1, a), (2, b), (3, a)):
            case.plan.set_grads(other.grad.split(case.sizes))
            before = dict(case.host(), grad=other.grad.cpu().numpy())
            run(case, t, seed=t)
            case.check(before, t, t, what=f"set_grads {t}")
        sq = torch.zeros(1, dtype=torch.float64, device=dev())
        case.plan.grad_norm(sq, case.plan.new_workspace())
        want = float(a.grad.double().square().sum())
        assert abs(float(sq) - want) <= norm_rel_tol(case.n) * want
        with pytest.raises(ValueError, match="elements"):
            case.plan.set_grads(a.grad.split(list(reversed(case.sizes))))
        with pytest.raises(TypeError):
            case.plan.set_grads(a.grad.bfloat16().split(case.sizes))
        with pytest.raises(fp.FlatParamError, match="overlaps"):
            case.plan.set_grads(case.master.split(case.sizes))
    # moments may not overlap the gradients of now, but those of before
    w, (old, new) = torch.zeros(64, device=dev()), (torch.zeros(64, device=dev()) for _ in range(2))
    plan, other = fp.Params([old], [w]), torch.zeros(64, device=dev())
    with pytest.raises(fp.FlatParamError, match="overlaps a gradient"):
        plan.step([old, other], step=1, **HPS[0])
    plan.set_grads([new])
    plan.step([old, other], step=1, **HPS[0])
    plan.set_grads([old])
    with pytest.raises(fp.FlatParamError, match="overlaps a gradient"):
        plan.step([old, other], step=1, **HPS[0])


def test_groups_without_a_tensor_and_a_changed_rate(fp):
    """More groups than this rank holds tensors of, and a new rate per call."""
    say("groups")
    for bits in (32, 8):
        case = Case(fp, SIZES["edges"], bits=bits, groups=False)
        three = columns([HPS[0], HPS[1], HPS[1]])
        step = case.plan.stepper(case.moments, **three)
        before = case.host()
        step(2, **({"seed": 2} if bits == 8 else {}))
        case.check(before, 2, 2, what="three groups")
        before = case.host()
        step(3, lr=[0.25, 0.0, 0.0], **({"seed": 3} if bits == 8 else {}))
        case.hps = [dict(HPS[0], lr=0.25)]
        case.check(before, 3, 3, what="new rate")
        before = case.host()
        step(4, lr=0.5, **({"seed": 4} if bits == 8 else {}))
        case.hps = [dict(HPS[0], lr=0.5)]
        case.check(before, 4, 4, what="new rate for all")


def test_refused_steps(fp):
    say("refusals")
    case = Case(fp, SIZES["edges"], bits=8)
    P, kw = case.plan.partition, columns(case.hps)
    c8, c32 = case.plan.new_moments(8), case.plan.new_moments(32)
    with pytest.raises(ValueError, match="seed"):
        case.plan.step(c8, step=1, **kw)
    with pytest.raises(ValueError, match="seed"):
        case.plan.step(c32, step=1, seed=1, **kw)
    with pytest.raises(ValueError, match="moments"):
        case.plan.step(c32[:1], step=1, **kw)
    with pytest.raises(ValueError, match="needs"):
        case.plan.step([x[:-1] for x in c32], step=1, **kw)
    with pytest.raises(TypeError):
        case.plan.step([x.half() for x in c32], step=1, **kw)
    with pytest.raises(ValueError, match="groups"):
        case.plan.step(c32, step=1, **dict(kw, lr=[1e-3]))
    with pytest.raises(ValueError, match="groups"):
        case.plan.step(c32, step=1, **dict(kw, lr=[1e-3] * 3))
    with pytest.raises(ValueError, match="groups"):
        case.plan.stepper(c32, **kw)(1, lr=[1e-3])
    with pytest.raises(fp.FlatParamError, match="n_groups"):
        case.plan.step(c32, step=1, **dict.fromkeys(kw, [0.5] * 17))
    for bad, match in ((dict(step=0), "step"), (dict(step=1, lr=[1.0, math.nan]), "finite"),
                       (dict(step=1, beta1=[0.9, 1.0]), "betas"), (dict(step=1, eps=[0.0, -1.0]), "eps")):
        with pytest.raises(fp.FlatParamError, match=match):
            case.plan.step(c32, **dict(dict(kw, step=1), **bad))
    with pytest.raises(fp.FlatParamError, match="overlaps"):
        case.plan.step([c32[0], c32[0]], step=1, **kw)
    big = torch.zeros(P + 8, device=dev())
    with pytest.raises(fp.FlatParamError, match="aligned"):
        case.plan.step([big[1:], c32[1]], step=1, **kw)
    with pytest.raises(fp.FlatParamError, match="overlaps"):
        case.plan.step([c8[0], c8[0].view(torch.uint8)[:P // 32], c8[2], c8[3]], step=1, seed=1, **kw)
    L = fp.lib()
    hp = (fp._lib.fp_adamw_hparams * 2)(*[fp._lib.fp_adamw_hparams(1e-3, 0.9, 0.999, 1e-8, 0.0, 1)] * 2)
    h, p = case.plan._h, [x.data_ptr() for x in c32]
    assert L.fp_params_adamw(h, 1, hp, *p, None, None, None) == -2      # the tensors use two groups
    assert L.fp_params_adamw(h, 17, hp, *p, None, None, None) == -2
    assert L.fp_params_adamw(h, 2, None, *p, None, None, None) == -1
    assert L.fp_params_adamw(h, 2, hp, None, p[1], None, None, None) == -1
    assert L.fp_params_adamw(h, 2, hp, *p, p[0] + 2, None, None) == -3
    assert L.fp_params_adamw(h, 2, hp, *p, None, p[0] + 4, None) == -3
    q = [x.data_ptr() for x in c8]
    for k in range(4):
        assert L.fp_params_adamw8(h, 2, hp, *q[:k], None, *q[k + 1:], 1, None, None, None) == -1
    sq = torch.zeros(2, dtype=torch.float64, device=dev())
    ws = case.plan.new_workspace()
    assert L.fp_params_grad_norm(h, None, None, ws.data_ptr(), None) == -1
    assert L.fp_params_grad_norm(h, None, sq.data_ptr(), None, None) == -1
    assert L.fp_params_grad_norm(h, None, sq.data_ptr() + 4, ws.data_ptr(), None) == -3
    assert L.fp_params_grad_norm(h, ws.data_ptr() + 2, sq.data_ptr(), ws.data_ptr(), None) == -3
    assert L.fp_params_offsets(h, None) == -1
    case.grad.requires_grad_(False)
    t = torch.zeros(4, 4, device=dev())
    with pytest.raises(ValueError, match="contiguous"):
        fp.Params([t.t()[:2]], [torch.zeros(8, device=dev())])
    with pytest.raises(ValueError, match="elements"):
        fp.Params([t], [torch.zeros(8, device=dev())])
    with pytest.raises(TypeError):
        fp.Params([t.double()], [t])
    with pytest.raises(TypeError):
        fp.Params([t], [t.half()])
    with pytest.raises(ValueError, match="groups"):
        fp.Params([t], [torch.zeros(16, device=dev())], groups=[0, 1])


@pytest.mark.parametrize("n", [1, 4, 5, 31, 32, 33, 1023, 1024, 1025, 70_001])
@pytest.mark.parametrize("root", [False, True])
def test_mx8(fp, n, root):
    say("mx8", n, root)
    r = np.random.default_rng(n)
    x = (r.standard_normal(n) * np.exp2(r.integers(-40, 40, n))).astype(np.float32)
    x[r.random(n) < 0.1] = 0.0
    x[r.random(n) < 0.05] = -0.0
    if root:
        x = np.abs(x) if n != 5 else x * x
    t = torch.from_numpy(x).to(dev())
    blocks = -(-n // 32)
    # canaries past both ends of the codes and scales
    codes = torch.full((n + 64,), 0x5A, dtype=torch.uint8, device=dev())
    scales = torch.full((blocks + 2,), 0x5A, dtype=torch.uint8, device=dev())
    fp.mx8_quantize(t, codes[16:16 + n], scales[1:1 + blocks], root=root)
    c, s = codes[16:16 + n].cpu().numpy(), scales[1:1 + blocks].cpu().numpy()
    v = np.sqrt(x.astype(np.float64)) if root else x.astype(np.float64)
    ref.check_mx8(c, s, v, root=root, what=f"quantize {n}")
    assert (codes[:16] == 0x5A).all() and (codes[16 + n:] == 0x5A).all() and scales[0] == 0x5A and scales[-1] == 0x5A
    out = torch.full((n + 8,), 7.0, device=dev())
    fp.mx8_dequantize(codes[16:16 + n], scales[1:1 + blocks], out[:n], root=root)
    want = ref.decode(c, s)
    want = want * want if root else want
    np.testing.assert_array_equal(out[:n].cpu().numpy(), want.astype(np.float32))
    assert (out[n:] == 7.0).all()
    if not root:  # what MXFP8 holds comes back as it is
        c2, s2 = fp.mx8_quantize(out[:n].clone())
        assert torch.equal(fp.mx8_dequantize(c2, s2), out[:n])


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_mx8_of_what_is_not_finite(fp, bad):
    say("mx8 not finite", bad)
    x = torch.linspace(0.1, 1.0, 100, device=dev())
    x[40] = bad
    for root in (False, True):
        c, s = fp.mx8_quantize(x, root=root)
        y = fp.mx8_dequantize(c, s, root=root)
        assert bool(torch.isnan(y[32:64]).all()) and int(torch.isnan(y).sum()) == 32
    codes = torch.arange(256, dtype=torch.uint8, device=dev())
    scales = torch.arange(8, dtype=torch.uint8, device=dev()) * 36
    with np.errstate(over="ignore"):
        want = ref.decode(codes.cpu().numpy(), scales.cpu().numpy()).astype(np.float32)
    np.testing.assert_array_equal(fp.mx8_dequantize(codes, scales).cpu().numpy(), want)
    scales[:] = 255
    assert bool(torch.isnan(fp.mx8_dequantize(codes, scales)).all())


def test_on_another_stream(fp):
    say("stream")
    case = Case(fp, SIZES["ragged"], bits=8)
    before = case.host()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sq = torch.zeros(1, dtype=torch.float64, device=dev())
    ws = case.plan.new_workspace()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            torch.cuda._sleep(100_000)
        case.plan.grad_norm(sq, ws)
        case.plan.step(case.moments, step=4, seed=4, **columns(case.hps))
    s.synchronize()
    case.check(before, 4, 4, what="other stream")
    want = float(np.square(before["grad"].astype(np.float64)).sum())
    assert abs(float(sq) - want) <= norm_rel_tol(case.n) * want


@pytest.mark.parametrize("bits", [32, 8])
def test_two_at_once(fp, bits):
    """Norm, factor and step on two streams at once, each with a plan, moments and
    a workspace of its own: as one after the other."""
    say("two at once", bits)
    sizes = [700_001, 33, 4097, 250_000]
    pair, twin = ([Case(fp, sizes, bits=bits, seed=k) for k in (1, 2)] for _ in range(2))
    streams = [torch.cuda.Stream() for _ in pair]

    def calls(c):
        sq, coef = (torch.zeros(1, dtype=torch.float64, device=dev()) for _ in range(2))
        found = torch.zeros(1, dtype=torch.int32, device=dev())
        ws = c.plan.new_workspace()
        step = c.plan.stepper(c.moments, found_inf=found, grad_coef=coef, **columns(c.hps))

        def once(t):
            c.plan.grad_norm(sq, ws, found)
            fp.grad_coef(coef, sq_norm=sq, max_norm=0.3)
            step(t, **({"seed": t} if bits == 8 else {}))
        return once

    both = [calls(c) for c in pair]
    torch.cuda.synchronize()
    for t in range(1, 21):
        for s, f in zip(streams, both):
            with torch.cuda.stream(s):
                f(t)
    torch.cuda.synchronize()
    for c, d in zip(pair, twin):
        f = calls(d)
        for t in range(1, 21):
            f(t)
        torch.cuda.synchronize()
        assert torch.equal(c.master, d.master) and torch.equal(c.copy, d.copy)
        assert all(torch.equal(x, y) for x, y in zip(c.moments, d.moments))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured(fp, bits):
    """Norm, factor and step in one graph, replayed with eager work between:
    every replay equals the eager calls from the same state, bit for bit."""
    say("captured", bits)
    case, twin = (Case(fp, SIZES["ragged"] + SIZES["small"], bits=bits, seed=3) for _ in range(2))
    state = []
    for c in (case, twin):
        found = torch.zeros(1, dtype=torch.int32, device=dev())
        sq, coef = (torch.zeros(1, dtype=torch.float64, device=dev()) for _ in range(2))
        state.append((found, sq, coef, c.plan.new_workspace(),
                      c.plan.stepper(c.moments, found_inf=found, grad_coef=coef, **columns(c.hps))))

    def once(c, k):
        found, sq, coef, ws, step = state[k]
        found.zero_()
        c.plan.grad_norm(sq, ws, found)
        fp.grad_coef(coef, sq_norm=sq, max_norm=0.05)
        step(7, **({"seed": 21} if bits == 8 else {}))

    keep = [t.clone() for t in (case.master, case.grad, *case.moments)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once(case, 0)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once(case, 0)
        with pytest.raises(fp.FlatParamError, match="captured"):
            case.plan.set_grads(case.grad.split(case.sizes))
    for t, k in zip((case.master, case.grad, *case.moments), keep):
        t.copy_(k)
    for i in range(6):
        for c in (case, twin):
            c.grad.copy_(keep[1] * (i + 1))
            if i == 3:
                c.grad[9] = math.inf
        graph.replay()
        once(twin, 1)
        torch.cuda.synchronize()
        assert int(state[0][0]) == int(state[1][0]) == (1 if i == 3 else 0)
        pairs = [(state[0][1], state[1][1]), (state[0][2], state[1][2]), (case.master, twin.master), (case.copy, twin.copy)]
        for x, y in pairs + list(zip(case.moments, twin.moments)):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)), f"replay {i}"
        torch.zeros(1 << 20, device=dev()).sum().item()
    # a replay reads the table that set_grads wrote last
    other = keep[1] * 0.5
    case.plan.set_grads(other.split(case.sizes))
    twin.plan.set_grads(other.split(case.sizes))
    graph.replay()
    once(twin, 1)
    torch.cuda.synchronize()
    assert torch.equal(state[0][1], state[1][1]) and torch.equal(case.master, twin.master)


def test_together_on_the_dim0_layout(fp):
    """A parameter group's dim-0 layout trained three steps with 8-bit moments:
    norm, scaler, clipping, step, unpack; then its moments out of 8 bits, cut for
    another rank count and back into 8 bits."""
    say("together")
    shapes, world, rank = [(40, 24), (40,), (7, 33), (129,), ()], 2, 1
    plan0 = fp.Shard0Plan(shapes, world)
    g = torch.Generator().manual_seed(4)
    full = [torch.randn(s, generator=g).to(dev()) * 0.02 for s in shapes]
    weights = plan0.pack(full)[rank * plan0.shard:(rank + 1) * plan0.shard].clone()
    low = torch.zeros(world * plan0.shard, dtype=torch.bfloat16, device=dev())
    own = low[rank * plan0.shard:(rank + 1) * plan0.shard]
    grads = torch.zeros(plan0.shard, dtype=torch.float16, device=dev())
    parts = [plan0.views(b, rank) for b in (grads, weights, own)]
    params = fp.Params(*parts, groups=[int(len(s) < 2) for s in shapes])
    mom = params.new_moments(8)
    found, clean = (torch.zeros(1, dtype=torch.int32, device=dev()) for _ in range(2))
    scale = torch.full((1,), 1024.0, device=dev())
    sq, coef = (torch.zeros(1, dtype=torch.float64, device=dev()) for _ in range(2))
    ws = params.new_workspace()
    hps = HPS
    step = params.stepper(mom, found_inf=found, grad_coef=coef, **columns(hps))
    t = 0
    for it in range(4):
        grads.copy_(torch.randn(plan0.shard, generator=g) * 1e-3 * float(scale))
        if it == 2:
            grads[3] = math.inf
        before = dict(weights=weights.cpu().numpy(), mom=[x.view(torch.uint8).cpu().numpy() for x in mom],
                      grads=grads.float().cpu().numpy())
        used = float(scale)
        found.zero_()
        params.grad_norm(sq, ws, found)
        fp.grad_coef(coef, sq_norm=sq, loss_scale=scale, max_norm=0.02)
        step(t + 1, seed=t + 1)
        fp.scaler_update(found, scale, clean, growth_interval=2)
        torch.cuda.synchronize()
        after = [x.view(torch.uint8).cpu().numpy() for x in mom]
        if it == 2:
            assert int(found) == 1 and float(scale) == used * 0.5
            np.testing.assert_array_equal(weights.cpu().numpy(), before["weights"])
            for x, y in zip(after, before["mom"]):
                np.testing.assert_array_equal(x, y)
            continue
        t += 1
        real = [p.reshape(-1).float().cpu().numpy() for p in plan0.views(torch.from_numpy(before["grads"]), rank)]
        norm = math.sqrt(sum(float(np.square(x.astype(np.float64)).sum()) for x in real)) / used
        k = min(1.0, 0.02 / (norm + 1e-6)) / used
        assert abs(float(coef) - k) <= 1e-12 * k
        w0 = plan0.views(torch.from_numpy(before["weights"]), rank)
        w1 = plan0.views(weights.cpu(), rank)
        for i, x in enumerate(real):
            o, n = params.offsets[i], params.sizes[i]
            p, b = slice(o, o + n), slice(o // 32, o // 32 + -(-n // 32))
            old, hp = before["mom"], hps[params.groups[i]]
            th, m, v, terms, change = ref.adamw(x, w0[i].reshape(-1).numpy(), ref.decode(old[0][p], old[1][b]),
                                        ref.decode(old[2][p], old[3][b]) ** 2, hp, t, float(coef))
            ref.near(w1[i].reshape(-1).numpy(), th, terms, f"step {t} tensor {i}", change)
            dm, dr = ref.dither(np.arange(o, o + n), t)
            ref.check_mx8(after[0][p], after[1][b], m, dm, what=f"step {t} tensor {i}")
            ref.check_mx8(after[2][p], after[3][b], np.sqrt(v), dr, root=True, what=f"step {t} tensor {i}")
        assert torch.equal(own, weights.bfloat16()) or all(
            torch.equal(a, b.bfloat16()) for a, b in zip(plan0.views(own, rank), plan0.views(weights, rank)))
    out = plan0.unpack(low)
    assert out[0].shape == (40, 24) and bool((out[0][20:] == plan0.views(weights, rank)[0].bfloat16()).all())
    # a checkpoint of one tensor's moments into two ranks' shards and back
    i = 0
    m32 = fp.mx8_dequantize(params.tensor_slice(mom[0], i), params.tensor_slice(mom[1], i))
    v32 = fp.mx8_dequantize(params.tensor_slice(mom[2], i), params.tensor_slice(mom[3], i), root=True)
    for x, root, codes, scales in ((m32, False, mom[0], mom[1]), (v32, True, mom[2], mom[3])):
        cut = fp.ReshardPlan(x.numel(), 1, 3).reshard([x])
        back = fp.ReshardPlan(x.numel(), 3, 1).reshard(list(cut.split(x.numel() // 3)))
        c, s = fp.mx8_quantize(back, root=root)
        assert torch.equal(fp.mx8_dequantize(c, s, root=root), x)


@pytest.mark.parametrize("bits", [32, 8])
def test_together_on_a_flat_shard(fp, bits):
    """The flat step with parameter groups and 8-bit moments: a rank's fragments
    of a FlatParameter, reduced, clipped, stepped as tensors, gathered."""
    say("flat shard", bits)
    shapes, world, rank = [(33, 5), (33,), (7, 70), (3,), (64, 9), (10,)], 4, 2
    plan = fp.Plan(shapes, world)
    S = plan.shard
    gen = torch.Generator().manual_seed(8)
    rows = (torch.randn(world, S, generator=gen) * 1e-3).bfloat16().to(dev())
    master = plan.pack([torch.randn(s, generator=gen).to(dev()) * 0.02 for s in shapes])[rank * S:(rank + 1) * S].clone()
    others = [None if q == rank else torch.randn(S, generator=gen).bfloat16().to(dev()) for q in range(world)]
    acc, full = torch.zeros(S, device=dev()), torch.zeros(world * S, dtype=torch.bfloat16, device=dev())
    own = full[rank * S:(rank + 1) * S]
    found = torch.zeros(1, dtype=torch.int32, device=dev())
    sq, coef = (torch.zeros(1, dtype=torch.float64, device=dev()) for _ in range(2))
    ws = fp.new_workspace(dev(), S)
    parts = [plan.views(b, rank) for b in (acc, master, own)]
    assert any(v.numel() == 0 for v in parts[0]) and sum(v.numel() for v in parts[0]) <= S
    params = fp.Params(*parts, groups=[int(len(s) < 2) for s in shapes])
    mom = params.new_moments(bits)
    step = params.stepper(mom, found_inf=found, grad_coef=coef, **columns(HPS))
    state = [(np.zeros(n), np.zeros(n)) for n in params.sizes]
    for t in (1, 2, 3):
        w0 = master.cpu().numpy()
        fp.reduce_shard(rows * t, acc, scale=1 / world, found_inf=found, sq_norm=sq, workspace=ws)
        fp.grad_coef(coef, sq_norm=sq, max_norm=0.01)
        step(t, **({"seed": t} if bits == 8 else {}))
        fp.unshard(others, full)
        torch.cuda.synchronize()
        for i, (d, n) in enumerate(zip(plan.view_descriptors(rank), params.sizes)):
            if n == 0:
                continue
            f, o = slice(d["buf_offset"], d["buf_offset"] + n), params.offsets[i]
            hp = HPS[params.groups[i]]
            th, m, v, terms, change = ref.adamw(acc[f].cpu().numpy(), w0[f], *state[i], hp, t, float(coef))
            ref.near(master[f].cpu().numpy(), th, terms, f"step {t} tensor {i}", change if bits == 8 else 0.0)
            raw = [x.view(torch.uint8).cpu().numpy() if bits == 8 else x.cpu().numpy() for x in mom]
            if bits == 8:
                b = slice(o // 32, o // 32 + -(-n // 32))
                dm, dr = ref.dither(np.arange(o, o + n), t)
                ref.check_mx8(raw[0][o:o + n], raw[1][b], m, dm, what=f"step {t} tensor {i}")
                ref.check_mx8(raw[2][o:o + n], raw[3][b], np.sqrt(v), dr, root=True, what=f"step {t} tensor {i}")
                state[i] = ref.decode(raw[0][o:o + n], raw[1][b]), ref.decode(raw[2][o:o + n], raw[3][b]) ** 2
            else:
                state[i] = raw[0][o:o + n], raw[1][o:o + n]
                ref.near(state[i][0], m, np.abs(m) + 1e-2, f"step {t} tensor {i}")
                ref.near(state[i][1], v, None, f"step {t} tensor {i}")
            assert torch.equal(own[f], master[f].bfloat16())
        assert all(torch.equal(full[q * S:(q + 1) * S], x) for q, x in enumerate(others) if x is not None)


def test_the_readmes_example(fp):
    """The README's loop over separate tensors runs and moves the weights."""
    say("README")
    text = open(os.path.join(ROOT, "README.md")).read()
    block = next(b for b in text.split("```python")[1:] if "fp.Params(" in b).split("```")[0]
    weights = [torch.nn.Parameter(torch.randn(s, device=dev()) * 0.02) for s in ((33, 20), (33,), (5, 7))]
    for p in weights:
        p.grad = torch.randn_like(p)
    before = [p.detach().clone() for p in weights]
    low = [torch.zeros_like(p, dtype=torch.bfloat16) for p in weights]
    ns = dict(torch=torch, fp=fp, dev=dev(), weights=weights, bf16_weights=low)
    exec(block, ns)
    torch.cuda.synchronize()
    assert int(ns["flag"]) == 0 and 0 < float(ns["coef"]) < 1
    for p, b, c in zip(weights, before, low):
        assert torch.isfinite(p).all() and not torch.equal(p.detach(), b)
        assert torch.equal(c, p.detach().bfloat16())
        # a constant gradient: the update is against its sign, lr a step once the moments have settled
        moved = (b - p.detach()) * p.grad.sign()
        assert (moved > 0).float().mean() > 0.99


def test_past_32_bit_offsets(fp):
    """A tensor of more than 2^32 elements and a small one behind it."""
    n = (1 << 32) + 5 * 1024 + 7
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB of free GPU memory")
    for bits in (8, 32):
        say("past 32 bits", bits)
        g = torch.zeros(n, dtype=torch.bfloat16, device=dev())
        w = torch.zeros(n, device=dev())
        tail_g, tail_w = torch.full((50,), 0.5, device=dev()).bfloat16(), torch.ones(50, device=dev())
        plan = fp.Params([g, tail_g], [w, tail_w])
        mom = plan.new_moments(bits)
        r = np.random.default_rng(0)
        spots = [slice(0, 64), slice((1 << 31) - 32, (1 << 31) + 32), slice((1 << 32) - 32, (1 << 32) + 32), slice(n - 39, n)]
        host = []
        for s in spots:
            x = torch.from_numpy(r.standard_normal(s.stop - s.start).astype(np.float32)).bfloat16()
            g[s] = x.to(dev())
            w[s] = x.float().to(dev())
            host.append(x.float().numpy())
        sq = torch.zeros(1, dtype=torch.float64, device=dev())
        plan.grad_norm(sq, plan.new_workspace())
        want = sum(float(np.square(x.astype(np.float64)).sum()) for x in host) + 50 * 0.25
        assert abs(float(sq) - want) <= 1e-12 * want
        plan.step(mom, step=1, seed=3 if bits == 8 else None, **HPS[0])
        torch.cuda.synchronize()
        for s, x in list(zip(spots, host)) + [(None, np.full(50, 0.5, np.float32))]:
            o = s.start if s else plan.offsets[1]
            k = x.size
            w0 = x if s else np.ones(50, np.float32)
            th, m, v, terms, change = ref.adamw(x, w0, np.zeros(k), np.zeros(k), HPS[0], 1)
            ref.near((w[s] if s else tail_w).cpu().numpy(), th, terms, f"weights at {o}", change if bits == 8 else 0.0)
            if bits == 32:
                ref.near(mom[0][o:o + k].cpu().numpy(), m, None, f"first moment at {o}")
                ref.near(mom[1][o:o + k].cpu().numpy(), v, None, f"second moment at {o}")
            elif o % 32 == 0:
                dm, dr = ref.dither(np.arange(o, o + k), 3)
                b = slice(o // 32, o // 32 + -(-k // 32))
                q = [t.view(torch.uint8) for t in mom]
                ref.check_mx8(q[0][o:o + k].cpu().numpy(), q[1][b].cpu().numpy(), m, dm, what=f"at {o}")
                ref.check_mx8(q[2][o:o + k].cpu().numpy(), q[3][b].cpu().numpy(), np.sqrt(v), dr, root=True, what=f"at {o}")
        del g, w, mom, plan
        torch.cuda.empty_cache()
