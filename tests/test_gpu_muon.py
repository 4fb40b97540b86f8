"""The orthogonalisation and the step that takes it, on the GPU against 64 bits.

How far the iteration may be off, relative and in the 2-norm: its products see X, A and B off their diagonals in fp16.  A
rounding changes an element by 2^-12 of itself (root mean square), so that a step adds to X, in parts of |X|,
|R| 2^-12 <= 2.8 * 2^-12 from the rounded X (|R| <= b^2 / 4c, the largest |b t + c t^2|), about 1.2 |R| 2^-12 from the
rounded R, and about |b + 2c| 2^-12 of what A's rounding leaves in B, less than the others.  The roundings of a step are
independent, and the later steps neither add nor remove much of what the first ones left (p' is at most 3.4, where X is
still small and so is R): over the three last steps sqrt(3) * (2.8^2 + 3.4^2)^(1/2) * 2^-12 = 1.9e-3.  Twice that:
"""

import math
import os
import subprocess
import sys

import pytest
import torch

import matrix_ref as ref
from gpu_common import dev, say

pytestmark = pytest.mark.gpu

OFF = 4e-3
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HP = dict(lr=0.01, beta=0.9, weight_decay=0.1, nesterov=True)


def gradient(r, c, seed, kind="normal"):
    gen = torch.Generator().manual_seed(seed)
    g = torch.randn(r, c, generator=gen)
    if kind == "spiked":
        k = max(1, min(r, c) // 16)
        g = g + 4 * (torch.randn(r, k, generator=gen) @ torch.randn(k, c, generator=gen))
    if kind == "rows":  # rows that no token has reached
        g[torch.rand(r, generator=gen) < 0.3] = 0
    return g * 1e-3


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


SHAPES = [(1, 1), (1, 7), (5, 3), (64, 64), (65, 130), (200, 100), (33, 1000), (1000, 33), (300, 300), (128, 256), (0, 5), (17, 0)]


@pytest.mark.parametrize("gd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ud", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["normal", "spiked", "rows"])
def test_orthogonalize(fp, gd, ud, kind):
    grads = [gradient(r, c, 10 * i + 1, kind).to(DT[gd]) for i, (r, c) in enumerate(SHAPES)]
    out = [torch.full((r, c), 9.0, dtype=DT[ud], device=dev()) for r, c in SHAPES]
    plan = fp.Muon([g.to(dev()) for g in grads], updates=out)
    got = plan.orthogonalize(plan.new_workspace())
    torch.cuda.synchronize()
    for g, x, u in zip(grads, out, got):
        assert x is u
        if g.numel() == 0:
            continue
        say("orthogonalize", tuple(g.shape), gd, ud, kind)
        want = ref.orthogonalize(g)
        if float(want.norm()) == 0:
            assert bool((x == 0).all())
            continue
        assert rel(x.cpu(), want) <= OFF + torch.finfo(DT[ud]).eps / 2


@pytest.mark.parametrize("shape", [(512, 512), (700, 1900), (1900, 700), (2100, 2050), (128, 288), (288, 128), (130, 140), (64, 830)])
def test_orthogonalize_large(fp, shape):
    g = gradient(*shape, 4, "spiked")
    x = torch.empty(shape, device=dev())
    plan = fp.Muon([g.to(dev())], updates=[x])
    plan.orthogonalize(plan.new_workspace())
    assert rel(x.cpu(), ref.orthogonalize(g)) <= OFF


@pytest.mark.parametrize("shape", [(4090, 4001), (3800, 5000), (5000, 3800), (1, 300000), (300000, 3), (40, 70000),
                                   (70000, 90), (130, 9001), (9001, 130), (600, 9000), (9000, 700), (200, 2000)])
def test_orthogonalize_larger(fp, shape):
    g = gradient(*shape, 6, "spiked").to(dev())
    x = torch.empty(shape, device=dev())
    plan = fp.Muon([g], updates=[x])
    plan.orthogonalize(plan.new_workspace())
    assert rel(x, ref.orthogonalize(g)) <= OFF


def test_many_small_and_one_large(fp):
    """A batch of sizes that lie far apart shares its launches."""
    shapes = [(1400, 1300)] + [(16 + i % 40, 8 + i % 23) for i in range(300)]
    grads = [gradient(r, c, i) for i, (r, c) in enumerate(shapes)]
    out = [torch.empty(s, device=dev()) for s in shapes]
    plan = fp.Muon([g.to(dev()) for g in grads], updates=out)
    plan.orthogonalize(plan.new_workspace())
    for g, x in zip(grads, out):
        assert rel(x.cpu(), ref.orthogonalize(g)) <= OFF


@pytest.mark.parametrize("steps,coefs", [
    (1, ref.COEFS), (3, (1.5, -0.5, 0.0)), (10, (1.875, -1.25, 0.375)),
    (4, [ref.COEFS, ref.COEFS, (1.875, -1.25, 0.375), (1.875, -1.25, 0.375)]),
])
def test_other_coefficients(fp, steps, coefs):
    g = gradient(90, 140, 3)
    x = torch.empty(90, 140, device=dev())
    plan = fp.Muon([g.to(dev())], updates=[x])
    plan.orthogonalize(plan.new_workspace(), steps=steps, coefs=coefs)
    assert rel(x.cpu(), ref.orthogonalize(g, steps, coefs)) <= OFF


def test_scales_of_the_input(fp):
    """Norms from far below eps to the edge of fp32: eps counts, and squares neither vanish nor overflow."""
    base = gradient(40, 70, 8)
    for scale in (1e-30, 1e-9, 1e-4, 1e3, 1e30):
        g = base * scale
        x = torch.empty(40, 70, device=dev())
        plan = fp.Muon([g.to(dev())], updates=[x])
        plan.orthogonalize(plan.new_workspace())
        want = ref.orthogonalize(g)
        # below eps the iteration only scales its input: to fp16's precision of each element, or its smallest step
        assert float((x.cpu().double() - want).norm()) <= OFF * float(want.norm()) + 1e-30, scale


def test_zeros_and_not_finite(fp):
    g = [torch.zeros(30, 50), gradient(30, 50, 1), gradient(50, 30, 2), gradient(20, 20, 3)]
    g[1][3, 4] = float("inf")
    g[2][7, 0] = float("nan")
    out = [torch.empty(t.shape, device=dev()) for t in g]
    plan = fp.Muon([t.to(dev()) for t in g], updates=out)
    plan.orthogonalize(plan.new_workspace())
    assert bool((out[0] == 0).all())
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[2]).all())
    assert rel(out[3].cpu(), ref.orthogonalize(g[3])) <= OFF  # its neighbours are not touched


def state(shapes, gd, cd, odd=0):
    """A plan's tensors as views of one buffer each, from element `odd` on, with canaries between the matrices."""
    def views(dtype, make):
        sizes = [r * c for r, c in shapes]
        flat = torch.full((odd + sum(sizes) + 3 * len(sizes) + 3,), 7.0, dtype=dtype, device=dev())
        got, at = [], odd
        for i, (r, c) in enumerate(shapes):
            v = flat[at:at + r * c].view(r, c)
            v.copy_(make(i, r, c))
            got.append(v)
            at += r * c + 3
        return flat, got

    fg, grads = views(DT[gd], lambda i, r, c: gradient(r, c, i, "spiked"))
    fw, master = views(torch.float32, lambda i, r, c: gradient(r, c, 100 + i) * 20)
    fc, copies = views(DT[cd], lambda i, r, c: torch.zeros(r, c)) if cd else (None, None)
    return (fg, fw, fc), grads, master, copies


def gaps(flat, shapes, odd):
    """The buffer's elements outside the matrices."""
    keep = torch.ones(flat.numel(), dtype=torch.bool)
    at = odd
    for r, c in shapes:
        keep[at:at + r * c] = False
        at += r * c + 3
    return flat.cpu()[keep]


STEP_SHAPES = [(64, 64), (1, 9), (9, 1), (67, 130), (300, 100), (33, 500)]


@pytest.mark.parametrize("gd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cd", [None, "bf16", "f16"])
@pytest.mark.parametrize("nesterov,adjust,odd", [(True, "rms", 0), (False, "shape", 1), (True, None, 3)])
def test_step(fp, gd, cd, nesterov, adjust, odd):
    flats, grads, master, copies = state(STEP_SHAPES, gd, cd, odd)
    plan = fp.Muon(grads, master, copies)
    mom, ws = plan.new_momentum(), plan.new_workspace()
    mom.fill_(3.0)  # between the matrices it stays
    coef = torch.tensor([0.37], dtype=torch.float64, device=dev())
    ms = []
    for i, (r, c) in enumerate(STEP_SHAPES):
        m = gradient(r, c, 50 + i) * 0.3
        ms.append(m)
        plan.tensor_slice(mom, i).copy_(m.reshape(-1))
    before = [w.cpu().clone() for w in master]
    hp = {**HP, "nesterov": nesterov}
    plan.step(mom, ws, **hp, adjust=adjust, grad_coef=coef)
    torch.cuda.synchronize()
    for i, s in enumerate(STEP_SHAPES):
        say("step", s, gd, cd)
        m, w, x = ref.muon(grads[i].cpu(), ms[i], before[i], **hp, adjust=adjust, coef=0.37)
        got_m = plan.tensor_slice(mom, i).cpu().view(s)
        # one rounding of a sum that 64 bits hold to 2^-51
        assert bool(((got_m.double() - m.double()).abs() <= 2.0 ** -23 * m.double().abs() + 2.0 ** -149).all())
        got = master[i].cpu()
        rate = hp["lr"] * ref.adjust_of(s, adjust)
        assert float((got.double() - w).norm()) <= OFF * rate * float(x.norm()) + 2.0 ** -24 * float(w.norm())
        if copies:
            assert torch.equal(copies[i].cpu(), got.to(DT[cd]))
    for f in flats:
        assert f is None or bool((gaps(f, STEP_SHAPES, odd) == 7).all())
    used = torch.zeros(plan.partition, dtype=torch.bool)
    for o, n in zip(plan.offsets, plan.sizes):
        used[o:o + n] = True
    assert bool((mom.cpu()[~used] == 3).all())


# Matrices that one workgroup takes through everything, by what a wave of it holds; each list a plan of its own.
SMALL = [[(1, 1), (1, 7), (5, 3), (16, 16), (32, 48), (48, 32), (64, 32)], [(64, 64), (64, 60), (33, 127), (128, 64), (1, 256)],
         [(100, 90), (128, 128), (90, 130), (32, 500)], [(160, 160), (159, 131), (128, 256), (250, 100), (32, 1024), (1024, 1)]]


@pytest.mark.parametrize("shapes", SMALL)
@pytest.mark.parametrize("gd,cd,ud,odd", [("f32", None, "f32", 0), ("bf16", "bf16", "bf16", 1), ("f16", "f16", "f16", 3)])
def test_small(fp, shapes, gd, cd, ud, odd):
    flats, grads, master, copies = state(shapes, gd, cd, odd)
    fu = torch.full((odd + sum(r * c + 3 for r, c in shapes) + 3,), 7.0, dtype=DT[ud], device=dev())
    out, at = [], odd
    for r, c in shapes:
        out.append(fu[at:at + r * c].view(r, c))
        at += r * c + 3
    plan = fp.Muon(grads, master, copies, out)
    assert plan.workspace_bytes == 0
    ws, mom = plan.new_workspace(), plan.new_momentum()
    plan.orthogonalize(ws)
    for g, x, sh in zip(grads, out, shapes):
        say("orthogonalize", sh, gd, ud)
        assert rel(x.cpu(), ref.orthogonalize(g.cpu())) <= OFF + torch.finfo(DT[ud]).eps / 2
    for nesterov in (True, False):
        ms = [plan.tensor_slice(mom, i).cpu().view(sh) for i, sh in enumerate(shapes)]
        before = [w.cpu().clone() for w in master]
        plan.step(mom, ws, **{**HP, "nesterov": nesterov})
        for i, sh in enumerate(shapes):
            say("step", sh, gd, cd, nesterov)
            m, w, x = ref.muon(grads[i].cpu(), ms[i], before[i], **{**HP, "nesterov": nesterov})
            got_m = plan.tensor_slice(mom, i).cpu().view(sh).double()
            assert bool(((got_m - m.double()).abs() <= 2.0 ** -23 * m.double().abs() + 2.0 ** -149).all())
            rate = HP["lr"] * ref.adjust_of(sh, "rms")
            assert float((master[i].cpu().double() - w).norm()) <= OFF * rate * float(x.norm()) + 2.0 ** -24 * float(w.norm())
            if copies:
                assert torch.equal(copies[i].cpu(), master[i].cpu().to(DT[cd]))
    for f in (*flats, fu):
        assert f is None or bool((gaps(f, shapes, odd) == 7).all())


def test_many_small(fp):
    """More small matrices than one launch takes, of sizes far apart."""
    shapes = [(8 + i % 30, 8 + i % 23) for i in range(700)] + [(128, 100 + i) for i in range(20)]
    grads = [gradient(r, c, i) for i, (r, c) in enumerate(shapes)]
    out = [torch.empty(s, device=dev()) for s in shapes]
    plan = fp.Muon([g.to(dev()) for g in grads], updates=out)
    plan.orthogonalize(plan.new_workspace())
    for g, x in zip(grads, out):
        assert rel(x.cpu(), ref.orthogonalize(g)) <= OFF


BIG = [(1300, 2050), (2300, 700), (512, 1408), (31, 40)]


LONG = [(20, 5000), (5000, 30), (128, 4096), (64, 64), (300, 310), (7000, 65)]


@pytest.mark.parametrize("shapes", [BIG, LONG])
@pytest.mark.parametrize("gd,cd,odd", [("f32", "f16", 0), ("bf16", "bf16", 1), ("bf16", None, 0)])
def test_step_of_large_matrices(fp, shapes, gd, cd, odd):
    """Steps through the launches that a batch shares, one of them skipped; nothing is written outside the matrices, nor
    behind the workspace."""
    flats, grads, master, copies = state(shapes, gd, cd, odd)
    plan = fp.Muon(grads, master, copies)
    mom = plan.new_momentum()
    whole = torch.full((plan.workspace_bytes + 256,), 0xA5, dtype=torch.uint8, device=dev())
    step = plan.stepper(mom, whole[:plan.workspace_bytes], **HP, found_inf=(flag := torch.zeros(1, dtype=torch.int32, device=dev())))
    for t in range(2):
        ms = [plan.tensor_slice(mom, i).cpu().view(s) for i, s in enumerate(shapes)]
        before = [w.cpu().clone() for w in master]
        step()
        for i, s in enumerate(shapes):
            say("step", t, s, gd, cd)
            m, w, x = ref.muon(grads[i].cpu(), ms[i], before[i], **HP)
            got_m = plan.tensor_slice(mom, i).cpu().view(s).double()
            assert bool(((got_m - m.double()).abs() <= 2.0 ** -23 * m.double().abs() + 2.0 ** -149).all())
            rate = HP["lr"] * ref.adjust_of(s, "rms")
            assert float((master[i].cpu().double() - w).norm()) <= OFF * rate * float(x.norm()) + 2.0 ** -24 * float(w.norm())
            if copies:
                assert torch.equal(copies[i].cpu(), master[i].cpu().to(DT[cd]))
        if t == 0:
            flag.fill_(1)
            keep = [w.clone() for w in master], mom.clone()
            for c in copies or ():
                c.zero_()
            grads[0][5, 6] = float("nan")
            step()
            assert all(torch.equal(a, b) for a, b in zip(master, keep[0])) and torch.equal(mom, keep[1])
            assert all(torch.equal(c, w.to(c.dtype)) for c, w in zip(copies or (), master))
            grads[0][5, 6] = 0
            flag.zero_()
    for f in flats:
        assert f is None or bool((gaps(f, shapes, odd) == 7).all())
    assert bool((whole[plan.workspace_bytes:] == 0xA5).all())


def test_large_matrices_with_zeros_and_not_finite(fp):
    g = [torch.zeros(500, 600), gradient(700, 500, 1), gradient(500, 700, 2), gradient(400, 420, 3)]
    g[1][3, 4] = float("inf")
    g[2][7, 0] = float("nan")
    out = [torch.empty(t.shape, device=dev()) for t in g]
    plan = fp.Muon([t.to(dev()) for t in g], updates=out)
    plan.orthogonalize(plan.new_workspace())
    assert bool((out[0] == 0).all())
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[2]).all())
    assert rel(out[3].cpu(), ref.orthogonalize(g[3])) <= OFF


def test_more_than_one_batch(fp):
    """Matrices whose workspace passes what one batch holds: bit for bit what each gives in a plan of its own."""
    shapes = [(6000, 16000), (16000, 6000), (5990, 16001), (6000, 16000), (300, 500)]
    grads = [(torch.randn(s, generator=torch.Generator(device=dev()).manual_seed(i), device=dev()) * 1e-3).bfloat16()
             for i, s in enumerate(shapes)]
    out = [torch.zeros(s, dtype=torch.bfloat16, device=dev()) for s in shapes]
    plan = fp.Muon(grads, updates=out)
    plan.orthogonalize(plan.new_workspace())
    alone = 0
    for g, x in zip(grads, out):
        say("batch", tuple(g.shape))
        y = torch.empty_like(x)
        one = fp.Muon([g], updates=[y])
        one.orthogonalize(one.new_workspace())
        assert torch.equal(x, y)
        alone += one.workspace_bytes
    assert plan.workspace_bytes < alone
    assert rel(out[4].cpu(), ref.orthogonalize(grads[4].cpu())) <= OFF + 2.0 ** -8


@pytest.mark.parametrize("shape", [(2176, 1000001), (1000001, 2176)])
def test_more_than_31_bits_of_elements(fp, shape):
    """The iteration is a polynomial Q of A times X; Q comes from A in 64 bits, for parts of X far apart."""
    say("orthogonalize", shape)
    assert shape[0] * shape[1] > 1 << 31
    g = torch.randn(shape, generator=torch.Generator(device=dev()).manual_seed(3), dtype=torch.bfloat16, device=dev())
    x = torch.empty(shape, dtype=torch.float16, device=dev())
    plan = fp.Muon([g], updates=[x])
    plan.orthogonalize(plan.new_workspace())
    tall = shape[0] > shape[1]
    part = lambda t, lo, hi: (t[lo:hi].double().t() if tall else t[:, lo:hi].double())  # noqa: E731
    m, n = min(shape), max(shape)
    a = torch.zeros(m, m, dtype=torch.float64, device=dev())
    for lo in range(0, n, 1 << 17):
        p = part(g, lo, min(n, lo + (1 << 17))).contiguous()
        a += p @ p.t().contiguous()
    norm = float(a.diagonal().sum()) ** 0.5
    a /= norm * norm
    q = torch.eye(m, dtype=torch.float64, device=dev())
    for ca, cb, cc in [ref.COEFS] * 5:
        s = q @ a @ q.t().contiguous()
        q = (ca * torch.eye(m, dtype=torch.float64, device=dev()) + cb * s + cc * (s @ s)) @ q
    for lo in (0, 493447, 986895, n - 300):  # at 2^30 and 2^31 elements among them
        assert rel(part(x, lo, lo + 300), q @ (part(g, lo, lo + 300).contiguous() / norm)) <= OFF + 2.0 ** -11, lo


def test_steps_follow_the_formula(fp):
    """Several steps with changing gradients and rates, groups of their own hyperparameters."""
    shapes = [(40, 60), (60, 40), (30, 30)]
    _, grads, master, copies = state(shapes, "f32", "bf16")
    plan = fp.Muon(grads, master, copies, groups=[0, 1, 0])
    mom, ws = plan.new_momentum(), plan.new_workspace()
    step = plan.stepper(mom, ws, lr=[0.01, 0.003], beta=[0.9, 0.8], weight_decay=[0.1, 0.0])
    ms = [torch.zeros(s) for s in shapes]
    ws_ = [w.cpu().double() for w in master]
    off = [0.0] * 3
    for t in range(4):
        new = [gradient(*s, 200 + 10 * t + i) for i, s in enumerate(shapes)]
        if t == 2:
            plan.set_grads([g.to(dev()) for g in new])
        else:
            for a, b in zip(plan._keep[0], new):
                a.copy_(b)
        if t == 3:
            step(lr=[0.02, 0.001])
        else:
            step()
        rates = [0.02, 0.001] if t == 3 else [0.01, 0.003]
        for i, s in enumerate(shapes):
            k = [0, 1, 0][i]
            hp = dict(lr=rates[k], beta=[0.9, 0.8][k], weight_decay=[0.1, 0.0][k], nesterov=True)
            ms[i], ws_[i], x = ref.muon(new[i], ms[i], ws_[i], **hp)
            off[i] += OFF * hp["lr"] * ref.adjust_of(s, "rms") * float(x.norm()) + 2.0 ** -23 * float(ws_[i].norm())
    for i in range(3):
        assert float((master[i].cpu().double() - ws_[i]).norm()) <= off[i]
        assert torch.equal(copies[i].cpu(), master[i].cpu().bfloat16())


def test_skip(fp):
    """A set flag: weights and momentum bit for bit as they were, the copies the weights."""
    shapes = [(40, 60), (70, 33)]
    _, grads, master, copies = state(shapes, "bf16", "bf16")
    grads[0][3, 3] = float("inf")
    plan = fp.Muon(grads, master, copies)
    mom, ws = plan.new_momentum(), plan.new_workspace()
    mom.normal_()
    flag = torch.ones(1, dtype=torch.int32, device=dev())
    keep = [w.clone() for w in master], mom.clone()
    plan.step(mom, ws, **HP, found_inf=flag)
    assert all(torch.equal(a, b) for a, b in zip(master, keep[0])) and torch.equal(mom, keep[1])
    assert all(torch.equal(c, w.bfloat16()) for c, w in zip(copies, master))
    flag.zero_()
    grads[0][3, 3] = 0
    plan.step(mom, ws, **HP, found_inf=flag)
    assert not any(torch.equal(a, b) for a, b in zip(master, keep[0]))


def test_repeatable_and_in_any_workspace(fp):
    """Bitwise the same again, from a workspace full of NaN, and on another stream."""
    shapes = [(100, 260), (260, 100), (500, 500)]
    grads = [gradient(r, c, 5 + r).to(dev()) for r, c in shapes]
    out = [torch.empty(s, device=dev()) for s in shapes]
    plan = fp.Muon(grads, updates=out)
    ws = plan.new_workspace()
    plan.orthogonalize(ws)
    first = [x.clone() for x in out]
    ws.fill_(0xFF)
    plan.orthogonalize(ws)
    assert all(torch.equal(a, b) for a, b in zip(out, first))
    other = plan.new_workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        plan.orthogonalize(other)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_no_elements(fp):
    """A plan whose matrices are all empty: its calls do nothing."""
    shapes = [(0, 5), (3, 0)]
    _, grads, master, copies = state(shapes, "bf16", "bf16")
    plan = fp.Muon(grads, master, copies, [torch.empty(s, device=dev()) for s in shapes])
    assert plan.partition == 0 and plan.workspace_bytes == 0
    mom, ws = plan.new_momentum(), plan.new_workspace()
    plan.step(mom, ws, **HP)
    plan.orthogonalize(ws)
    plan.set_grads(grads)
    torch.cuda.synchronize()


def test_one_gradient_for_two_matrices(fp):
    """One gradient for two matrices: each as by itself."""
    g = gradient(70, 50, 3).to(dev())
    w = [gradient(70, 50, 10 + i).to(dev()) for i in range(2)]
    plan = fp.Muon([g, g], w)
    mom, ws = plan.new_momentum(), plan.new_workspace()
    want = [ref.muon(g.cpu(), torch.zeros(70, 50), x.cpu(), **HP) for x in w]
    plan.step(mom, ws, **HP)
    for i in range(2):
        m, x, o = want[i]
        assert float((w[i].cpu().double() - x).norm()) <= OFF * HP["lr"] * ref.adjust_of((70, 50), "rms") * float(o.norm()) + 2.0 ** -24 * float(x.norm())
    assert torch.equal(plan.tensor_slice(mom, 0), plan.tensor_slice(mom, 1))


def test_first_calls_in_a_capture(fp):
    """Calls that have not run before are captured as they are; replays against eager calls, with new gradients."""
    code = """
import sys, torch
sys.path[:0] = [%r, %r]
import sharded_flatparameter_pack_amd as fp
d = torch.device("cuda:0")
g = [torch.randn(s, device=d) for s in ((1500, 1300), (300, 4000), (90, 70), (4000, 3900))]
out = [torch.zeros_like(t) for t in g]
plan = fp.Muon(g, updates=out)
ws = plan.new_workspace()
x, w = torch.randn(700, 900, device=d), torch.randn(500, 900, device=d)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    plan.orthogonalize(ws)
    y = fp.mx4_matmul(fp.mx4_quantize(x), fp.mx4_quantize(w, seed=3))
for t in range(3):
    for k in (*g, x):
        k.normal_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in out], y.clone()
    plan.orthogonalize(ws)
    assert all(torch.equal(a, b) for a, b in zip(out, got[0]))
    assert torch.equal(fp.mx4_matmul(fp.mx4_quantize(x), fp.mx4_quantize(w, seed=3)), got[1])
    assert abs(float(out[0].norm()) / 1300 ** 0.5 - 1) < 0.3
print("captured")
"""
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code % (here, os.path.join(here, "tests"))], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_streams_at_once(fp):
    """Two plans with workspaces of their own on two streams beside each other."""
    shapes = [(600, 900), (900, 300), (40, 50)]
    grads = [[gradient(r, c, 5 + r + k).to(dev()) for r, c in shapes] for k in range(2)]
    out = [[torch.empty(s, device=dev()) for s in shapes] for _ in range(2)]
    plans = [fp.Muon(g, updates=o) for g, o in zip(grads, out)]
    ws = [p.new_workspace() for p in plans]
    want = []
    for p, w, o in zip(plans, ws, out):
        p.orthogonalize(w)
        want.append([t.clone() for t in o])
    streams = [torch.cuda.Stream() for _ in plans]
    torch.cuda.synchronize()
    for _ in range(5):
        for o in out:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for p, w, s in zip(plans, ws, streams):
            with torch.cuda.stream(s):
                p.orthogonalize(w)
                p.orthogonalize(w)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o, v in zip(out, want) for a, b in zip(o, v))


@pytest.mark.parametrize("shapes", [[(64, 96), (130, 50)], [(1200, 900), (300, 700), (20, 30)], [(100, 6000), (6000, 40)]])
def test_captured_step(fp, shapes):
    """A step captured into a graph: every replay against an eager step from the same state, with new gradients and with
    eager work between the replays."""
    _, grads, master, copies = state(shapes, "bf16", "bf16")
    plan = fp.Muon(grads, master, copies)
    mom, ws = plan.new_momentum(), plan.new_workspace()
    flag = torch.zeros(1, dtype=torch.int32, device=dev())
    step = plan.stepper(mom, ws, **HP, found_inf=flag)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(4):
        for i, g in enumerate(grads):
            g.copy_(gradient(*shapes[i], 70 + 5 * t + i))
        flag.fill_(int(t == 2))
        keep = [w.clone() for w in master], mom.clone()
        step()
        want = [w.clone() for w in master], mom.clone(), [c.clone() for c in copies]
        for w, k in zip(master, keep[0]):
            w.copy_(k)
        mom.copy_(keep[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(master, want[0]))
        assert torch.equal(mom, want[1])
        assert all(torch.equal(a, b) for a, b in zip(copies, want[2]))


def test_binding_refuses(fp):
    g = [gradient(200, 300, 1).to(dev())]
    w = [torch.zeros(200, 300, device=dev())]
    with pytest.raises(ValueError, match="neither"):
        fp.Muon(g)
    with pytest.raises(ValueError, match="shape"):
        fp.Muon(g, [torch.zeros(300, 200, device=dev())])
    with pytest.raises(ValueError, match="contiguous"):
        fp.Muon([g[0].t()], [torch.zeros(300, 200, device=dev())])
    with pytest.raises(TypeError):
        fp.Muon(g, [w[0].double()])
    with pytest.raises(fp._lib.FlatParamError, match="overlap"):
        fp.Muon(g, updates=g)
    plan = fp.Muon(g, w)
    mom, ws = plan.new_momentum(), plan.new_workspace()
    with pytest.raises(ValueError, match="no updates"):
        plan.orthogonalize(ws)
    with pytest.raises(ValueError, match="adjust"):
        plan.step(mom, ws, **HP, adjust="other")
    with pytest.raises(ValueError, match="workspace"):
        plan.step(mom, ws[:-1], **HP)
    with pytest.raises(fp._lib.FlatParamError, match="aligned"):
        plan.step(mom, torch.empty(ws.numel() + 16, dtype=torch.uint8, device=dev())[16:], **HP)
    with pytest.raises(fp._lib.FlatParamError, match="overlaps"):
        plan.step(ws[:4 * plan.partition].view(torch.float32), ws, **HP)
    for bad in (dict(beta=1.0), dict(lr=float("nan")), dict(steps=0), dict(steps=33), dict(eps=0.0),
                dict(coefs=(9.0, 0.0, 9.0)), dict(coefs=(float("inf"), 0.0, 0.0)),
                # a singular value of 0.54 goes to 1.35, 2.0, 8, 10^4 and on
                dict(steps=4, coefs=[(4.0, -6.0, 3.0), ref.COEFS, (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)])):
        with pytest.raises((fp._lib.FlatParamError, ValueError)):
            plan.step(mom, ws, **{**HP, **bad})
    step = plan.stepper(mom, ws, **HP)
    with pytest.raises(fp._lib.FlatParamError):
        step(lr=float("inf"))
    assert step._hp[0].lr == HP["lr"]
    with pytest.raises(ValueError, match="values for"):
        step(lr=[1.0, 2.0])
    no = fp.Muon(g, updates=[torch.empty(200, 300, device=dev())])
    with pytest.raises(ValueError, match="no master"):
        no.stepper(mom, ws, **HP)
    with pytest.raises(ValueError, match="shape"):
        plan.set_grads([g[0].t().contiguous()])
    assert bool((w[0] == 0).all())


def test_step_then_quantize_then_layer(fp):
    """As they are used together: the gradient of a layer run in MXFP4 goes into the step, whose weights give the next
    forms.  Each part against its reference on what the part before wrote."""
    t, n, k = 200, 96, 160
    w = (torch.randn(n, k, generator=torch.Generator().manual_seed(1)) * 0.05).to(dev())
    grad = torch.zeros(n, k, device=dev())
    copy = torch.zeros(n, k, dtype=torch.bfloat16, device=dev())
    plan = fp.Muon([grad], [w], [copy])
    mom, ws = plan.new_momentum(), plan.new_workspace()
    step = plan.stepper(mom, ws, **HP)
    m = torch.zeros(n, k)
    for i in range(3):
        x = gradient(t, k, 300 + i).mul(1e3).bfloat16().to(dev())
        dy = gradient(t, n, 400 + i).bfloat16().to(dev())
        qw = fp.mx4_quantize(w, transposed=True)
        qx, qd = fp.mx4_quantize(x, transposed=True), fp.mx4_quantize(dy, transposed=True, seed=i)
        y = fp.mx4_matmul(qx[:2], qw[:2])
        dx = fp.mx4_matmul(qd[:2], qw[2:])
        fp.mx4_matmul(qd[2:], qx[2:], grad)
        val = lambda q, j, c: torch.from_numpy(ref.values(q[j].cpu().numpy(), q[j + 1].view(torch.uint8).cpu().numpy(), c))  # noqa: E731
        wc, wt = w.cpu(), val(qw, 2, n)
        want = ref.quantize(wc.numpy())
        assert torch.equal(qw[0].cpu(), torch.from_numpy(want[0]))
        for got, p, q in ((y, val(qx, 0, k), val(qw, 0, k)), (dx, val(qd, 0, n), wt), (grad, val(qd, 2, t), val(qx, 2, t))):
            exact, size = p @ q.t(), p.abs() @ q.t().abs()
            slack = torch.finfo(got.dtype).eps / 2 * 1.01
            assert bool(((got.cpu().double() - exact).abs() <= (p.shape[1] + 1) * 2.0 ** -24 * size + slack * exact.abs()).all())
        g = grad.cpu().clone()
        step()
        m, want_w, o = ref.muon(g, m, wc, **HP)
        assert float((w.cpu().double() - want_w).norm()) <= OFF * HP["lr"] * ref.adjust_of((n, k), "rms") * float(o.norm()) + 2.0 ** -24 * float(want_w.norm())
        assert torch.equal(copy, w.bfloat16())
        m = plan.tensor_slice(mom, 0).cpu().view(n, k).clone()
    assert math.isfinite(float(w.sum()))
