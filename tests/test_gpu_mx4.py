"""MXFP4 on the GPU against the 64-bit reference: codes and scales bit for bit, values exactly, products within what
fp32 sums and one rounding of the output allow."""

import numpy as np
import pytest
import torch

import matrix_ref as ref
from gpu_common import dev, say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def matrix(rows, cols, dtype, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)) * spread)
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


def canaries(*shape):
    """A byte buffer with 64 bytes of 0xA5 on both sides, and the view between them."""
    n = int(np.prod(shape))
    whole = torch.full((n + 128,), 0xA5, dtype=torch.uint8, device=dev())
    return whole, whole[64:64 + n].view(shape)


def intact(whole):
    return bool((whole[:64] == 0xA5).all()) and bool((whole[-64:] == 0xA5).all())


def quantized(fp, x, **kw):
    """mx4_quantize into guarded buffers, as numpy: (codes, scales, codes_t, scales_t)."""
    r, c = x.shape
    held = [canaries(r, ref.padded(c) // 2), canaries(r, ref.padded(c) // 32),
            canaries(c, ref.padded(r) // 2), canaries(c, ref.padded(r) // 32)]
    fp.mx4_quantize(x, *[v for _, v in held], transposed=True, **kw)
    torch.cuda.synchronize()
    assert all(intact(w) for w, _ in held)
    return [v.cpu().numpy() for _, v in held]


SHAPES = [(1, 1), (1, 33), (33, 1), (2, 256), (31, 257), (64, 64), (128, 128), (129, 300), (257, 40), (5, 2000), (700, 9)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", [None, 12345])
def test_quantize(fp, shape, dtype, seed):
    say("quantize", shape, dtype, seed)
    x = matrix(*shape, dtype, 7 + shape[0], 1.0)
    v = x.float().numpy()
    h = None if seed is None else ref.dither(*shape, seed)
    want = (*ref.quantize(v, None if h is None else h >> np.uint64(16)),
            *ref.quantize(np.ascontiguousarray(v.T), None if h is None else np.ascontiguousarray((h & np.uint64(0xFFFF)).T)))
    got = quantized(fp, x.to(dev()), seed=seed)
    for g, w, name in zip(got, want, ("codes", "scales", "codes_t", "scales_t")):
        assert np.array_equal(g, w), (name, np.argwhere(g != w)[:5])
    # either form alone is the same
    alone = fp.mx4_quantize(x.to(dev()), seed=seed)
    other = fp.mx4_quantize(x.to(dev()), rows=False, transposed=True, seed=seed)
    for t, w in zip((*alone, *other), want):
        assert np.array_equal(t.view(torch.uint8).cpu().numpy(), w)


@pytest.mark.parametrize("seed", [None, 99])
def test_quantize_every_rounding(fp, seed):
    """Every value of 16 mantissa bits around every border, at the ends of fp32's range, zeros and their signs."""
    m = np.arange(1 << 16, dtype=np.uint32)
    rows = []
    for e in (0, 1, 2, 3, 100, 127, 200, 252, 253, 254):
        top = np.uint32((min(e + 2, 254) << 23) | 0x400000)  # holds the block's scale in place
        v = ((np.uint32(e) << 23) | (m << 7)).astype(np.uint32)
        v[::2] |= 0x80000000
        v = v.reshape(-1, 31)[:, :31] if len(v) % 31 == 0 else np.resize(v, (2115, 31))
        rows.append(np.concatenate([np.full((len(v), 1), top, np.uint32), v], 1))
    bits = np.concatenate(rows)
    bits[0, 5], bits[1, 7] = 0, 0x80000000
    x = np.ascontiguousarray(bits).view(np.float32)
    h = None if seed is None else ref.dither(*x.shape, seed)
    want = ref.quantize(x, None if h is None else h >> np.uint64(16))
    got = fp.mx4_quantize(torch.from_numpy(x).to(dev()), seed=seed)
    assert np.array_equal(got[1].view(torch.uint8).cpu().numpy(), want[1])
    g = got[0].cpu().numpy()
    assert np.array_equal(g, want[0]), np.argwhere(g != want[0])[:5]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("what", [float("inf"), -float("inf"), float("nan")])
def test_not_finite_blocks_are_nan(fp, dtype, what):
    x = matrix(70, 100, dtype, 3, 0.5)
    x[3, 40] = what
    x[69, 99] = what
    got = quantized(fp, x.to(dev()))
    v = x.float().numpy()
    with np.errstate(invalid="ignore"):
        want = (*ref.quantize(v), *ref.quantize(np.ascontiguousarray(v.T)))
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    back = fp.mx4_dequantize(*[torch.from_numpy(a).to(dev()) for a in got[:2]], 100, dtype=torch.float32).cpu().numpy()
    nan = np.zeros((70, 100), bool)
    nan[3, 32:64] = nan[69, 96:] = True
    assert np.array_equal(np.isnan(back), nan)


def test_largest_and_smallest(fp):
    x = torch.zeros(5, 64)
    x[0, 0] = 1.75 * 2.0 ** 127          # the scale would pass fp32's range: NaN
    x[1, 0] = float(np.nextafter(np.float32(1.75 * 2.0 ** 127), np.float32(0)))
    x[2, 0] = 2.0 ** -149
    x[3] = -0.0
    x[4, :32] = torch.tensor([2.0 ** -126 * k / 8 for k in range(32)])
    got = quantized(fp, x.to(dev()))
    want = ref.quantize(x.numpy())
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert got[1][0, 0] == 255 and got[1][1, 0] == 252 and (got[0][3, :32] == 0x88).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_strided_source(fp, dtype):
    """Rows apart, from an odd element on; the values beside them take no part."""
    whole = torch.full((50, 301), float("nan")).to(DT[dtype])
    x = matrix(50, 131, dtype, 11)
    whole[:, 7:138] = x
    got = fp.mx4_quantize(whole.to(dev())[:, 7:138], transposed=True, seed=5)
    want = fp.mx4_quantize(x.to(dev()), transposed=True, seed=5)
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (31, 257), (130, 1000)])
def test_dequantize(fp, shape, dtype):
    say("dequantize", shape, dtype)
    x = matrix(*shape, "f32", 5, 1.0)
    codes, scales = ref.quantize(x.numpy())
    want = torch.from_numpy(ref.values(codes, scales, shape[1])).to(DT[dtype])
    c, s = torch.from_numpy(codes).to(dev()), torch.from_numpy(scales).to(dev())
    got = fp.mx4_dequantize(c, s, shape[1], dtype=DT[dtype])
    assert torch.equal(got.cpu(), want)
    # into rows that lie apart: what is between them stays
    whole = torch.full((shape[0], shape[1] + 5), 77.0, dtype=DT[dtype], device=dev())
    fp.mx4_dequantize(c, s, shape[1], whole[:, 3:3 + shape[1]])
    assert torch.equal(whole[:, 3:3 + shape[1]].cpu(), want)
    assert bool((whole[:, :3] == 77).all()) and bool((whole[:, 3 + shape[1]:] == 77).all())


def test_dequantize_every_code_under_every_scale(fp):
    codes = np.tile(np.arange(256, dtype=np.uint8), 2)[None].repeat(2, 0).reshape(2, 512)[:, :256].reshape(4, 128)
    c = np.empty((256, 128), np.uint8)
    s = np.empty((256, 8), np.uint8)
    for b in range(256):
        c[b] = codes[b % 4]
        s[b] = b
    with np.errstate(invalid="ignore"):
        want = ref.values(c, s, 256).astype(np.float32)
    got = fp.mx4_dequantize(torch.from_numpy(c).to(dev()), torch.from_numpy(s).to(dev()), 256, dtype=torch.float32).cpu().numpy()
    assert np.array_equal(got[:255], want[:255])
    assert np.isnan(got[255]).all()


def product(a, b):
    return torch.from_numpy(a) @ torch.from_numpy(b).t()


def check_product(fp, m, n, k, dtype, accumulate, seed, pitch=None):
    """|got - want| <= (terms of the sum) 2^-24 sum |a b| + half a step of the output."""
    say("product", m, n, k, dtype, accumulate)
    a, b = matrix(m, k, "f32", seed, 1.0), matrix(n, k, "f32", seed + 1, 1.0)
    qa, qb = ref.quantize(a.numpy()), ref.quantize(b.numpy())
    va, vb = ref.values(*qa, k), ref.values(*qb, k)
    want, size = product(va, vb), product(np.abs(va), np.abs(vb))
    da = [torch.from_numpy(t).to(dev()) for t in qa]
    db = [torch.from_numpy(t).to(dev()) for t in qb]
    whole = torch.full((m, n + 9), 5.0, dtype=DT[dtype], device=dev())
    out = whole[:, 4:4 + n]
    if accumulate:
        old = matrix(m, n, dtype, seed + 2, 0.5)
        out.copy_(old.to(dev()))
        want, size = want + old.double(), size + old.double().abs()
    fp.mx4_matmul(da, db, out, accumulate=accumulate)
    got = out.cpu().double()
    bound = (k + 1) * 2.0 ** -24 * size + torch.finfo(DT[dtype]).eps / 2 * want.abs() * 1.01
    if dtype == "f16":
        bound += 2.0 ** -25
    assert bool((want.abs() < 60000).all()) or dtype != "f16"
    bad = (got - want).abs() > bound
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())
    assert bool((whole[:, :4] == 5).all()) and bool((whole[:, 4 + n:] == 5).all())


PRODUCTS = [(1, 1, 1), (1, 17, 31), (2, 16, 256), (3, 500, 700), (16, 16, 512), (15, 130, 2000), (17, 64, 64), (33, 77, 300),
            (64, 1000, 1024), (65, 130, 300), (100, 63, 5000), (257, 300, 513)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(fp, m, n, k, dtype):
    check_product(fp, m, n, k, dtype, False, m + n + k)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(1, 100, 600), (40, 41, 42), (200, 311, 1000)])
def test_product_accumulates(fp, m, n, k, dtype):
    check_product(fp, m, n, k, dtype, True, 5)


@pytest.mark.parametrize("m,n,k", [(1500, 1700, 300), (3900, 4200, 520)])
def test_product_of_many_tiles(fp, m, n, k):
    check_product(fp, m, n, k, "f32", False, 9)


def test_product_scales_of_every_block(fp):
    """Each block of each row under a scale of its own: a scale taken for another block or row would show."""
    m, n, k = 48, 80, 2048
    rng = np.random.default_rng(2)
    a = (rng.standard_normal((m, k // 32, 32)) * np.exp2(rng.integers(-9, 10, (m, k // 32, 1)))).reshape(m, k)
    b = (rng.standard_normal((n, k // 32, 32)) * np.exp2(rng.integers(-9, 10, (n, k // 32, 1)))).reshape(n, k)
    qa, qb = ref.quantize(a.astype(np.float32)), ref.quantize(b.astype(np.float32))
    va, vb = ref.values(*qa, k), ref.values(*qb, k)
    got = fp.mx4_matmul([torch.from_numpy(t).to(dev()) for t in qa], [torch.from_numpy(t).to(dev()) for t in qb],
                        dtype=torch.float32).cpu().double()
    assert bool(((got - product(va, vb)).abs() <= k * 2.0 ** -24 * product(np.abs(va), np.abs(vb))).all())


def test_product_with_nan_blocks(fp):
    """A NaN block makes its row's (or column's) outputs NaN and no others."""
    a, b = matrix(40, 100, "f32", 1), matrix(50, 100, "f32", 2)
    a[7, 33], b[11, 99] = float("inf"), float("nan")
    y = fp.mx4_matmul(fp.mx4_quantize(a.to(dev())), fp.mx4_quantize(b.to(dev())), dtype=torch.float32).cpu()
    nan = torch.zeros(40, 50, dtype=torch.bool)
    nan[7], nan[:, 11] = True, True
    assert torch.equal(torch.isnan(y), nan)


@pytest.mark.parametrize("t,n,k", [(1, 40, 70), (37, 300, 130), (260, 64, 257)])
def test_layer_forward_and_backward(fp, t, n, k):
    """y = x w^T and its gradients through both forms of each operand, against the formulas and against differences."""
    x, w, dy = (matrix(*s, "f32", 20 + i, 0.3) for i, s in enumerate(((t, k), (n, k), (t, n))))
    qx, qw, qd = (fp.mx4_quantize(v.to(dev()), transposed=True, seed=s) for v, s in ((x, None), (w, None), (dy, 3)))
    y = fp.mx4_matmul(qx[:2], qw[:2], dtype=torch.float32).cpu().double()
    dx = fp.mx4_matmul(qd[:2], qw[2:], dtype=torch.float32).cpu().double()
    dw = fp.mx4_matmul(qd[2:], qx[2:], dtype=torch.float32).cpu().double()

    def val(q, cols, i=0):
        return torch.from_numpy(ref.values(q[i].cpu().numpy(), q[i + 1].view(torch.uint8).cpu().numpy(), cols))

    xr, wr, dr = val(qx, k), val(qw, k), val(qd, n)
    xc, wc, dc = val(qx, t, 2).t(), val(qw, n, 2).t(), val(qd, t, 2).t()
    for got, p, q in ((y, xr, wr.t()), (dx, dr, wc), (dw, dc.t(), xc)):
        assert bool(((got - p @ q).abs() <= (p.shape[1] + 1) * 2.0 ** -24 * (p.abs() @ q.abs())).all())
    # the loss sum(dy y) is linear in x and in w: a difference along any direction is the gradient times it.  What
    # is left is the quantisation's: each operand's elements are off by half a step at most (the stochastic one's by a
    # step), which is a quarter (a half) of the value or of a twelfth (a sixth) of the block's largest.
    for g, base, other, towards in ((dx, x, w, torch.ones_like(x)), (dw, w, x, torch.ones_like(w))):
        dyd, o, d = dy.double(), other.double(), towards.double()
        exact = float((dyd * (d @ o.t() if base is x else o @ d.t())).sum())
        got = float((g * d).sum())
        dev_o = (o.abs() / 4 + o.abs().max() / 12)
        dev_d = (dyd.abs() / 2 + dyd.abs().max() / 6)
        spread = ((dyd.abs() + dev_d).t() if base is w else (dyd.abs() + dev_d)) @ (o.abs() + dev_o)
        plain = (dyd.abs().t() if base is w else dyd.abs()) @ o.abs()
        assert abs(got - exact) <= float((spread - plain).sum())


def test_other_stream_and_graph(fp):
    """Quantise and multiply on another stream, captured and replayed with new inputs between the replays."""
    x, w = matrix(70, 300, "bf16", 1).to(dev()), matrix(90, 300, "f32", 2).to(dev())
    qw = fp.mx4_quantize(w)
    held, out = fp.mx4_empty(70, 300, dev()), torch.zeros(70, 90, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fp.mx4_quantize(x, *held)
        fp.mx4_matmul(held, qw, out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp.mx4_quantize(x, *held)
        fp.mx4_matmul(held, qw, out, accumulate=True)
    for i in range(4):
        x.copy_(matrix(70, 300, "bf16", 10 + i))
        before = out.clone()
        want = fp.mx4_matmul(fp.mx4_quantize(x), qw, before.clone(), accumulate=True)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("seed", [None, 7])
def test_given_buffers_of_one_form(fp, seed):
    """Either form alone into the caller's buffers, which count as changed in place."""
    x = matrix(50, 300, "bf16", 3).to(dev())
    want = fp.mx4_quantize(x, transposed=True, seed=seed)
    rows, cols = fp.mx4_empty(50, 300, dev()), fp.mx4_empty(300, 50, dev())
    before = [t._version for t in (*rows, *cols)]
    assert fp.mx4_quantize(x, *rows, seed=seed) == rows
    assert fp.mx4_quantize(x, None, None, *cols, rows=False, transposed=True, seed=seed) == cols
    for got, w in zip((*rows, *cols), want):
        assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))
    assert all(t._version > v for t, v in zip((*rows, *cols), before))
    out = torch.zeros(50, 50, device=dev())
    v = out._version
    fp.mx4_matmul(rows, rows, out)
    assert out._version > v
    # one form given, the other allocated
    both = fp.mx4_quantize(x, None, None, *cols, transposed=True, seed=seed)
    for got, w in zip(both, want):
        assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("m,n,k", [(16, 300, 5000), (17, 300, 300), (32, 90, 4000), (33, 90, 700), (64, 20, 3000), (65, 20, 3000),
                                   (5, 4099, 256), (2000, 7, 500), (16, 8192, 300), (16, 8193, 300), (32, 4096, 40), (20, 5000, 40),
                                   (3, 40000, 256), (100, 40000, 40)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_product_of_few_rows(fp, m, n, k, dtype):
    check_product(fp, m, n, k, dtype, True, 31)


def test_one_operand_for_both_sides(fp):
    q = fp.mx4_quantize(matrix(300, 400, "f32", 3).to(dev()))
    y = fp.mx4_matmul(q, q, dtype=torch.float32)
    assert torch.equal(y, y.t())


def test_two_streams_at_once(fp):
    """Calls on two streams beside each other: bit for bit what they give one after the other."""
    x = [matrix(700, 900, "bf16", 40 + i).to(dev()) for i in range(2)]
    want = [fp.mx4_matmul(fp.mx4_quantize(t), fp.mx4_quantize(t, seed=5)) for t in x]
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fp.mx4_matmul(fp.mx4_quantize(x[i]), fp.mx4_quantize(x[i], seed=5)))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


def test_more_than_32_bits_of_elements(fp):
    """Both forms, their values and a product whose output has over 2^32 elements: their last rows and columns."""
    r, c, seed = 66001, 65120, 77
    assert r * c > 1 << 32
    say("quantize", r, c)
    x = torch.zeros(r, c, dtype=torch.bfloat16, device=dev())
    tail_r, tail_c = matrix(3, c, "bf16", 1, 1.0), matrix(r, 2, "bf16", 2, 1.0)
    x[-3:] = tail_r.to(dev())
    x[:, -2:] = tail_c.to(dev())
    tail_r[:, -2:] = tail_c[-3:]
    for s in (None, seed):
        codes, scales, codes_t, scales_t = fp.mx4_quantize(x, transposed=True, seed=s)
        at_r = np.arange(r - 3, r, dtype=np.uint64)[:, None] * np.uint64(c) + np.arange(c, dtype=np.uint64)
        at_c = np.arange(r, dtype=np.uint64) * np.uint64(c) + np.arange(c - 2, c, dtype=np.uint64)[:, None]
        at_r, at_c = at_r & np.uint64(ref.M32), at_c & np.uint64(ref.M32)
        want = ref.quantize(tail_r.float().numpy(), None if s is None else ref.hashes(at_r, s) >> np.uint64(16))
        want_t = ref.quantize(np.ascontiguousarray(tail_c.float().numpy().T),
                              None if s is None else ref.hashes(at_c, s) & np.uint64(0xFFFF))
        assert np.array_equal(codes[-3:].cpu().numpy(), want[0])
        assert np.array_equal(scales[-3:].view(torch.uint8).cpu().numpy(), want[1])
        assert np.array_equal(codes_t[-2:].cpu().numpy(), want_t[0])
        assert np.array_equal(scales_t[-2:].view(torch.uint8).cpu().numpy(), want_t[1])
    del codes_t, scales_t
    say("dequantize", r, c)
    fp.mx4_dequantize(codes, scales, c, x)
    assert np.array_equal(x[-3:].float().cpu().numpy(), ref.values(*want, c).astype(np.float32))
    del codes, scales
    say("product", r, c)
    k = 40
    a, b = matrix(r, k, "f32", 3, 0.5), matrix(c, k, "f32", 4, 0.5)
    qa, qb = fp.mx4_quantize(a.to(dev())), fp.mx4_quantize(b.to(dev()))
    x.fill_(5)
    fp.mx4_matmul(qa, qb, x)
    va, vb = (torch.from_numpy(ref.values(*ref.quantize(t.numpy()), k)) for t in (a, b))
    for rows in (slice(0, 3), slice(r - 300, r)):
        y = va[rows] @ vb.t()
        bound = (k + 1) * 2.0 ** -24 * (va[rows].abs() @ vb.t().abs()) + 2.0 ** -8 * y.abs() * 1.01
        assert bool(((x[rows].cpu().double() - y).abs() <= bound).all())


def test_binding_refuses(fp):
    x = torch.zeros(8, 64, device=dev())
    with pytest.raises(ValueError, match="contiguous"):
        fp.mx4_quantize(x.t())
    with pytest.raises(TypeError):
        fp.mx4_quantize(x.double())
    with pytest.raises(ValueError, match="dimensions"):
        fp.mx4_quantize(x[0])
    with pytest.raises(ValueError, match="neither"):
        fp.mx4_quantize(x, rows=False)
    with pytest.raises(ValueError, match="not wanted"):
        fp.mx4_quantize(x, codes_t=torch.zeros(64, 128, dtype=torch.uint8, device=dev()))
    with pytest.raises(ValueError, match="go together"):
        fp.mx4_quantize(x, codes=torch.zeros(8, 128, dtype=torch.uint8, device=dev()))
    q = fp.mx4_quantize(x)
    with pytest.raises(ValueError, match="expected"):
        fp.mx4_dequantize(*q, 257)
    with pytest.raises(ValueError, match="shape"):
        fp.mx4_dequantize(*q, 64, torch.zeros(8, 63, device=dev()))
    with pytest.raises(ValueError, match="shape"):
        fp.mx4_matmul(q, q, torch.zeros(8, 7, device=dev()))
    with pytest.raises(ValueError, match="needs out"):
        fp.mx4_matmul(q, q, accumulate=True)
    with pytest.raises(TypeError):
        fp.mx4_matmul(q, q, dtype=torch.float64)
    with pytest.raises(ValueError, match="device"):
        fp.mx4_matmul(q, tuple(t.cpu() for t in q))
    assert fp.mx4_quantize(torch.zeros(0, 5, device=dev()))[0].shape == (0, 128)
    assert fp.mx4_matmul(q, fp.mx4_quantize(torch.zeros(0, 64, device=dev()))).shape == (8, 0)
