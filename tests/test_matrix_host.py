"""Argument checks of fp_muon_* and fp_mx4_* that need no GPU: every call here
is refused before anything is enqueued or allocated on a device, or has nothing
to do.  And the references against facts that are independent of them."""

import ctypes as C

import numpy as np
import pytest
import torch

import matrix_ref as ref
from sharded_flatparameter_pack_amd import _lib

F32, BF16, F16 = 0, 1, 2
A = 0x10000  # a made-up device address; no call here reads it
INVALID, RANGE, ALIGN, DEVICE = -1, -2, -3, -4


def ptrs(*p):
    return (C.c_void_p * len(p))(*p)


def create(lib, rows=(8, 10), cols=(4, 4), group=None, gd=BF16, grads=(A, A + 0x1000), master=(A + 0x2000, A + 0x3000),
           cd=BF16, copies=(A + 0x4000, A + 0x5000), ud=BF16, updates=None, n=None, out=True):
    h = C.c_void_p()
    n = len(rows) if n is None else n
    side = lambda x: (C.c_int64 * len(x))(*x) if x else None  # noqa: E731
    tab = lambda x: ptrs(*x) if x else None  # noqa: E731
    st = lib.fp_muon_create(n, side(rows), side(cols), (C.c_int32 * len(group))(*group) if group else None, gd, tab(grads),
                            tab(master), cd, tab(copies), ud, tab(updates), C.byref(h) if out else None)
    if st == 0:
        lib.fp_muon_destroy(h)
    return st


@pytest.mark.parametrize("want,kw", [
    (RANGE, dict(n=0)),
    (RANGE, dict(rows=(8, -1))),
    (RANGE, dict(cols=(4, (1 << 20) + 1))),
    (RANGE, dict(rows=(8, 1 << 20), cols=(4, 1 << 20), grads=(1 << 50, 1 << 51), master=None, copies=None,
                 updates=(1 << 52, 1 << 53))),                     # more tiles than one launch holds
    (RANGE, dict(group=(0, 16))),
    (RANGE, dict(group=(-1, 0))),
    (INVALID, dict(out=False)),
    (INVALID, dict(grads=None)),
    (INVALID, dict(rows=None, n=2)),
    (INVALID, dict(cols=None)),
    (INVALID, dict(grads=(A, None))),
    (INVALID, dict(master=(None, A))),
    (INVALID, dict(copies=(A + 0x4000, None))),
    (INVALID, dict(updates=(None, A + 0x6000))),
    (INVALID, dict(master=None)),                                  # copies of no weights
    (INVALID, dict(master=None, copies=None)),                     # nothing to write
    (INVALID, dict(gd=3)),
    (INVALID, dict(cd=F32)),
    (INVALID, dict(updates=(A + 0x6000, A + 0x7000), ud=3)),
    (ALIGN, dict(grads=(A + 1, A + 0x1000))),
    (ALIGN, dict(grads=(A + 2, A + 0x1000), gd=F32)),
    (ALIGN, dict(master=(A + 0x2002, A + 0x3000))),
    (ALIGN, dict(copies=(A + 0x4001, A + 0x5000))),
    (ALIGN, dict(updates=(A + 0x6002, A + 0x7000), ud=F32)),
    (INVALID, dict(master=(A + 0x2000, A + 0x207c))),              # weights overlap
    (INVALID, dict(copies=(A + 0x2010, A + 0x5000))),              # a copy in the weights
    (INVALID, dict(updates=(A + 0x403e, A + 0x7000))),             # an update in a copy
    (INVALID, dict(grads=(A, A + 0x3010))),                        # a gradient in the weights
])
def test_create_refuses(fp, want, kw):
    assert create(fp.lib(), **kw) == want
    assert fp.lib().fp_last_error()


def test_null_handles(fp):
    L = fp.lib()
    L.fp_muon_destroy(None)
    c = (C.c_double * 3)(*ref.COEFS)
    hp = _lib.fp_muon_hparams(1e-3, 0.9, 0.0, 1, 1)
    assert L.fp_muon_info(None, None, None) == INVALID
    assert L.fp_muon_offsets(None, None) == INVALID
    assert L.fp_muon_set_grads(None, None, None) == INVALID
    assert L.fp_muon_orthogonalize(None, 1, c, 1e-7, None, None) == INVALID
    assert L.fp_muon_step(None, 1, C.byref(hp), 1, c, 1e-7, None, None, None, None, None) == INVALID


def test_struct_layout(fp):
    assert C.sizeof(_lib.fp_muon_hparams) == 32
    assert _lib.fp_muon_hparams.nesterov.offset == 24


Q = dict(rows=40, cols=64, pitch=64, dtype=BF16, x=A, codes=A + 0x10000, scales=A + 0x20000, codes_t=None, scales_t=None)


@pytest.mark.parametrize("want,kw", [
    (0, dict(rows=0)),
    (0, dict(cols=0)),
    (0, dict(rows=0, x=None, codes=None, scales=None)),
    (RANGE, dict(rows=-1)),
    (RANGE, dict(cols=-1)),
    (RANGE, dict(rows=(1 << 31) + 1)),
    (RANGE, dict(pitch=63)),
    (RANGE, dict(rows=1 << 31, cols=1 << 20, pitch=1 << 20, codes=1 << 60, scales=1 << 61)),
    (INVALID, dict(dtype=3)),
    (INVALID, dict(x=None)),
    (INVALID, dict(codes=None, scales=None)),
    (INVALID, dict(scales=None)),
    (INVALID, dict(codes_t=A + 0x30000)),
    (ALIGN, dict(x=A + 1)),
    (ALIGN, dict(codes=A + 0x10008)),
    (ALIGN, dict(scales=A + 0x20004)),
    (ALIGN, dict(codes_t=A + 0x30008, scales_t=A + 0x40000)),
    (INVALID, dict(codes=A + 0x10)),                               # codes in x
    (INVALID, dict(scales=A + 0x10010)),                           # scales in the codes
    (INVALID, dict(codes_t=A + 0x10100, scales_t=A + 0x40000)),    # the two forms
])
def test_quantize_refuses(fp, want, kw):
    a = {**Q, **kw}
    assert fp.lib().fp_mx4_quantize(a["rows"], a["cols"], a["pitch"], a["dtype"], a["x"], a["codes"], a["scales"],
                                    a["codes_t"], a["scales_t"], 0, 0, None) == want


@pytest.mark.parametrize("want,kw", [
    (0, dict(rows=0)),
    (RANGE, dict(cols=-1)),
    (RANGE, dict(pitch=63)),
    (RANGE, dict(rows=1 << 31, cols=1 << 20, pitch=1 << 20, codes=1 << 60, scales=1 << 61)),
    (INVALID, dict(dtype=-1)),
    (INVALID, dict(x=None)),
    (INVALID, dict(codes=None)),
    (ALIGN, dict(x=A + 2, dtype=F32)),
    (ALIGN, dict(codes=A + 0x10004)),
    (INVALID, dict(x=A + 0x10010)),
])
def test_dequantize_refuses(fp, want, kw):
    a = {**Q, **kw}
    assert fp.lib().fp_mx4_dequantize(a["rows"], a["cols"], a["codes"], a["scales"], a["dtype"], a["x"], a["pitch"],
                                      None) == want


P = dict(m=8, n=16, k=300, a=A, asc=A + 0x10000, b=A + 0x20000, bsc=A + 0x30000, dtype=F32, out=A + 0x40000, pitch=16)


@pytest.mark.parametrize("want,kw", [
    (0, dict(m=0)),
    (0, dict(n=0, pitch=0)),
    (RANGE, dict(m=-1)),
    (RANGE, dict(k=0)),
    (RANGE, dict(k=(1 << 22) + 1)),
    (RANGE, dict(pitch=15)),
    (RANGE, dict(m=1 << 31, n=1 << 31, pitch=1 << 31, k=1, a=1 << 45, asc=1 << 46, b=1 << 47, bsc=1 << 48, out=1 << 55)),
    (INVALID, dict(dtype=7)),
    (INVALID, dict(a=None)),
    (INVALID, dict(bsc=None)),
    (INVALID, dict(out=None)),
    (ALIGN, dict(a=A + 8)),
    (ALIGN, dict(bsc=A + 0x30004)),
    (ALIGN, dict(out=A + 0x40002)),
    (INVALID, dict(out=A + 0x100)),
    (INVALID, dict(out=A + 0x30010)),
])
def test_matmul_refuses(fp, want, kw):
    a = {**P, **kw}
    assert fp.lib().fp_mx4_matmul(a["m"], a["n"], a["k"], a["a"], a["asc"], a["b"], a["bsc"], a["dtype"], a["out"], a["pitch"],
                                  0, None) == want


def test_padded(fp):
    assert [fp.mx4_padded(n) for n in (0, 1, 256, 257, 1 << 31)] == [0, 256, 256, 512, 1 << 31]
    for n in (-1, (1 << 31) + 1):
        with pytest.raises(ValueError):
            fp.mx4_padded(n)


def test_the_binding_refuses(fp):
    g = [torch.zeros(4, 4)]
    with pytest.raises(ValueError, match="device tensor"):
        fp.Muon(g, g)
    with pytest.raises(ValueError, match="at least one"):
        fp.Muon([])
    with pytest.raises(ValueError, match="dimensions"):
        fp.Muon([torch.zeros(8)], g)
    with pytest.raises(TypeError, match="is None"):
        fp.Muon([None], g)
    with pytest.raises(ValueError, match="device tensor"):
        fp.mx4_quantize(torch.zeros(4, 32))
    codes, scales = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        fp.mx4_dequantize(codes, scales, 32)
    with pytest.raises(ValueError, match="expected"):
        fp.mx4_dequantize(codes, scales, 300)
    with pytest.raises(ValueError, match="device tensor"):
        fp.mx4_matmul((codes, scales), (codes, scales))
    with pytest.raises(ValueError, match="padded"):
        fp.mx4_matmul((codes, scales), (codes[:, :64], scales))
    with pytest.raises(ValueError, match="sets of coefficients"):
        fp._muon_coefs(3, [ref.COEFS] * 2)
    with pytest.raises(ValueError, match=r"\(a, b, c\)"):
        fp._muon_coefs(1, (1.0, 2.0))


# ------------------------------------------------------------------ the references
def test_quantize_reference_is_the_nearest_value():
    """Every rounded value is a level of its block's scale with no nearer one, and the block's top is 4 or 6 (or was
    rounded there)."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((50, 96)) * np.exp(rng.standard_normal((50, 1)) * 4)).astype(np.float32)
    codes, scales = ref.quantize(x)
    got = ref.values(codes, scales, 96)
    s = np.repeat(np.exp2(scales[:, :3].astype(np.float64) - 127), 32, axis=1)
    grid = np.concatenate([ref.LEVELS, -ref.LEVELS])
    best = np.abs(x.astype(np.float64)[..., None] - grid * s[..., None]).min(-1)
    assert (np.abs(got - x) == best).all()
    top = np.abs(got / s).reshape(50, 3, 32).max(-1)
    assert set(top.ravel()) <= {4.0, 6.0}


def test_stochastic_reference_is_unbiased():
    x = np.full((1, 4096), 0.3, np.float32)
    x[0, ::32] = 6.0
    d = (np.arange(4096, dtype=np.uint64) * 40503 % 65536).reshape(1, -1)  # every sixteenth of the range alike
    got = ref.values(*ref.quantize(x, d), 4096)
    rest = np.delete(got, np.arange(0, 4096, 32))
    assert set(rest) == {0.0, 0.5} and abs(rest.mean() - 0.3) < 0.5 * 0.5 / 63 ** 0.5


def test_iteration_reference_by_singular_values():
    """On singular vectors the iteration is its polynomial."""
    gen = torch.Generator().manual_seed(3)
    u = torch.randn(20, 33, generator=gen, dtype=torch.float64)
    a, s, b = torch.linalg.svd(u, full_matrices=False)
    s = s / (s.norm() + 1e-7)
    for _ in range(5):
        s = ref.COEFS[0] * s + ref.COEFS[1] * s ** 3 + ref.COEFS[2] * s ** 5
    want = a @ torch.diag(s) @ b
    for x, y in ((ref.orthogonalize(u), want), (ref.orthogonalize(u.t()), want.t())):
        assert (x - y).norm() <= 1e-11 * y.norm()
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3
