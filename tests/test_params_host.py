"""Argument checks of fp_params_* and fp_mx8_* that need no GPU: every call
here is refused before anything is enqueued or allocated on a device."""

import ctypes as C

import pytest
import torch

from sharded_flatparameter_pack_amd import _lib

F32, BF16, F16 = 0, 1, 2
A = 0x10000  # a made-up device address; no call here reads it


def ptrs(*p):
    return (C.c_void_p * len(p))(*p)


def create(lib, numel=(8, 40), group=None, gd=BF16, grads=(A, A + 0x1000), master=(A + 0x2000, A + 0x3000), cd=BF16,
           copies=(A + 0x4000, A + 0x5000), n=None, out=True):
    h = C.c_void_p()
    n = len(numel) if n is None else n
    st = lib.fp_params_create(n, (C.c_int64 * len(numel))(*numel) if numel is not None else None,
                              (C.c_int32 * len(group))(*group) if group else None, gd,
                              ptrs(*grads) if grads else None, ptrs(*master) if master else None, cd,
                              ptrs(*copies) if copies else None, C.byref(h) if out else None)
    if st == 0:
        lib.fp_params_destroy(h)
    return st


INVALID, RANGE, ALIGN, DEVICE = -1, -2, -3, -4


@pytest.mark.parametrize("want,kw", [
    (RANGE, dict(n=0)),
    (RANGE, dict(n=-3)),
    (RANGE, dict(numel=(8, -1))),
    (RANGE, dict(numel=(8, (1 << 40) + 1))),
    (RANGE, dict(numel=(8, 1 << 40), copies=None, master=None)),   # more tiles than one launch holds
    (RANGE, dict(group=(0, 16))),
    (RANGE, dict(group=(-1, 0))),
    (INVALID, dict(out=False)),
    (INVALID, dict(grads=None)),
    (INVALID, dict(grads=(A, None))),
    (INVALID, dict(master=(None, A))),
    (INVALID, dict(copies=(A + 0x4000, None))),
    (INVALID, dict(master=None)),                                  # copies of no weights
    (INVALID, dict(gd=3)),
    (INVALID, dict(gd=-1)),
    (INVALID, dict(cd=F32)),
    (ALIGN, dict(grads=(A + 1, A + 0x1000))),
    (ALIGN, dict(grads=(A + 2, A + 0x1000), gd=F32)),
    (ALIGN, dict(master=(A + 0x2002, A + 0x3000))),
    (ALIGN, dict(copies=(A + 0x4001, A + 0x5000))),
    (INVALID, dict(master=(A + 0x2000, A + 0x201c))),              # weights overlap
    (INVALID, dict(master=(A + 0x2000, A + 0x2000))),              # the same tensor twice
    (INVALID, dict(copies=(A + 0x2010, A + 0x5000))),              # a copy in the weights
    (INVALID, dict(grads=(A, A + 0x3010))),                        # a gradient in the weights
    (INVALID, dict(grads=(A + 0x4fb0, A), numel=(64, 40), copies=(A + 0x4000, A + 0x5000))),
])
def test_create_refuses(fp, want, kw):
    assert create(fp.lib(), **kw) == want
    assert fp.lib().fp_last_error()


def test_null_handles_and_buffers(fp):
    L = fp.lib()
    L.fp_params_destroy(None)
    assert L.fp_params_info(None, None, None) == INVALID
    assert L.fp_params_offsets(None, None) == INVALID
    assert L.fp_params_set_grads(None, None, None) == INVALID
    assert L.fp_params_grad_norm(None, None, None, None, None) == INVALID
    hp = _lib.fp_adamw_hparams(1e-3, 0.9, 0.999, 1e-8, 0.0, 1)
    assert L.fp_params_adamw(None, 1, C.byref(hp), None, None, None, None, None) == INVALID
    assert L.fp_params_adamw8(None, 1, C.byref(hp), None, None, None, None, 0, None, None, None) == INVALID


@pytest.mark.parametrize("want,n,x,codes,scales", [
    (0, 0, None, None, None),
    (RANGE, -1, A, A, A),
    (RANGE, 1 << 40, A, A + (1 << 44), A + (1 << 45)),
    (INVALID, 32, None, A, A),
    (INVALID, 32, A, None, A),
    (INVALID, 32, A, A + 0x1000, None),
    (ALIGN, 32, A + 4, A + 0x1000, A + 0x2000),
    (ALIGN, 32, A, A + 0x1004, A + 0x2000),
    (INVALID, 32, A, A + 0x70, A + 0x2000),
    (INVALID, 32, A, A + 0x1000, A + 0x101f),
    (INVALID, 33, A, A + 0x1000, A + 0x83),
])
def test_mx8_refuses(fp, want, n, x, codes, scales):
    L = fp.lib()
    assert L.fp_mx8_quantize(n, 0, x, codes, scales, None) == want
    assert L.fp_mx8_dequantize(n, 1, codes, scales, x, None) == want


def test_the_binding_refuses(fp):
    g = [torch.zeros(8), torch.zeros(8)]
    with pytest.raises(ValueError, match="device tensor"):
        fp.Params(g, g)
    with pytest.raises(ValueError, match="at least one"):
        fp.Params([])
    with pytest.raises(ValueError, match="device tensor"):
        fp.mx8_quantize(torch.zeros(32))
    with pytest.raises(ValueError, match="device tensor"):
        fp.mx8_dequantize(torch.zeros(32, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8))
