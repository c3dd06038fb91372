"""Argument checks of the 4-bit products and the experts' layer, on the host
before any device work: the C interface's statuses, and the binding's exceptions
(those on device tensors need a GPU, but launch nothing)."""

import ctypes

import pytest
import torch

import sparse_dense_matmul_amd as sdm
from helpers import need_gpu
from sparse_dense_matmul_amd.mx4 import _Expert, _Struct

NULL, DIM, ENUM, WORKSPACE, UNSUPPORTED = 1, 2, 3, 5, 6
F32, F64, BF16, F16, MX4 = range(5)
BIG, ROWS, WIDE = 2**31, 2**30 + 1, 2**24 + 1
D = ctypes.c_void_p(0x10000)  # never read: every call below is refused first


def mx4(codes=0x10000, scales=0x20000, ld_codes=16, ld_scales=1):
    return _Struct(codes, scales, ld_codes, ld_scales)


def caller(f, ok):
    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = ctypes.byref(v) if isinstance(v, ctypes.Structure) else v
        return f(*a)
    return call


def bad_matrices(call, i):
    """Refusals of a 4-bit matrix at argument i."""
    at = f"_{i}"
    assert call(**{at: None}) == NULL
    assert call(**{at: mx4(codes=None)}) == NULL and call(**{at: mx4(scales=None)}) == NULL
    assert call(**{at: mx4(ld_codes=-1)}) == DIM and call(**{at: mx4(ld_scales=-1)}) == DIM


def test_quantize_statuses():
    call = caller(sdm.lib.vspmm_mx4_quantize, [BF16, 0, 4, 8, D, 8, D, D, None])
    for elt in (F64, MX4, 5, -1):
        assert call(_0=elt) == ENUM
    assert call(_2=-1) == DIM and call(_2=BIG) == DIM and call(_3=-1) == DIM and call(_5=-1) == DIM
    assert call(_2=ROWS) == UNSUPPORTED and call(_3=WIDE) == UNSUPPORTED
    assert call(_1=1, _2=WIDE) == UNSUPPORTED
    assert call(_4=None) == NULL and call(_6=None) == NULL and call(_7=None) == NULL
    assert call(_2=0, _4=None, _6=None, _7=None) == 0 and call(_3=0, _4=None, _6=None, _7=None) == 0


def test_dequantize_statuses():
    w = mx4()
    call = caller(sdm.lib.vspmm_mx4_dequantize, [BF16, 4, 8, ctypes.byref(w), D, 8, None])
    for elt in (F64, MX4, 5, -1):
        assert call(_0=elt) == ENUM
    assert call(_1=-1) == DIM and call(_2=-1) == DIM and call(_2=BIG) == DIM
    assert call(_1=ROWS) == UNSUPPORTED and call(_2=WIDE) == UNSUPPORTED
    assert call(_5=7) == DIM and call(_5=-1) == DIM and call(_4=None) == NULL
    bad_matrices(call, 3)
    assert call(_1=0, _3=mx4(None, None), _4=None) == 0


@pytest.mark.parametrize("name", ["vspmm_mx4_matmul", "vspmm_mx4_matmul_grad"])
def test_product_statuses(name):
    w = mx4()
    grad = name.endswith("grad")
    call = caller(getattr(sdm.lib, name), [BF16, 4, 8, 8, D, 8, ctypes.byref(w), D, 8, None])
    for elt in (F32, F64, MX4, 5, -1):
        assert call(_0=elt) == ENUM
    for i in (1, 2, 3):
        assert call(**{f"_{i}": -1}) == DIM and call(**{f"_{i}": BIG}) == DIM
    assert call(_1=ROWS) == UNSUPPORTED and call(_2=ROWS) == UNSUPPORTED and call(_3=WIDE) == UNSUPPORTED
    assert call(_2=WIDE, _8=WIDE) == UNSUPPORTED
    assert call(_5=-1) == DIM and call(_8=7) == DIM and call(_8=-1) == DIM
    assert call(_4=None) == NULL and call(_7=None) == NULL
    bad_matrices(call, 6)
    assert call(_1=0, _4=None, _7=None) == 0
    assert call(**{"_3" if grad else "_2": 0}, _6=mx4(None, None), _7=None) == 0


def test_product_of_two_statuses():
    x, w = mx4(), mx4()
    call = caller(sdm.lib.vspmm_mx4_matmul_mx4,
                  [BF16, 4, 8, 8, ctypes.byref(x), ctypes.byref(w), D, 8, None])
    for elt in (F64, MX4, 5, -1):
        assert call(_0=elt) == ENUM
    for i in (1, 2, 3):
        assert call(**{f"_{i}": -1}) == DIM and call(**{f"_{i}": BIG}) == DIM
    assert call(_1=ROWS) == UNSUPPORTED and call(_2=ROWS) == UNSUPPORTED and call(_3=WIDE) == UNSUPPORTED
    assert call(_7=7) == DIM and call(_6=None) == NULL
    bad_matrices(call, 4)
    bad_matrices(call, 5)
    assert call(_1=0, _4=mx4(None, None), _6=None) == 0 and call(_2=0, _5=mx4(None, None), _6=None) == 0


def test_expert_mlp_statuses():
    size = sdm.lib.vspmm_expert_mlp_workspace_size
    n = ctypes.c_size_t()
    assert size(4, 2, 8, 16, 32, None) == NULL
    for i in range(5):
        a = [4, 2, 8, 16, 32]
        a[i] = -1
        assert size(*a, ctypes.byref(n)) == DIM
        a[i] = BIG
        assert size(*a, ctypes.byref(n)) == DIM
        a[i] = 0
        assert size(*a, ctypes.byref(n)) == 0 and n.value == 0
    for a in ((1025, 2, 8, 16, 32), (4, 4097, 8, 16, 32), (4, 2, 4097, 16, 32), (4, 2, 8, WIDE, 32),
              (4, 2, 8, 16, WIDE)):
        assert size(*a, ctypes.byref(n)) == UNSUPPORTED
    assert size(1024, 4096, 4096, 2**24, 2**24, ctypes.byref(n)) == 0
    assert n.value >= 1024 * 4096 * 2**24 * 4
    assert size(4, 2, 8, 16, 32, ctypes.byref(n)) == 0 and n.value > 0
    need = n.value
    m = [_Expert(0x10000, 16, 512, 0x20000, 1, 32) for _ in range(3)]
    call = caller(sdm.lib.vspmm_expert_mlp,
                  [BF16, BF16, 0, 0, 4, 2, 8, 16, 32, D, 16, D, D, *map(ctypes.byref, m), D, 16, D, need, None])
    for elt in (F32, F64, MX4, 5, -1):
        assert call(_0=elt) == ENUM
    for elt in (F32, F64, F16, 5, -1):
        assert call(_1=elt) == ENUM
    assert call(_2=2) == ENUM and call(_3=2) == ENUM and call(_3=-1) == ENUM
    for i in range(4, 9):
        assert call(**{f"_{i}": -1}) == DIM and call(**{f"_{i}": BIG}) == DIM
    assert call(_4=1025) == UNSUPPORTED and call(_6=4097) == UNSUPPORTED and call(_8=WIDE) == UNSUPPORTED
    assert call(_10=-1) == DIM and call(_17=15) == DIM
    for i in (9, 11, 12, 13, 14, 15, 16):
        assert call(**{f"_{i}": None}) == NULL
    for i in (13, 14, 15):
        assert call(**{f"_{i}": _Expert(None, 16, 512, 0x20000, 1, 32)}) == NULL
        assert call(**{f"_{i}": _Expert(0x10000, -1, 512, 0x20000, 1, 32)}) == DIM
        assert call(**{f"_{i}": _Expert(0x10000, 16, -1, 0x20000, 1, 32)}) == DIM
        assert call(_1=MX4, **{f"_{i}": _Expert(0x10000, 16, 512, None, 1, 32)}) == NULL
        assert call(_1=MX4, **{f"_{i}": _Expert(0x10000, 16, 512, 0x20000, -1, 32)}) == DIM
        assert call(_1=MX4, **{f"_{i}": _Expert(0x10000, 16, 512, 0x20000, 1, -1)}) == DIM
    assert call(_18=None) == WORKSPACE and call(_19=need - 1) == WORKSPACE
    assert call(_18=ctypes.c_void_p(0x10010)) == WORKSPACE  # not 256-byte aligned
    assert call(_4=0, _9=None, _16=None) == 0 and call(_7=0, _9=None, _16=None, _10=0, _17=0) == 0


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = sdm.Mx4(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8), 64)
    for f in (lambda: sdm.quantize_mx4(x), lambda: sdm.dequantize_mx4(w), lambda: sdm.matmul_mx4(x, w),
              lambda: sdm.matmul_mx4(w, w), lambda: sdm.matmul_mx4_grad(x[:, :8], w),
              lambda: sdm.expert_mlp(x, None, None, None, None, None)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: sdm.quantize_mx4(x.double()), lambda: sdm.quantize_mx4(3), lambda: sdm.dequantize_mx4(x),
              lambda: sdm.matmul_mx4(x.float(), w), lambda: sdm.matmul_mx4_grad(x.float(), w)):
        with pytest.raises(TypeError):
            f()


@pytest.mark.gpu
def test_binding_refusals():
    dev = need_gpu()
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    w = sdm.quantize_mx4(torch.zeros(8, 64, device=dev))
    g = torch.zeros(4, 8, dtype=torch.bfloat16, device=dev)

    def refused(error, f, *a, **kw):
        with pytest.raises(error):
            f(*a, **kw)
    refused(ValueError, sdm.quantize_mx4, x[0])
    refused(TypeError, sdm.matmul_mx4, x, x)
    refused(TypeError, sdm.matmul_mx4, x, w, dtype=torch.float32)
    refused(TypeError, sdm.matmul_mx4, w, w, dtype=torch.float64)
    refused(TypeError, sdm.dequantize_mx4, w, torch.float64)
    refused(ValueError, sdm.matmul_mx4, x[:, :32], w)
    refused(ValueError, sdm.matmul_mx4_grad, x, w)
    for bad in (w._replace(width=65), w._replace(width=32), w._replace(width=-1), w._replace(scales=w.scales[:7]),
                w._replace(codes=w.codes[0]), w._replace(scales=w.scales.cpu())):
        refused(ValueError, sdm.matmul_mx4, x, bad)
        refused(ValueError, sdm.dequantize_mx4, bad)
    refused(TypeError, sdm.matmul_mx4, x, w._replace(codes=w.codes.int()))
    # out: shape, type, rows that overlap, and memory shared with what is read
    refused(ValueError, sdm.matmul_mx4, x, w, out=x[:, :7])
    refused(TypeError, sdm.matmul_mx4, x, w, out=g.half())
    refused(ValueError, sdm.matmul_mx4, x, w, out=g[:1].expand(4, 8))
    refused(ValueError, sdm.matmul_mx4, x, w, out=x[:, 8:16])
    refused(ValueError, sdm.matmul_mx4_grad, x[:, :8], w, out=x)
    raw = w.codes.view(torch.bfloat16)  # 8 x 16
    refused(ValueError, sdm.matmul_mx4, x, w, out=raw[:4, :8])
    refused(ValueError, sdm.matmul_mx4, w, w, out=raw[:8, :8])
    refused(ValueError, sdm.dequantize_mx4, sdm.Mx4(w.codes[:2], w.scales[:2], 64), out=raw.view(-1, 64)[:2])
    assert sdm.matmul_mx4(x, w, out=torch.zeros(4, 20, dtype=x.dtype, device=dev)[:, 5:13]).shape == (4, 8)


@pytest.mark.gpu
def test_expert_binding_refusals():
    dev = need_gpu()
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    x, gate, up, down = b(4, 16), b(3, 32, 16), b(3, 32, 16), b(3, 16, 32)
    e, w = torch.zeros(4, 2, dtype=torch.int64, device=dev), torch.zeros(4, 2, device=dev)
    ok = dict(x=x, experts=e, weights=w, gate=gate, up=up, down=down)

    def refused(error, **kw):
        with pytest.raises(error):
            sdm.expert_mlp(**{**ok, **kw})
    refused(TypeError, x=x.float())
    refused(TypeError, experts=e.short())
    refused(TypeError, weights=w.double())
    refused(TypeError, gate=gate.half())
    refused(TypeError, gate=sdm.Mx4(torch.zeros(3, 32, 16, dtype=torch.uint8, device=dev),
                                    torch.zeros(3, 32, 1, dtype=torch.uint8, device=dev), 16))
    refused(ValueError, experts=e[:3])
    refused(ValueError, experts=e[:, 0])
    refused(ValueError, weights=w[:, :1])
    refused(ValueError, gate=gate[0])
    refused(ValueError, up=up[:2])
    refused(ValueError, down=up)
    refused(ValueError, activation="relu")
    refused(ValueError, experts=e.cpu())
    refused(ValueError, up=up.cpu())
    refused(ValueError, out=x)
    refused(ValueError, out=b(4, 15))
    refused(ValueError, out=gate[1, :4])
    refused(ValueError, out=gate[:, :, :][2, 3:7])
    refused(ValueError, workspace=gate)
    refused(sdm.VspmmError, workspace=torch.zeros(16, dtype=torch.uint8, device=dev))
    refused(sdm.VspmmError, x=b(1025, 16), experts=e[:1].expand(1025, 2), weights=w[:1].expand(1025, 2))
    n = sdm.expert_mlp_workspace(4, 2, 3, 16, 32)
    ws = torch.zeros(n + 512, dtype=torch.uint8, device=dev)
    refused(sdm.VspmmError, workspace=ws[8:])
    refused(ValueError, workspace=ws, out=ws[:128].view(torch.bfloat16).view(4, 16))
    assert sdm.expert_mlp(**ok, workspace=ws).shape == (4, 16)
