"""The selection products' argument checks, on the host before any device
work: the C interface's statuses and the binding's exceptions. Needs the built
library, no GPU."""

import ctypes

import pytest
import torch

import sparse_dense_matmul_amd as sdm

NULL, DIM, ENUM, WORKSPACE, UNSUPPORTED = 1, 2, 3, 5, 6
BIG = 2**31
D = ctypes.c_void_p(0x10000)  # never read: every call below is refused first


def test_embed_statuses():
    f = sdm.lib.vspmm_embed
    ok = [0, 10, 8, D, 8, 0, 4, D, 1.0, D, 8, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_0=4) == ENUM and call(_0=-1) == ENUM and call(_5=2) == ENUM
    assert call(_1=-1) == DIM and call(_1=BIG) == DIM and call(_2=-1) == DIM
    assert call(_2=BIG) == DIM and call(_6=-1) == DIM and call(_6=BIG) == DIM
    assert call(_4=-1) == DIM and call(_10=7) == DIM
    assert call(_3=None) == NULL and call(_7=None) == NULL and call(_9=None) == NULL
    # nothing to write: no pointer is needed and nothing is enqueued
    assert f(0, 0, 8, None, 8, 0, 0, None, 1.0, None, 8, None) == 0
    assert f(0, 10, 0, None, 0, 0, 4, D, 1.0, None, 0, None) == 0


def test_embed_grad_statuses():
    size = sdm.lib.vspmm_embed_grad_workspace_size
    n = ctypes.c_size_t()
    assert size(0, 10, 8, 4, None) == NULL
    assert size(4, 10, 8, 4, ctypes.byref(n)) == ENUM
    assert size(0, 2**31 - 1, 8, 4, ctypes.byref(n)) == DIM
    assert size(0, 10, -1, 4, ctypes.byref(n)) == DIM
    assert size(0, 10, 8, BIG, ctypes.byref(n)) == DIM
    for args in ((0, 0, 8, 4), (0, 10, 0, 4), (0, 10, 8, 0)):
        assert size(*args, ctypes.byref(n)) == 0 and n.value == 0
    assert size(0, 10, 8, 4, ctypes.byref(n)) == 0 and n.value > 0
    need = n.value
    f = sdm.lib.vspmm_embed_grad
    ok = [0, 0, 10, 8, 0, 4, D, D, 8, 1.0, 0, D, 8, D, need, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_0=9) == ENUM and call(_1=9) == ENUM and call(_4=2) == ENUM
    # grad's type is dout's, or float32 for a 16-bit dout
    for elt, grad in ((0, 1), (0, 2), (0, 3), (1, 0), (1, 2), (2, 1), (2, 3), (3, 1), (3, 2)):
        assert call(_0=elt, _1=grad) == ENUM
    assert call(_2=-1) == DIM and call(_3=BIG) == DIM and call(_5=-1) == DIM
    assert call(_8=-1) == DIM and call(_12=7) == DIM
    assert call(_6=None) == NULL and call(_7=None) == NULL and call(_11=None) == NULL
    assert call(_13=None) == WORKSPACE and call(_14=need - 1) == WORKSPACE
    assert call(_13=ctypes.c_void_p(0x10010)) == WORKSPACE  # not 256-byte aligned
    assert f(0, 0, 0, 8, 0, 4, D, D, 8, 1.0, 0, None, 8, None, 0, None) == 0


def test_route_statuses():
    size = sdm.lib.vspmm_route_workspace_size
    n = ctypes.c_size_t()
    assert size(4, 2, 8, None) == NULL
    for args in ((-1, 2, 8), (4, -1, 8), (4, 2, -1), (BIG, 1, 8), (2**30, 2, 8)):
        assert size(*args, ctypes.byref(n)) == DIM
    assert size(4, 2, 4097, ctypes.byref(n)) == UNSUPPORTED
    assert size(4, 2, 4096, ctypes.byref(n)) == 0
    for args in ((0, 4, 9), (4, 0, 9), (0, 0, 0)):
        assert size(*args, ctypes.byref(n)) == 0
    assert size(4, 2, 8, ctypes.byref(n)) == 0
    need = n.value
    f = sdm.lib.vspmm_route
    assert f(2, 4, 2, 8, D, D, D, D, D, need, None) == ENUM
    assert f(0, 4, -2, 8, D, D, D, D, D, need, None) == DIM
    assert f(0, 4, 2, 5000, D, D, D, D, D, 1 << 30, None) == UNSUPPORTED
    for i in range(4):
        p = [D, D, D, D]
        p[i] = None
        assert f(0, 4, 2, 8, *p, D, need, None) == NULL
    if need:
        assert f(0, 4, 2, 8, D, D, D, D, None, need, None) == WORKSPACE
        assert f(0, 4, 2, 8, D, D, D, D, D, need - 1, None) == WORKSPACE


def test_dispatch_and_combine_statuses():
    L = sdm.lib
    f = L.vspmm_dispatch
    assert f(7, 4, 2, 8, D, 8, D, D, 8, None) == ENUM
    assert f(0, -4, 2, 8, D, 8, D, D, 8, None) == DIM
    assert f(0, 2**30, 2, 8, D, 8, D, D, 8, None) == DIM
    assert f(0, 4, 2, BIG, D, 8, D, D, 8, None) == DIM
    assert f(0, 4, 2, 8, D, -8, D, D, 8, None) == DIM
    assert f(0, 4, 2, 8, D, 8, D, D, 7, None) == DIM
    assert f(0, 4, 2, 8, None, 8, D, D, 8, None) == NULL
    assert f(0, 4, 2, 8, D, 8, None, D, 8, None) == NULL
    assert f(0, 4, 2, 8, D, 8, D, None, 8, None) == NULL
    assert f(0, 0, 2, 8, None, 8, None, None, 8, None) == 0
    f = L.vspmm_combine
    assert f(7, 4, 2, 8, D, 8, D, D, D, 8, None) == ENUM
    assert f(0, 4, -2, 8, D, 8, D, D, D, 8, None) == DIM
    assert f(0, 4, 2, 8, D, 8, D, D, D, 7, None) == DIM
    assert f(0, 4, 2, 8, None, 8, D, D, D, 8, None) == NULL
    assert f(0, 4, 2, 8, D, 8, None, D, D, 8, None) == NULL
    assert f(0, 4, 2, 8, D, 8, D, D, None, 8, None) == NULL
    assert f(0, 4, 2, 0, None, 0, D, D, None, 0, None) == 0
    f = L.vspmm_combine_grad
    assert f(7, 4, 2, 8, D, 8, D, 8, D, D, D, 8, D, None) == ENUM
    assert f(0, 4, 2, -8, D, 8, D, 8, D, D, D, 8, D, None) == DIM
    assert f(0, 4, 2, 8, D, 8, D, 8, D, D, D, 7, D, None) == DIM
    for i in (4, 6, 8, 9, 10, 12):
        a = [0, 4, 2, 8, D, 8, D, 8, D, D, D, 8, D, None]
        a[i] = None
        assert f(*a) == NULL, i
    assert f(0, 0, 2, 8, None, 8, None, 8, None, None, None, 8, None, None) == 0


def test_binding_refusals():
    """Wrong types and host tensors are refused before the library is called."""
    x = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    pos = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        sdm.embedding(x, ids)  # a host tensor
    with pytest.raises(TypeError):
        sdm.embedding(x.int(), ids)
    with pytest.raises(TypeError):
        sdm.embedding([[1.0]], ids)
    with pytest.raises(ValueError):
        sdm.embedding_grad(x, ids, 10)
    with pytest.raises(TypeError):
        sdm.embedding_grad(x, ids.float(), 10)
    with pytest.raises(ValueError):
        sdm.route(pos, 4)
    with pytest.raises(ValueError):
        sdm.dispatch(x, pos)
    with pytest.raises(ValueError):
        sdm.combine(x, pos, torch.zeros(2, 2))
    with pytest.raises(ValueError):
        sdm.combine_grad(x, x, pos, torch.zeros(2, 2))
    with pytest.raises(sdm.VspmmError) as e:
        sdm.embedding_grad_workspace(-1, 8, 4, torch.float32)
    assert e.value.status == DIM


@pytest.mark.parametrize("width", [1, 7, 64, 300, 1024, 4096, 20_000])
def test_workspaces_do_not_shrink(width):
    """A workspace for n tokens serves every shorter list: the size does not
    fall as n grows, also where the sort or the segments change."""
    size, n = sdm.lib.vspmm_embed_grad_workspace_size, ctypes.c_size_t()
    lengths = sorted({*range(1, 300, 7), *(2**k + d for k in range(5, 22) for d in (-1, 0, 1)),
                      *range(4000, 140_000, 777)})
    for elt in (0, 1, 2):
        last = 0
        for t in lengths:
            assert size(elt, 50_000, width, t, ctypes.byref(n)) == 0
            assert n.value >= last, (elt, t)
            last = n.value
    last = 0
    for t in lengths:
        assert sdm.lib.vspmm_route_workspace_size(t, 3, 500, ctypes.byref(n)) == 0
        assert n.value >= last, t
        last = n.value


def test_workspace_follows_documented_limits():
    size, n = sdm.lib.vspmm_embed_grad_workspace_size, ctypes.c_size_t()
    assert size(2, 100, 64, 2**30, ctypes.byref(n)) == 0
    assert size(2, 100, 512, 2**30, ctypes.byref(n)) == 0
    assert size(2, 100, 512, 2**30 + 1, ctypes.byref(n)) == UNSUPPORTED
    assert size(2, 100, 2**14, 2**25, ctypes.byref(n)) == 0
    assert size(2, 100, 2**14, 2**26, ctypes.byref(n)) == UNSUPPORTED
    assert size(2, 100, 2**24 + 1, 4, ctypes.byref(n)) == UNSUPPORTED
    f = sdm.lib.vspmm_embed
    assert f(2, 10, 2**24 + 1, D, 2**25, 0, 4, D, 1.0, D, 2**25, None) == UNSUPPORTED
