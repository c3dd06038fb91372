"""Products with a selection matrix: embedding lookup and its gradient, tokens
routed to experts and back, and the routing's gradients (``vspmm_embed`` and
the calls after it in include/vspmm.h).

    out = embedding(table, ids, scale=s)                   # ids: any shape
    grad = embedding_grad(grad_out, ids, table.shape[0], scale=s)

    r = route(experts, n_experts)                          # experts: tokens x top_k
    rows = dispatch(x, r.position)                         # rows sorted by expert
    ...                                                    # expert e: rows[r.offsets[e]:r.offsets[e + 1]]
    out = combine(rows, r.position, weights)
    grad_rows, grad_weights = combine_grad(grad_out, rows, r.position, weights)
    grad_x = dispatch_grad(grad_rows, r.position)

Argument marshalling only, as in the rest of the binding: every gradient is a
call of its own and nothing is recorded for autograd. Dense operands are
bfloat16, float16, float32 or float64; rows may be strided (any row stride,
elements of a row contiguous; others are copied). Ids and experts are int32 or
int64, and values outside their range select nothing. A given ``out`` or
``workspace`` shares no element with another array of its call (ValueError).
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _check, lib


def _public_raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# the current stream's handle without the Stream object around it: 0.1 us where
# the public way takes 2, of a 7 us call. A torch without this private function
# takes the public way; importing the package needs neither.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_raw_stream)

__all__ = ["Routing", "combine", "combine_grad", "dispatch", "dispatch_grad", "embedding",
           "embedding_grad", "embedding_grad_workspace", "route"]

ELTS = {torch.float32: 0, torch.float64: 1, torch.bfloat16: 2, torch.float16: 3}
INDICES = {torch.int32: 0, torch.int64: 1}


class Routing(NamedTuple):
    """Slots (token t's k-th expert is slot t * top_k + k) sorted by expert."""

    order: torch.Tensor     # int32 [slots]: the slot of each row
    position: torch.Tensor  # int32 [tokens, top_k]: the row p of each slot, ~p if dropped
    offsets: torch.Tensor   # int32 [n_experts + 1]: the first row of each expert


def _rows(t, name, shape=None, dtype=None, device=None, write=False):
    """A 2-d operand as (tensor, row stride): a read one is copied when the
    elements of its rows are not contiguous, a written one refused."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in ELTS or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'one of ' + str(list(ELTS))}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"{tuple(shape) if shape is not None else '(rows, width)'}")
    n, w = t.shape
    if t.is_contiguous():
        return t, w
    ld = t.stride(0) if n > 1 else w
    if (w > 1 and t.stride(1) != 1) or (write and ld < w):
        if write:
            raise ValueError(f"{name} must have contiguous rows that do not overlap")
        t = t.contiguous()
        ld = w
    return t, ld


def _index(t, name, device):
    if not isinstance(t, torch.Tensor) or t.dtype not in INDICES:
        raise TypeError(f"{name} must be an int32 or int64 tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.contiguous()


def _position(t, device):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32:
        raise TypeError("position must be an int32 tensor")
    if t.device != device:
        raise ValueError(f"position is on {t.device}, expected {device}")
    if t.dim() != 2:
        raise ValueError(f"position has shape {tuple(t.shape)}, expected (tokens, top_k)")
    return t.contiguous()


def _weights(t, shape, like, device):
    dtype = torch.float64 if like == torch.float64 else torch.float32
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"weights must be a {dtype} tensor")
    if t.device != device:
        raise ValueError(f"weights are on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"weights have shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.contiguous()


def _call(device, where, fn, *args):
    i = device.index
    if torch._C._cuda_getDevice() == i:
        st = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(i))
    if st:
        _check(st, where)


def _workspace(nbytes, workspace, device):
    if workspace is None:
        return (torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None), nbytes
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.numel() * workspace.element_size()


def _region(t, ld=None):
    """The bytes of a tensor's rows of stride ld (None: a contiguous tensor), as
    (address, rows, bytes of a row, bytes from row to row)."""
    if ld is None:
        return t.data_ptr(), 1, t.nbytes, 0
    (n, w), size = t.shape, t.element_size()
    return t.data_ptr(), n, w * size, ld * size


def _overlap(a, b):
    """Whether two regions share a byte."""
    (a0, na, wa, la), (b0, nb, wb, lb) = a, b
    if not (na and wa and nb and wb):
        return False
    if a0 + (na - 1) * la + wa <= b0 or b0 + (nb - 1) * lb + wb <= a0:
        return False
    # rows without gaps are one row
    if la <= wa:
        na, wa = 1, (na - 1) * la + wa
    if lb <= wb:
        nb, wb = 1, (nb - 1) * lb + wb
    if nb == 1:
        a0, na, wa, la, b0, nb, wb, lb = b0, nb, wb, lb, a0, na, wa, la
    if nb == 1:
        return True
    if na > 1 and la == lb:
        # only the distance of two rows counts: the first one of a against all of them
        b0, nb, na = b0 - (na - 1) * la, nb + na - 1, 1
    for r in range(na):
        at = a0 + r * la
        q = max((at - b0 - wb) // lb + 1, 0)  # the first row of b that ends behind it
        if q < nb and b0 + q * lb < at + wa:
            return True
    return False


def _apart(name, written, **others):
    """Refuses a written region (the caller's out or workspace) that overlaps
    another array of the call: rows written by one wave may be read by another."""
    for other, region in others.items():
        if _overlap(written, region):
            raise ValueError(f"{name} must not overlap {other}")


def embedding(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """``scale * table[ids]``, shaped ``ids.shape + (width,)``; an id outside the
    table gives a row of zeros (``vspmm_embed``). ``out``: 2-d, one row per id
    in order."""
    table, ld = _rows(table, "table")
    dev = table.device
    ids = _index(ids, "ids", dev)
    n, (v, w) = ids.numel(), table.shape
    if out is None:
        result, ld_out = table.new_empty(*ids.shape, w), w
    else:
        result, ld_out = _rows(out, "out", (n, w), table.dtype, dev, write=True)
        _apart("out", _region(result, ld_out), table=_region(table, ld), ids=_region(ids))
    _call(dev, "vspmm_embed", lib.vspmm_embed, ELTS[table.dtype], v, w, table.data_ptr(), ld,
          INDICES[ids.dtype], n, ids.data_ptr(), scale, result.data_ptr(), ld_out)
    return result


def embedding_grad_workspace(n_rows: int, width: int, n: int, dtype: torch.dtype) -> int:
    """Workspace bytes of :func:`embedding_grad` for ``n`` tokens (``dtype``: the
    type of ``grad_out``)."""
    need = ctypes.c_size_t(0)
    _check(lib.vspmm_embed_grad_workspace_size(ELTS[dtype], n_rows, width, n, ctypes.byref(need)),
           "vspmm_embed_grad_workspace_size")
    return int(need.value)


def embedding_grad(grad_out: torch.Tensor, ids: torch.Tensor, n_rows: int, scale: float = 1.0,
                   dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                   accumulate: bool = False, workspace: torch.Tensor | None = None):
    """The gradient of :func:`embedding` with respect to its table, n_rows x
    width (``vspmm_embed_grad``): row v is scale times the sum of grad_out's rows
    over the ids equal to v, in order. ``dtype`` (or out's type): grad_out's, or
    float32. ``accumulate`` adds to ``out``, touching only the rows selected.
    ``workspace``: see :func:`embedding_grad_workspace`; calls that overlap in
    time need one each (None: one is allocated for the call)."""
    if not isinstance(grad_out, torch.Tensor) or grad_out.dim() < 1:
        raise TypeError("grad_out must be a tensor of at least one dimension")
    dev = grad_out.device
    ids = _index(ids, "ids", dev)
    n, w = ids.numel(), grad_out.shape[-1]
    if tuple(grad_out.shape) not in ((*ids.shape, w), (n, w)):
        raise ValueError(f"grad_out has shape {tuple(grad_out.shape)}, expected "
                         f"{(*ids.shape, w)}")
    grad_out, ld = _rows(grad_out if grad_out.dim() == 2 else grad_out.reshape(n, w), "grad_out")
    need = embedding_grad_workspace(n_rows, w, n, grad_out.dtype)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        dtype = dtype or grad_out.dtype
        if dtype not in ELTS:
            raise TypeError(f"dtype must be one of {list(ELTS)}, got {dtype}")
        out, ld_out = grad_out.new_empty(n_rows, w, dtype=dtype), w
    else:
        out, ld_out = _rows(out, "out", (n_rows, w), dtype, dev, write=True)
        _apart("out", _region(out, ld_out), grad_out=_region(grad_out, ld), ids=_region(ids))
    ws, ws_bytes = _workspace(need, workspace, dev)
    if workspace is not None:
        _apart("workspace", (ws.data_ptr(), 1, min(need, ws_bytes), 0),
               grad_out=_region(grad_out, ld), ids=_region(ids), out=_region(out, ld_out))
    _call(dev, "vspmm_embed_grad", lib.vspmm_embed_grad, ELTS[grad_out.dtype], ELTS[out.dtype],
          n_rows, w, INDICES[ids.dtype], n, ids.data_ptr(), grad_out.data_ptr(), ld, scale,
          int(accumulate), out.data_ptr(), ld_out, ws.data_ptr() if ws is not None else None, ws_bytes)
    return out


def route(experts: torch.Tensor, n_experts: int,
          workspace: torch.Tensor | None = None) -> Routing:
    """Tokens sorted by expert (``vspmm_route``): ``experts`` is tokens x top_k;
    slots whose expert is outside [0, n_experts) are dropped. Stable: an
    expert's rows are in token order."""
    if not isinstance(experts, torch.Tensor) or experts.device.type != "cuda":
        raise ValueError("experts must be a CUDA tensor")
    dev = experts.device
    experts = _index(experts, "experts", dev)
    if experts.dim() != 2:
        raise ValueError(f"experts has shape {tuple(experts.shape)}, expected (tokens, top_k)")
    t, k = experts.shape
    need = ctypes.c_size_t(0)
    _check(lib.vspmm_route_workspace_size(t, k, n_experts, ctypes.byref(need)),
           "vspmm_route_workspace_size")
    ws, ws_bytes = _workspace(int(need.value), workspace, dev)
    if workspace is not None:
        _apart("workspace", (ws.data_ptr(), 1, min(need.value, ws_bytes), 0),
               experts=_region(experts))
    order = torch.empty(t * k, dtype=torch.int32, device=dev)
    position = torch.empty(t, k, dtype=torch.int32, device=dev)
    offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
    _call(dev, "vspmm_route", lib.vspmm_route, INDICES[experts.dtype], t, k, n_experts,
          experts.data_ptr(), order.data_ptr(), position.data_ptr(), offsets.data_ptr(),
          ws.data_ptr() if ws is not None else None, ws_bytes)
    return Routing(order, position, offsets)


def dispatch(x: torch.Tensor, position: torch.Tensor,
             out: torch.Tensor | None = None) -> torch.Tensor:
    """Every token's row copied to its experts' rows (``vspmm_dispatch``): x is
    tokens x width, the result (tokens * top_k) x width in the order of
    :func:`route`; rows of dropped slots are zeros."""
    x, ld = _rows(x, "x")
    dev = x.device
    position = _position(position, dev)
    t, k = position.shape
    w = x.shape[1]
    if x.shape[0] != t:
        raise ValueError(f"x has {x.shape[0]} rows, position {t}")
    if out is None:
        out, ld_out = x.new_empty(t * k, w), w
    else:
        out, ld_out = _rows(out, "out", (t * k, w), x.dtype, dev, write=True)
        _apart("out", _region(out, ld_out), x=_region(x, ld), position=_region(position))
    _call(dev, "vspmm_dispatch", lib.vspmm_dispatch, ELTS[x.dtype], t, k, w, x.data_ptr(), ld,
          position.data_ptr(), out.data_ptr(), ld_out)
    return out


def _sum_back(rows, position, weights, weighted, out):
    rows, ld = _rows(rows, "rows")
    dev = rows.device
    position = _position(position, dev)
    t, k = position.shape
    w = rows.shape[1]
    if rows.shape[0] != t * k:
        raise ValueError(f"rows has {rows.shape[0]} rows, expected {t * k}")
    if weighted:
        weights = _weights(weights, (t, k), rows.dtype, dev)
    if out is None:
        out, ld_out = rows.new_empty(t, w), w
    else:
        out, ld_out = _rows(out, "out", (t, w), rows.dtype, dev, write=True)
        _apart("out", _region(out, ld_out), rows=_region(rows, ld), position=_region(position))
        if weighted:
            _apart("out", _region(out, ld_out), weights=_region(weights))
    _call(dev, "vspmm_combine", lib.vspmm_combine, ELTS[rows.dtype], t, k, w, rows.data_ptr(), ld,
          position.data_ptr(), weights.data_ptr() if weighted else None, out.data_ptr(), ld_out)
    return out


def combine(rows: torch.Tensor, position: torch.Tensor, weights: torch.Tensor,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """The experts' rows back at their tokens (``vspmm_combine``): row t is the
    sum over k of ``weights[t, k] * rows[position[t, k]]``, dropped slots left
    out. weights: tokens x top_k, float32 (float64 for float64 rows)."""
    return _sum_back(rows, position, weights, True, out)


def dispatch_grad(grad_rows: torch.Tensor, position: torch.Tensor,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of :func:`dispatch` with respect to x: row t is the sum over
    k of ``grad_rows[position[t, k]]``, dropped slots left out."""
    return _sum_back(grad_rows, position, None, False, out)


def combine_grad(grad_out: torch.Tensor, rows: torch.Tensor, position: torch.Tensor,
                 weights: torch.Tensor, out: torch.Tensor | None = None):
    """The gradients of :func:`combine` (``vspmm_combine_grad``): ``(grad_rows,
    grad_weights)``, of the shapes and types of rows (written to ``out`` when
    given) and weights. A dropped slot's are zero."""
    rows, ld = _rows(rows, "rows")
    dev, dtype = rows.device, rows.dtype
    position = _position(position, dev)
    t, k = position.shape
    w = rows.shape[1]
    if rows.shape[0] != t * k:
        raise ValueError(f"rows has {rows.shape[0]} rows, expected {t * k}")
    grad_out, ld_grad_out = _rows(grad_out, "grad_out", (t, w), dtype, dev)
    weights = _weights(weights, (t, k), dtype, dev)
    if out is None:
        out, ld_out = rows.new_empty(t * k, w), w
    else:
        out, ld_out = _rows(out, "out", (t * k, w), dtype, dev, write=True)
        _apart("out", _region(out, ld_out), grad_out=_region(grad_out, ld_grad_out),
               rows=_region(rows, ld), position=_region(position), weights=_region(weights))
    grad_weights = weights.new_empty(t, k)
    _call(dev, "vspmm_combine_grad", lib.vspmm_combine_grad, ELTS[dtype], t, k, w,
          grad_out.data_ptr(), ld_grad_out, rows.data_ptr(), ld, position.data_ptr(),
          weights.data_ptr(), out.data_ptr(), ld_out, grad_weights.data_ptr())
    return out, grad_weights
