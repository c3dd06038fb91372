"""Microscaled 4-bit matrices, products with them, and a whole mixture-of-experts
layer for a few tokens (``vspmm_mx4_quantize`` and the calls after it in
include/vspmm.h).

    w = quantize_mx4(weight)                    # n x width, 17 bytes for 32 values
    y = matmul_mx4(x, w)                        # x @ weight.T, x dense: m x width
    grad_x = matmul_mx4_grad(grad_y, w)         # grad_y @ weight
    y = matmul_mx4(quantize_mx4(x), w)          # both sides in 4 bits

    # the gradients of a product with both sides in 4 bits, each side quantised
    # along what it contracts
    grad_x = matmul_mx4(quantize_mx4(grad_y), quantize_mx4(weight, transpose=True))
    grad_w = matmul_mx4(quantize_mx4(grad_y, transpose=True), quantize_mx4(x, transpose=True))

    out = expert_mlp(x, experts, weights, gate, up, down)   # experts, weights: tokens x top_k

Argument marshalling only, as in the rest of the binding: gradients are calls of
their own and nothing is recorded for autograd. Dense operands are bfloat16 or
float16 (quantisation takes float32, too); rows may be strided (any row stride,
elements of a row contiguous; others are copied). A given ``out`` or
``workspace`` shares no element with another array of its call (ValueError).
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _check, lib
from .selection import (ELTS, _apart, _call, _index, _overlap, _region, _rows, _weights,
                        _workspace)

__all__ = ["Mx4", "dequantize_mx4", "expert_mlp", "expert_mlp_workspace", "matmul_mx4",
           "matmul_mx4_grad", "quantize_mx4"]

BLOCK = 32
ELT_MX4 = 4
DENSE = (torch.bfloat16, torch.float16)
QUANTIZED = (torch.bfloat16, torch.float16, torch.float32)
ACTIVATIONS = {"silu": 0, "gelu": 1}


class Mx4(NamedTuple):
    """A microscaled 4-bit matrix, or one for each expert (3-d)."""

    codes: torch.Tensor   # uint8 [.., rows, 16 * blocks]: value 2 j in the low half of byte j
    scales: torch.Tensor  # uint8 [.., rows, blocks]: byte b is the scale 2^(b - 127) of 32 values
    width: int            # values of a row; codes past it are zero


class _Struct(ctypes.Structure):  # vspmm_mx4
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("ld_codes", ctypes.c_int64), ("ld_scales", ctypes.c_int64)]


class _Expert(ctypes.Structure):  # vspmm_expert_matrix
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("stride", ctypes.c_int64),
                ("scales", ctypes.c_void_p), ("ld_scales", ctypes.c_int64),
                ("stride_scales", ctypes.c_int64)]


def _dense(t, name, types, shape=None, dtype=None, device=None, write=False):
    if isinstance(t, torch.Tensor) and t.dtype not in types:
        raise TypeError(f"{name} must be one of {list(types)}, got {t.dtype}")
    return _rows(t, name, shape, dtype, device, write)


def _refuse(a, name, dims, device):
    """Raises for the first thing that is wrong with an Mx4."""
    codes, scales, width = a
    for t, part in ((codes, "codes"), (scales, "scales")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
            raise TypeError(f"{name}.{part} must be a uint8 tensor")
    if codes.dim() != dims:
        raise ValueError(f"{name}.codes has shape {tuple(codes.shape)}, expected {dims} dimensions")
    if width < 0:
        raise ValueError(f"{name}.width is negative")
    blocks = (width + BLOCK - 1) // BLOCK
    for t, part, row, on in ((codes, "codes", 16 * blocks, device),
                             (scales, "scales", blocks, codes.device)):
        if not t.is_cuda:
            raise ValueError(f"{name}.{part} must be a CUDA tensor")
        if on is not None and t.device != on:
            raise ValueError(f"{name}.{part} is on {t.device}, expected {on}")
        shape = (*codes.shape[:-1], row)
        if t.shape != shape:
            raise ValueError(f"{name}.{part} has shape {tuple(t.shape)}, expected {shape}")


def _mx4(a, name, dims, device=None):
    """An Mx4's checked arrays: (codes, scales, rows, width). One condition, since
    a call for one token takes less time on the device than on the host."""
    if not isinstance(a, Mx4):
        raise TypeError(f"{name} must be an Mx4")
    codes, scales, width = a
    if not (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor)):
        _refuse(a, name, dims, device)
    shape, blocks = codes.shape, (width + BLOCK - 1) // BLOCK
    if (len(shape) != dims or shape[-1] != 16 * blocks or scales.shape != (*shape[:-1], blocks)
            or codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or width < 0
            or not codes.is_cuda or scales.device != (device or codes.device)
            or (device is not None and codes.device != device)):
        _refuse(a, name, dims, device)
    # rows may be strided, the bytes of one are contiguous
    if codes.stride(-1) != 1 and shape[-1] > 1:
        codes = codes.contiguous()
    if scales.stride(-1) != 1 and blocks > 1:
        scales = scales.contiguous()
    return codes, scales, shape[-2], width


def _struct(codes, scales):
    return _Struct(codes.data_ptr(), scales.data_ptr(), codes.stride(-2), scales.stride(-2))


def _mx4_regions(name, codes, scales):
    return {f"{name}.codes": _region(codes, codes.stride(0)),
            f"{name}.scales": _region(scales, scales.stride(0))}


def quantize_mx4(x: torch.Tensor, transpose: bool = False) -> Mx4:
    """The rows of ``x`` (2-d) in 4 bits, or those of its transpose
    (``vspmm_mx4_quantize``): a block of 32 values shares the power of two of its
    largest magnitude, and each is rounded to the nearest code, ties to even. A
    block with an infinity or NaN becomes NaN."""
    x, ld = _dense(x, "x", QUANTIZED)
    rows, width = x.shape
    n, k = (width, rows) if transpose else (rows, width)
    blocks = (k + BLOCK - 1) // BLOCK
    codes = torch.empty(n, 16 * blocks, dtype=torch.uint8, device=x.device)
    scales = torch.empty(n, blocks, dtype=torch.uint8, device=x.device)
    _call(x.device, "vspmm_mx4_quantize", lib.vspmm_mx4_quantize, ELTS[x.dtype], int(transpose),
          rows, width, x.data_ptr(), ld, codes.data_ptr(), scales.data_ptr())
    return Mx4(codes, scales, k)


def dequantize_mx4(x: Mx4, dtype: torch.dtype = torch.bfloat16,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of a 4-bit matrix (``vspmm_mx4_dequantize``), in bfloat16,
    float16 or float32 (``dtype``, or out's)."""
    codes, scales, rows, width = _mx4(x, "x", 2)
    dev = codes.device
    if out is None:
        if dtype not in QUANTIZED:
            raise TypeError(f"dtype must be one of {list(QUANTIZED)}, got {dtype}")
        out, ld = torch.empty(rows, width, dtype=dtype, device=dev), width
    else:
        out, ld = _dense(out, "out", QUANTIZED, (rows, width), None, dev, write=True)
        _apart("out", _region(out, ld), **_mx4_regions("x", codes, scales))
    _call(dev, "vspmm_mx4_dequantize", lib.vspmm_mx4_dequantize, ELTS[out.dtype], rows, width,
          ctypes.byref(_struct(codes, scales)), out.data_ptr(), ld)
    return out


def matmul_mx4(x: torch.Tensor | Mx4, w: Mx4, dtype: torch.dtype | None = None,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """``x`` times the transpose of ``w`` (n x width, 4 bits): m x n, float32 sums
    of exact products, rounded once. ``x`` is dense (``vspmm_mx4_matmul``; the
    result has its type) or in 4 bits itself (``vspmm_mx4_matmul_mx4``; the result
    is ``dtype``, out's type or bfloat16)."""
    if isinstance(x, Mx4):
        xc, xs, m, width = _mx4(x, "x", 2)
        dev, types = xc.device, QUANTIZED
        dtype = dtype or (out.dtype if isinstance(out, torch.Tensor) else torch.bfloat16)
    else:
        x, ld = _dense(x, "x", DENSE)
        (m, width), dev, types = x.shape, x.device, DENSE
        if dtype is not None and dtype != x.dtype:
            raise TypeError(f"dtype must be x's, {x.dtype}, got {dtype}")
        dtype = x.dtype
    if dtype not in types:
        raise TypeError(f"dtype must be one of {list(types)}, got {dtype}")
    codes, scales, n, w_width = _mx4(w, "w", 2, dev)
    if w_width != width:
        raise ValueError(f"w has width {w_width}, x {width}")
    if out is None:
        out, ld_out = torch.empty(m, n, dtype=dtype, device=dev), n
    else:
        out, ld_out = _dense(out, "out", types, (m, n), dtype, dev, write=True)
        read = _mx4_regions("x", xc, xs) if isinstance(x, Mx4) else {"x": _region(x, ld)}
        _apart("out", _region(out, ld_out), **read, **_mx4_regions("w", codes, scales))
    ws = _struct(codes, scales)
    if isinstance(x, Mx4):
        _call(dev, "vspmm_mx4_matmul_mx4", lib.vspmm_mx4_matmul_mx4, ELTS[dtype], m, n, width,
              ctypes.byref(_struct(xc, xs)), ctypes.byref(ws), out.data_ptr(), ld_out)
    else:
        _call(dev, "vspmm_mx4_matmul", lib.vspmm_mx4_matmul, ELTS[dtype], m, n, width,
              x.data_ptr(), ld, ctypes.byref(ws), out.data_ptr(), ld_out)
    return out


def matmul_mx4_grad(grad_out: torch.Tensor, w: Mx4,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of :func:`matmul_mx4` with respect to a dense x
    (``vspmm_mx4_matmul_grad``): ``grad_out`` (m x n) times ``w`` (n x width)."""
    grad_out, ld = _dense(grad_out, "grad_out", DENSE)
    (m, n), dev = grad_out.shape, grad_out.device
    codes, scales, rows, width = _mx4(w, "w", 2, dev)
    if rows != n:
        raise ValueError(f"w has {rows} rows, grad_out {n} columns")
    if out is None:
        out, ld_out = grad_out.new_empty(m, width), width
    else:
        out, ld_out = _dense(out, "out", DENSE, (m, width), grad_out.dtype, dev, write=True)
        _apart("out", _region(out, ld_out), grad_out=_region(grad_out, ld),
               **_mx4_regions("w", codes, scales))
    _call(dev, "vspmm_mx4_matmul_grad", lib.vspmm_mx4_matmul_grad, ELTS[grad_out.dtype], m, n,
          width, grad_out.data_ptr(), ld, ctypes.byref(_struct(codes, scales)), out.data_ptr(),
          ld_out)
    return out


def _expert_matrix(t, name, like, shape, device):
    """One matrix of every expert as (its struct, whether in 4 bits, arrays to keep)."""
    if isinstance(t, Mx4):
        codes, scales, rows, width = _mx4(t, name, 3, device)
        if (codes.shape[0], rows, width) != shape:
            raise ValueError(f"{name} is {(codes.shape[0], rows, width)}, expected {shape}")
        return _Expert(codes.data_ptr(), codes.stride(1), codes.stride(0), scales.data_ptr(),
                       scales.stride(1), scales.stride(0)), True, (codes, scales)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor or an Mx4")
    if t.dtype != like:
        raise TypeError(f"{name} must be {like} or an Mx4, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.stride(2) != 1 and shape[2] > 1:
        t = t.contiguous()
    return _Expert(t.data_ptr(), t.stride(1), t.stride(0), None, 0, 0), False, (t,)


def _experts_apart(name, written, matrices):
    """_apart for arrays of every expert, as (name, tensor): one look at the bytes
    from the first to the last, and at each expert's rows only if those overlap."""
    for other, m in matrices:
        if not m.numel():
            continue
        last = sum((n - 1) * stride for n, stride in zip(m.shape, m.stride()))
        whole = (m.data_ptr(), 1, (last + 1) * m.element_size(), 0)
        if not _overlap(written, whole):
            continue
        if m.is_contiguous():
            _apart(name, written, **{other: whole})
        for e in range(m.shape[0]):
            _apart(name, written, **{f"{other}[{e}]": _region(m[e], m.stride(1))})


def expert_mlp_workspace(n_tokens: int, top_k: int, n_experts: int, width: int,
                         hidden: int) -> int:
    """Workspace bytes of :func:`expert_mlp`."""
    need = ctypes.c_size_t(0)
    _check(lib.vspmm_expert_mlp_workspace_size(n_tokens, top_k, n_experts, width, hidden,
                                               ctypes.byref(need)),
           "vspmm_expert_mlp_workspace_size")
    return int(need.value)


def expert_mlp(x: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor,
               gate: torch.Tensor | Mx4, up: torch.Tensor | Mx4, down: torch.Tensor | Mx4,
               activation: str = "silu", out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """A whole mixture-of-experts layer for a few tokens, up to 1,024
    (``vspmm_expert_mlp``): row t is the sum over k of ``weights[t, k]`` times
    ``down[e] @ (act(gate[e] @ x[t]) * (up[e] @ x[t]))``, e = ``experts[t, k]``.

    experts: tokens x top_k, int32 or int64; choices outside the experts held add
    nothing. weights: float32. gate and up: experts x hidden x width, down: experts
    x width x hidden, all of x's type (strided views are served) or all Mx4.
    activation: "silu" or "gelu". ``workspace``: see :func:`expert_mlp_workspace`;
    calls that overlap in time need one each (None: one is allocated for the
    call)."""
    x, ld = _dense(x, "x", DENSE)
    (t, width), dev = x.shape, x.device
    experts = _index(experts, "experts", dev)
    if experts.dim() != 2 or experts.shape[0] != t:
        raise ValueError(f"experts has shape {tuple(experts.shape)}, expected ({t}, top_k)")
    k = experts.shape[1]
    weights = _weights(weights, (t, k), torch.float32, dev)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, got {activation!r}")
    shape = gate.codes if isinstance(gate, Mx4) else gate
    if not isinstance(shape, torch.Tensor):
        raise TypeError("gate must be a tensor or an Mx4")
    shape = shape.shape
    if len(shape) != 3:
        raise ValueError(f"gate has shape {tuple(shape)}, expected (experts, hidden, width)")
    n, hidden = shape[0], shape[1]
    gate, mx4, a = _expert_matrix(gate, "gate", x.dtype, (n, hidden, width), dev)
    up, mx4_up, b = _expert_matrix(up, "up", x.dtype, (n, hidden, width), dev)
    down, mx4_down, c = _expert_matrix(down, "down", x.dtype, (n, width, hidden), dev)
    if mx4 != mx4_up or mx4 != mx4_down:
        raise TypeError("gate, up and down must all be in 4 bits, or none")
    need = expert_mlp_workspace(t, k, n, width, hidden)
    read = matrices = None
    if out is not None or workspace is not None:
        read = {"x": _region(x, ld), "experts": _region(experts), "weights": _region(weights)}
        matrices = [(name if len(arrays) == 1 else f"{name}.{part}", m)
                    for name, arrays in (("gate", a), ("up", b), ("down", c))
                    for part, m in zip(("codes", "scales"), arrays)]
    if out is None:
        out, ld_out = x.new_empty(t, width), width
    else:
        out, ld_out = _dense(out, "out", DENSE, (t, width), x.dtype, dev, write=True)
        _apart("out", _region(out, ld_out), **read)
        _experts_apart("out", _region(out, ld_out), matrices)
    ws, ws_bytes = _workspace(need, workspace, dev)
    if workspace is not None:
        region = ws.data_ptr(), 1, min(need, ws_bytes), 0
        _apart("workspace", region, out=_region(out, ld_out), **read)
        _experts_apart("workspace", region, matrices)
    _call(dev, "vspmm_expert_mlp", lib.vspmm_expert_mlp, ELTS[x.dtype],
          ELT_MX4 if mx4 else ELTS[x.dtype], 0 if experts.dtype == torch.int32 else 1,
          ACTIVATIONS[activation], t, k, n, width, hidden, x.data_ptr(), ld, experts.data_ptr(),
          weights.data_ptr(), ctypes.byref(gate), ctypes.byref(up), ctypes.byref(down),
          out.data_ptr(), ld_out, ws.data_ptr() if ws is not None else None, ws_bytes)
    return out
