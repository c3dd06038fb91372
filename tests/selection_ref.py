"""The selection products from their definitions, in float64 numpy, with the
bounds their float results are held to.

Bounds. A value in a type with unit roundoff u (half a step: 2^-24 float32,
2^-53 float64, 2^-8 bfloat16, 2^-11 float16) is within u of the exact one
relative to it, plus half the type's smallest step for results below its
normal range. A float sum of m products, in any order, is within m * ua of the
exact one relative to the sum of magnitudes (ua the sum's unit roundoff; each
product's rounding, or the fused one, counts as one of the m additions), to
first order; the second order is below 1e-3 of that for m * ua < 1e-3, covered
by the factor 1.01. The result is then rounded once to its type."""

import numpy as np
import torch

U = {torch.float32: 2.0**-24, torch.float64: 2.0**-53, torch.bfloat16: 2.0**-8,
     torch.float16: 2.0**-11}
# half the smallest step
TINY = {torch.float32: 2.0**-150, torch.float64: 0.0, torch.bfloat16: 2.0**-134,
        torch.float16: 2.0**-25}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def acc(dtype):
    return torch.float64 if dtype == torch.float64 else torch.float32


def check(got, want, terms, magnitude, dtype, where=""):
    """|got - want| within the bound for a sum of `terms` products of total
    magnitude `magnitude` in acc(dtype), rounded once to got's type."""
    g = f64(got)
    assert g.shape == want.shape, (where, g.shape, want.shape)
    sums = np.asarray(terms) * U[acc(dtype)] * magnitude * 1.01
    bound = sums + U[got.dtype] * (np.abs(want) + sums) + TINY[got.dtype]
    bad = np.abs(g - want) > bound
    assert not bad.any(), (where, int(bad.sum()), np.argwhere(bad)[:3],
                           float(np.max(np.abs(g - want) / np.maximum(bound, 1e-300))))


def embedding(table, ids, scale):
    """(out, magnitude)"""
    v = table.shape[0]
    ok = (ids >= 0) & (ids < v)
    out = np.zeros((ids.size, table.shape[1]))
    out[ok.reshape(-1)] = scale * table[ids[ok]]
    return out, np.abs(out)


def embedding_grad(dout, ids, n_rows, scale, old=None):
    """(grad, terms, magnitude), row by row over the tokens in order"""
    grad = np.zeros((n_rows, dout.shape[1])) if old is None else old.copy()
    mag = np.abs(grad)
    terms = np.full((n_rows, 1), 2.0)  # the scaling and the addition to the old value
    for t, v in enumerate(ids.reshape(-1)):
        if 0 <= v < n_rows:
            grad[v] += scale * dout[t]
            mag[v] += np.abs(scale * dout[t])
            terms[v] += 1
    return grad, terms, mag


def route(experts, n_experts):
    """(order, position, offsets) by a sequential counting sort"""
    e = experts.reshape(-1)
    key = np.where((e >= 0) & (e < n_experts), e, n_experts)
    order = np.argsort(key, kind="stable")
    position = np.empty(key.size, np.int64)
    position[order] = np.arange(key.size)
    offsets = np.searchsorted(key[order], np.arange(n_experts + 1))
    return order, np.where(key < n_experts, position, ~position).reshape(experts.shape), offsets


def dispatch(x, position):
    t, k = position.shape
    rows = np.zeros((t * k, x.shape[1]))
    for i in range(t):
        for j in range(k):
            if position[i, j] >= 0:
                rows[position[i, j]] = x[i]
    return rows


def combine(rows, position, weights):
    """(out, magnitude)"""
    t, k = position.shape
    out = np.zeros((t, rows.shape[1]))
    mag = np.zeros_like(out)
    for i in range(t):
        for j in range(k):
            if 0 <= position[i, j] < len(rows):
                out[i] += weights[i, j] * rows[position[i, j]]
                mag[i] += np.abs(weights[i, j] * rows[position[i, j]])
    return out, mag


def combine_grad(dout, rows, position, weights):
    """(grad_rows, grad_weights, magnitude of the latter)"""
    t, k = position.shape
    gr = np.zeros(rows.shape)
    gw, mag = np.zeros((t, k)), np.zeros((t, k))
    for i in range(t):
        for j in range(k):
            p = position[i, j]
            if p >= 0:
                gr[p] = weights[i, j] * dout[i]
                gw[i, j] = dout[i] @ rows[p]
                mag[i, j] = np.abs(dout[i]) @ np.abs(rows[p])
    return gr, gw, mag
