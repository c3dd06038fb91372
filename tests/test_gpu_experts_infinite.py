"""Infinite values in the experts' second product: one weight, one 4-bit value past
float32's, or a hidden value. What the definition makes infinite is infinite, with
its sign, NaN where infinities meet zeros or each other, and no other result
changes."""

import numpy as np
import pytest
import torch

import mx4_ref as R
from helpers import need_gpu
from test_gpu_experts_hidden import CASES, choices
from test_gpu_mx4 import host, packed, rounded, typed, up

pytestmark = pytest.mark.gpu

WIDTH = 40


def layer(rng, kind, weights, tokens, top_k, experts, hidden, dev):
    """Hidden values 128 s, s a whole number of -3 .. 3, and down's of -3 .. 3."""
    x = np.zeros((tokens, WIDTH))
    x[:, [0, 33]] = 1
    gate, upm = np.zeros((2, experts, hidden, WIDTH))
    s = rng.integers(-3, 4, (experts, hidden)).astype(float)
    gate[..., 0], upm[..., 33] = 128, s
    down = rng.integers(-3, 4, (experts, WIDTH, hidden)).astype(float)
    e = choices(rng, tokens, top_k, experts)
    mats = []
    for m in (gate, upm, down):
        if weights == "mx4":
            c, b = R.quantize(m.reshape(-1, m.shape[2]))
            mats.append(packed(c.reshape(*m.shape[:2], -1), b.reshape(*m.shape[:2], -1), m.shape[2], dev))
        else:
            mats.append(typed(m, kind, dev)[0])
    return typed(x, kind, dev)[0], e, 128 * s, down, mats


def spoil(rng, weights, h, down, mats):
    """Infinities in a third of the columns, one or two a column and expert; in 4 bits a value 4 or 6 over 2^126 with zeros
    around. In three of four such columns they agree on the result's sign, in the others they may meet zeros and each other."""
    n, width, hidden = down.shape
    sign = np.where(rng.random(width) < 0.5, -1, 1)
    for e in range(n):
        for c in range(0, width, 3):
            agree = c % 4 != 0
            for f in rng.permutation(np.flatnonzero(h[e]) if agree else hidden)[:1 + c % 2]:
                v = np.inf * (sign[c] * np.sign(h[e, f]) if agree else rng.choice([-1, 1]))
                if weights != "mx4":
                    down[e, c, f] = v
                    mats[2][e, c, f] = float(v)
                    continue
                b = f // 32
                down[e, c, 32 * b:32 * b + 32] = 0
                down[e, c, f] = v
                code = (6 if rng.random() < 0.5 else 7) | (8 if v < 0 else 0)
                mats[2].codes[e, c, 16 * b:16 * b + 16] = 0
                mats[2].codes[e, c, f // 2] = code << (4 * (f & 1))
                mats[2].scales[e, c, b] = 253


def layer_of(e, w, h, down):
    """The result where each token's hidden values are float32 of w h, w the float32 sum of its weights of an expert."""
    out = np.zeros((len(e), down.shape[1]))
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(len(e)):
            for i in set(e[t][e[t] < len(down)].tolist()):
                v = (w[t][e[t] == i].sum(dtype=np.float32) * h[i].astype(np.float32)).astype(np.float64)
                out[t] += (down[i] * v).sum(1)
    return out


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("kind,weights", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "mx4"), ("f16", "mx4")])
def test_infinite_weights(kind, weights, case):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    tokens, top_k, experts, hidden = case
    rng = np.random.default_rng([*case, len(weights), 2])
    x, e, h, down, mats = layer(rng, kind, weights, tokens, top_k, experts, hidden, dev)
    spoil(rng, weights, h, down, mats)
    got = sdm.expert_mlp(x, up(e, dev), torch.ones(tokens, top_k, device=dev), *mats)
    want = layer_of(e, np.ones((tokens, top_k), np.float32), h, down)
    # some infinities of either kind, some not
    assert np.isinf(want).any() and np.isfinite(want).any()
    np.testing.assert_array_equal(host(got), rounded(want, kind))


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("kind,weights", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "mx4"), ("f16", "mx4")])
def test_infinite_hidden_values(kind, weights, case):
    """A router's weight that takes one hidden value (the others are zero) past float32's."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    tokens, top_k, experts, hidden = case
    rng = np.random.default_rng([*case, len(weights), 3])
    x, e, h, down, mats = layer(rng, kind, weights, tokens, top_k, experts, hidden, dev)
    only = rng.integers(0, hidden, experts)
    for i in range(experts):
        h[i] = 0
        h[i, only[i]] = 128
        down[i, :, only[i]] = rng.integers(1, 4, WIDTH) * np.where(rng.random(WIDTH) < 0.5, -1, 1)
    sign = np.where(rng.random(WIDTH) < 0.5, -1, 1)  # a column's infinities agree
    down[:] = np.abs(down) * sign[:, None]
    upm = np.zeros((experts, hidden, WIDTH))
    upm[..., 33] = h / 128
    for at, m in ((1, upm), (2, down)):
        if weights == "mx4":
            c, b = R.quantize(m.reshape(-1, m.shape[2]))
            mats[at] = packed(c.reshape(*m.shape[:2], -1), b.reshape(*m.shape[:2], -1), m.shape[2], dev)
        else:
            mats[at] = typed(m, kind, dev)[0]
    w = np.where(rng.random((tokens, top_k)) < 0.5, 3e38, 1).astype(np.float32)
    w[0, 0] = 3e38
    e[0, 0] = 0
    got = sdm.expert_mlp(x, up(e, dev), up(w, dev), *mats)
    want = layer_of(e, w, h, down)
    np.testing.assert_array_equal(host(got), rounded(want, kind))
