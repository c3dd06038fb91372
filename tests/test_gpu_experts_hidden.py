"""The experts' hidden values keep float32's 24 bits between the layer's two
products: results that are differences of hidden values far larger than
themselves, on data whose float32 sums are exact."""

import numpy as np
import pytest
import torch

import mx4_ref as R
from helpers import need_gpu
from test_gpu_mx4 import host, packed, typed, up

pytestmark = pytest.mark.gpu

WIDTH = 70
CASES = [
    # tokens, top_k, experts, hidden
    (1, 1, 1, 40),
    (1, 8, 16, 256),
    (5, 2, 6, 96),
    (6, 1, 3, 3000),   # hidden values too many to be staged
    (16, 4, 9, 600),
    (16, 6, 12, 130),  # more choices than a wave has lanes
    (40, 2, 5, 200),
    (130, 2, 4, 700),
]


def tokens_of(rng, n, kind, dev):
    """gate's column 0 gives 128; up's columns 1, 34 and 66 (a block each) hold 2^19, multiples of 2^10 and units."""
    x = np.zeros((n, WIDTH))
    x[:, [0, 66]] = 1
    x[:, [1, 34]] = 1024
    return typed(x, kind, dev)[0]


def matrix(v, kind, weights, dev):
    if weights != "mx4":
        t, tv = typed(v, kind, dev)
        assert (tv == v).all()
        return t
    n, r, k = v.shape
    c, s = R.quantize(v.reshape(-1, k))
    assert (R.unpack(c, s, k) == v.reshape(-1, k)).all()
    return packed(c.reshape(n, r, -1), s.reshape(n, r, -1), k, dev)


def choices(rng, tokens, top_k, experts):
    return np.stack([rng.permutation(max(experts, top_k))[:top_k] for _ in range(tokens)])


@pytest.mark.parametrize("activation", ["silu", "gelu"])
@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("kind,weights", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "mx4"), ("f16", "mx4")])
def test_hidden_values_that_cancel(kind, weights, case, activation):
    """Units of 128 (2^19 + 2^10 + d), d of 0 to 3, 27 bits over the last of d; a column adds one and subtracts another.
    Both activations give 128 for 128, and every sum is a multiple of 64 of at most 2^29.1."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    tokens, top_k, experts, hidden = case
    rng = np.random.default_rng([*case, len(weights)])
    d = rng.integers(0, 4, (experts, hidden)).astype(float)
    gate, upm = np.zeros((2, experts, hidden, WIDTH))
    gate[..., 0], upm[..., 1], upm[..., 34], upm[..., 66] = 128, 512, 1, d
    down = np.zeros((experts, WIDTH, hidden))
    at = np.stack([rng.permutation(hidden)[:2] for _ in range(experts * WIDTH)]).reshape(experts, WIDTH, 2)
    i, c = np.ogrid[:experts, :WIDTH]
    down[i, c, at[..., 0]], down[i, c, at[..., 1]] = 1, -1
    e = choices(rng, tokens, top_k, experts)
    w = rng.choice([0.5, 1.0], (tokens, top_k))
    want = np.zeros((tokens, WIDTH))
    for t in range(tokens):
        for k in range(top_k):
            if e[t, k] < experts:
                p = at[e[t, k]]
                want[t] += 128 * w[t, k] * (d[e[t, k]][p[:, 0]] - d[e[t, k]][p[:, 1]])
    got = sdm.expert_mlp(tokens_of(rng, tokens, kind, dev), up(e, dev), up(w.astype(np.float32), dev),
                         *(matrix(m, kind, weights, dev) for m in (gate, upm, down)), activation=activation)
    np.testing.assert_array_equal(host(got), torch.from_numpy(want).to(got.dtype).double().numpy())


@pytest.mark.parametrize("case", CASES, ids=str)
def test_weights_of_eleven_bits_times_hidden_values(case):
    """float16 weights 1 + 7 * 2^-10 times 128 (2^19 + 2^11), less 128 times the same and d: every product of both sides'
    parts counts, and all sums are exact."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    tokens, top_k, experts, hidden = case
    rng = np.random.default_rng([*case, 5])
    first = rng.permutation(hidden)[:hidden // 2]
    second = np.setdiff1d(np.arange(hidden), first)
    d = rng.integers(0, 7, (experts, hidden)).astype(float)
    gate, upm = np.zeros((2, experts, hidden, WIDTH))
    gate[..., 0], upm[..., 1] = 128, 512
    upm[:, first, 34] = 2
    upm[:, second, 34], upm[:, second, 66] = 5.5, 14 + d[:, second]
    down = np.zeros((experts, WIDTH, hidden))
    a, b = rng.choice(first, (experts, WIDTH)), rng.choice(second, (experts, WIDTH))
    i, c = np.ogrid[:experts, :WIDTH]
    down[i, c, a], down[i, c, b] = 1 + 7 * 2.0 ** -10, -1
    e = choices(rng, tokens, top_k, experts)
    want = np.zeros((tokens, WIDTH))
    for t in range(tokens):
        for k in range(top_k):
            if e[t, k] < experts:
                want[t] -= 128 * d[e[t, k], b[e[t, k]]]
    got = sdm.expert_mlp(tokens_of(rng, tokens, "f16", dev), up(e, dev),
                         torch.ones(tokens, top_k, device=dev),
                         *(matrix(m, "f16", "f16", dev) for m in (gate, upm, down)))
    np.testing.assert_array_equal(host(got), want)
