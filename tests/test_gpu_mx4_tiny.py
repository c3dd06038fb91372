"""4-bit values far under float16's, down to 2^-128, with float16 tokens: none is
lost where something later scales it up, or where an infinity meets it. Blocks of
zeros stay zeros."""

import numpy as np
import pytest
import torch

import mx4_ref as R
from helpers import need_gpu
from test_gpu_mx4 import TYPES, host, packed, rounded, small_matrix, typed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("width", [70, 256, 400])
@pytest.mark.parametrize("tokens,top_k", [(1, 1), (6, 2), (16, 6), (40, 2)])
def test_experts_first_product(tokens, top_k, width, kind):
    """gate 2^-91 to 6 * 2^-90, whose activation is half of it; up 0.5 to 6; down one unit of 2^96 a column: the layer's
    result is a product of three exact values."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([tokens, width])
    n, hidden = 5, 90
    col = rng.integers(0, width, 2)  # one token column for both; another where all is zero
    x = np.zeros((tokens, width))
    x[:, col[0]] = 1
    mats = []
    a, b = (rng.integers(1, 8, (n, hidden)) for _ in range(2))
    for code, scale in ((a, 127 - 90), (b, 127)):
        c = np.zeros((n, hidden, 16 * R.blocks(width)), np.uint8)
        s = np.zeros((n, hidden, R.blocks(width)), np.uint8)
        c[..., col[0] // 2] = code << (4 * (col[0] & 1))
        s[..., col[0] // 32] = scale
        mats.append(packed(c, s, width, dev))
    unit = rng.integers(0, hidden, (n, width))
    down = np.zeros((n, width, hidden))
    i, c = np.ogrid[:n, :width]
    down[i, c, unit] = 2.0 ** 96
    q, s = R.quantize(down.reshape(-1, hidden))
    mats.append(packed(q.reshape(n, width, -1), s.reshape(n, width, -1), hidden, dev))
    ids = np.stack([rng.permutation(n + 2)[:top_k] for _ in range(tokens)])
    h = R.LEVELS[a] * R.LEVELS[b] * 2.0 ** 5
    want = np.zeros((tokens, width))
    for t in range(tokens):
        for e in ids[t][ids[t] < n]:
            want[t] += h[e, unit[e]]
    got = sdm.expert_mlp(typed(x, kind, dev)[0], torch.from_numpy(ids).to(dev),
                         torch.ones(tokens, top_k, device=dev), *mats)
    np.testing.assert_array_equal(host(got), rounded(want, kind))


def tiny(rng, n, width):
    """A small matrix in which a third of the blocks are at scales of 2^-127 to 2^-87, half of those zeros."""
    codes, scales = small_matrix(rng, n, width)
    far = rng.random(scales.shape) < 0.3
    scales[far] = rng.choice([0, 1, 20, 40], far.sum())
    zero = np.repeat(far & (rng.random(scales.shape) < 0.5), 16, 1)
    codes[zero] &= 0x88
    return codes, scales


def with_infinities(v, w):
    """v times w's transpose, in 64 bits; v's infinities, one a row, by IEEE's rules."""
    inf = np.isinf(v)
    out = np.where(inf, 0, v) @ w.T
    with np.errstate(invalid="ignore"):
        for r, k in zip(*np.nonzero(inf)):
            out[r] += v[r, k] * w[:, k]
    return out


@pytest.mark.parametrize("m", [1, 7, 20, 50, 64, 70, 130, 300, 1100])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_infinite_tokens_by_tiny_values(kind, m):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, 4])
    for n, width in ((60, 40), (90, 200), (200, 1030), (2200, 130)):
        codes, scales = tiny(rng, n, width)
        w, wv = packed(codes, scales, width, dev), R.unpack(codes, scales, width)
        for grad in (False, True):
            k = n if grad else width
            v = rng.integers(-8, 9, (m, k)).astype(float)
            v[np.arange(m), rng.integers(0, k, m)] = np.where(rng.random(m) < 0.5, np.inf, -np.inf)
            x, xv = typed(v, kind, dev)
            got = (sdm.matmul_mx4_grad if grad else sdm.matmul_mx4)(x, w)
            np.testing.assert_array_equal(host(got), rounded(with_infinities(xv, wv.T if grad else wv), kind))


def test_infinite_tokens_by_tiny_values_in_whole_tiles():
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(9)
    for n, width, product in ((4096, 512, sdm.matmul_mx4), (512, 4096, sdm.matmul_mx4_grad)):
        m = 4096
        codes, scales = tiny(rng, n, width)
        scales[:, ::3][scales[:, ::3] < 100] = 127  # tiles of either route
        w, wv = packed(codes, scales, width, dev), torch.from_numpy(R.unpack(codes, scales, width)).to(dev)
        if product is sdm.matmul_mx4_grad:
            wv = wv.t()
        g = torch.Generator(device=dev).manual_seed(n)
        x = torch.randint(-8, 9, (m, 512), device=dev, generator=g).to(TYPES["f16"])
        at = torch.randint(0, 512, (m,), device=dev, generator=g)
        rows = torch.arange(m, device=dev)
        x[rows, at] = 0
        ref = x.double() @ wv.t() + float("inf") * wv.t()[at]
        x[rows, at] = float("inf")
        got = product(x, w)
        assert torch.equal(got.nan_to_num(nan=12345.0), ref.float().half().nan_to_num(nan=12345.0))
