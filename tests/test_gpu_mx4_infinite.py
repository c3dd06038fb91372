"""Products of dense tokens with 4-bit values past float32's (scales 2^126 and
2^127, values 4 and 6): they count as infinite, and the result is what float32
products with an infinity give, whichever route the sizes and scales choose."""

import numpy as np
import pytest
import torch

import mx4_ref as R
from helpers import need_gpu
from test_gpu_mx4 import TYPES, host, packed, rounded, small_matrix, typed

pytestmark = pytest.mark.gpu


def spoiled(rng, n, width, every):
    """A small matrix with one infinite value in a block of zeros in every so many rows; where each lies."""
    codes, scales = small_matrix(rng, n, width)
    rows = np.arange(rng.integers(0, every), n, every)
    cols = rng.integers(0, width, len(rows))
    for r, c in zip(rows, cols):
        b = c // 32
        codes[r, 16 * b:16 * b + 16] = 0
        codes[r, c // 2] = (rng.choice([6, 7]) | rng.choice([0, 8])) << (4 * (c & 1))
        scales[r, b] = rng.choice([253, 254])
    v = R.unpack(codes, scales, width)
    return codes, scales, np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)


def product(x, w):
    """x times w's transpose in 64 bits, sums with infinities by IEEE's rules."""
    whole = x @ np.where(np.isinf(w), 0, w).T
    with np.errstate(invalid="ignore"):
        for n, k in zip(*np.nonzero(np.isinf(w))):
            whole[:, n] += x[:, k] * w[n, k]
    return whole


@pytest.mark.parametrize("m", [1, 7, 20, 50, 64, 70, 130, 300, 1100])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_values_past_float32(kind, m):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, 3])
    for n, width in ((60, 40), (90, 200), (200, 1030), (2200, 130)):
        codes, scales, wv = spoiled(rng, n, width, 5)
        w = packed(codes, scales, width, dev)
        x, xv = typed(rng.integers(-8, 9, (m, width)), kind, dev)
        np.testing.assert_array_equal(host(sdm.matmul_mx4(x, w)), rounded(product(xv, wv), kind))
        g, gv = typed(rng.integers(-8, 9, (m, n)), kind, dev)
        np.testing.assert_array_equal(host(sdm.matmul_mx4_grad(g, w)), rounded(product(gv, wv.T), kind))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_values_past_float32_in_whole_tiles(kind):
    """The same where tiles of 256 are streamed."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(6)
    m, n, width = 4096, 4096, 512
    codes, scales, wv = spoiled(rng, n, width, 64)
    w, inf = packed(codes, scales, width, dev), np.isinf(wv)
    flat = torch.from_numpy(np.where(inf, 0, wv)).to(dev)

    def want(v, at, values):
        for i, k, s in zip(*at, values):
            v[1][:, i] += v[0][:, k] * float(s)
        return v[1].float().to(TYPES[kind])
    g = torch.Generator(device=dev).manual_seed(2)
    x = torch.randint(-8, 9, (m, width), device=dev, generator=g).to(TYPES[kind])
    x[:, 7] = 0  # some infinities times zero
    ref = want((x.double(), x.double() @ flat.t()), np.nonzero(inf), wv[inf])
    assert torch.equal(sdm.matmul_mx4(x, w).nan_to_num(nan=12345.0), ref.nan_to_num(nan=12345.0))
    # the gradient of a matrix of 512 rows of 4,096
    codes, scales, wv = spoiled(rng, width, n, 16)
    w, inf = packed(codes, scales, n, dev), np.isinf(wv)
    flat = torch.from_numpy(np.where(inf, 0, wv)).to(dev)
    at = np.nonzero(inf)
    ref = want((x.double(), x.double() @ flat), at[::-1], wv[inf])
    assert torch.equal(sdm.matmul_mx4_grad(x, w).nan_to_num(nan=12345.0), ref.nan_to_num(nan=12345.0))


@pytest.mark.parametrize("tokens", [1, 6, 16, 40])
def test_experts_first_product(tokens):
    """float16 tokens by gates and ups past float32's: an infinite gate passes on infinite or zero."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([tokens, 8])
    n, hidden, width = 4, 70, 96
    x = np.zeros((tokens, width))
    x[:, [0, 33, 65]] = 1
    # gate 128; up 1, in one unit of each expert infinite; down one unit a column
    gate, upm, down = np.zeros((n, hidden, width)), np.zeros((n, hidden, width)), np.zeros((n, width, hidden))
    gate[..., 0], upm[..., 33] = 128, 1
    unit = rng.integers(0, hidden, (n, width))
    i, c = np.ogrid[:n, :width]
    down[i, c, unit] = 1
    bad = rng.integers(0, hidden, n)
    mats = []
    for m in (gate, upm, down):
        q, b = R.quantize(m.reshape(-1, m.shape[2]))
        mats.append(packed(q.reshape(*m.shape[:2], -1), b.reshape(*m.shape[:2], -1), m.shape[2], dev))
    for e in range(n):
        mats[1].codes[e, bad[e], 16 + 16 + 0] = 6 << 4  # column 65
        mats[1].scales[e, bad[e], 2] = 253
        unit[e, e] = bad[e]
        mats[2].codes[e, e] = 0
        mats[2].codes[e, e, bad[e] // 2] = 2 << (4 * (bad[e] & 1))
        mats[2].scales[e, e] = 127
    ids = rng.integers(0, n, (tokens, 1))
    got = sdm.expert_mlp(torch.from_numpy(x).half().to(dev), torch.from_numpy(ids).to(dev),
                         torch.ones(tokens, 1, device=dev), *mats)
    # a row of down with zeros at an infinite hidden value is NaN, the others infinite
    want = np.where(unit[ids[:, 0]] == bad[ids[:, 0]][:, None], np.inf, np.nan)
    np.testing.assert_array_equal(host(got), want)
