"""Paths of the 4-bit products that other sizes do not take: streamed tiles whose
last group of codes is half filled or whose steps are odd in number, rows with gaps
behind them, launches past the first, and products of two 4-bit matrices past
float32's range."""

import numpy as np
import pytest
import torch

import mx4_ref as R
from helpers import need_gpu
from test_gpu_mx4 import TYPES, host, packed, small_matrix, up

pytestmark = pytest.mark.gpu


def apart(t, gap, fill):
    """t's rows in a larger array, `gap` elements of `fill` behind each."""
    big = torch.full((t.shape[0], t.shape[1] + gap), fill, dtype=t.dtype, device=t.device)[:, :t.shape[1]]
    big.copy_(t)
    return big


def equal(got, ref, kind):
    want = ref.float().to(TYPES[kind])
    assert torch.equal(got, want), int((got != want).sum())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,width", [(4096, 4096, 128), (4096, 4096, 384), (3700, 3900, 640), (257, 60000, 896),
                                       (50001, 300, 1152)])
def test_half_filled_groups_of_codes(kind, m, n, width):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, n, width])
    codes, scales = small_matrix(rng, n, width)
    wv = torch.from_numpy(R.unpack(codes, scales, width)).to(dev)
    # 16-byte rows of codes and 4-byte rows of scales, not a number behind each
    w = sdm.Mx4(apart(up(codes, dev), 16, 0x77), apart(up(scales, dev), 4, 255), width)
    g = torch.Generator(device=dev).manual_seed(m)
    x = torch.randint(-8, 9, (m, width), device=dev, generator=g).to(TYPES[kind])
    x = apart(x, 8, float("nan"))
    ref = x.double() @ wv.t()
    equal(sdm.matmul_mx4(x, w), ref, kind)
    if kind == "f16":  # by the other route
        scales[5::256, -1] = 127 - 40
        wv = torch.from_numpy(R.unpack(codes, scales, width)).to(dev)
        w = sdm.Mx4(w.codes, apart(up(scales, dev), 4, 255), width)
        equal(sdm.matmul_mx4(x, w), x.double() @ wv.t(), kind)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,width", [(4096, 64, 4096), (4096, 192, 4096), (3700, 576, 3907), (50001, 1088, 300)])
def test_gradient_of_odd_steps(kind, m, n, width):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, n, width, 1])
    codes, scales = small_matrix(rng, n, width)
    wv = torch.from_numpy(R.unpack(codes, scales, width)).to(dev)
    w = sdm.Mx4(apart(up(codes, dev), 3, 0x77), apart(up(scales, dev), 1, 255), width)
    gen = torch.Generator(device=dev).manual_seed(n)
    g = apart(torch.randint(-8, 9, (m, n), device=dev, generator=gen).to(TYPES[kind]), 8, float("nan"))
    equal(sdm.matmul_mx4_grad(g, w), g.double() @ wv, kind)
    if kind == "f16":
        scales[n // 2, 3::8] = 127 - 40
        wv = torch.from_numpy(R.unpack(codes, scales, width)).to(dev)
        w = sdm.Mx4(w.codes, apart(up(scales, dev), 1, 255), width)
        equal(sdm.matmul_mx4_grad(g, w), g.double() @ wv, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,width", [(4096, 4096, 256), (3700, 3900, 768), (257, 60000, 1280)])
def test_both_sides_in_rows_with_gaps(kind, m, n, width):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, n, width, 2])
    sides, values = [], []
    for rows in (m, n):
        codes, scales = small_matrix(rng, rows, width, -1, 1)
        sides.append(sdm.Mx4(apart(up(codes, dev), 16, 0x77), apart(up(scales, dev), 4, 255), width))
        values.append(torch.from_numpy(R.unpack(codes, scales, width)).to(dev))
    equal(sdm.matmul_mx4(*sides, dtype=TYPES[kind]), values[0] @ values[1].t(), kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_quantize_past_one_launch(kind):
    """More than 2^30 lanes of eight values: rows that overlap, each one element further than the one before."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    width = 4099
    per_launch = 2**30 // (4 * 129)
    rows = per_launch + 100_001
    g = torch.Generator(device=dev).manual_seed(3)
    base = torch.randn(rows + width, device=dev, generator=g).to(TYPES[kind])
    x = base.as_strided((rows, width), (1, 1))
    q = sdm.quantize_mx4(x)
    spans = [slice(0, 300), slice(per_launch - 300, per_launch + 300), slice(rows - 300, rows)]
    for s in spans:
        part = sdm.quantize_mx4(x[s])
        assert torch.equal(q.codes[s], part.codes) and torch.equal(q.scales[s], part.scales)
    if kind == "bf16":
        back = sdm.dequantize_mx4(q)
        for s in spans:
            assert torch.equal(back[s], sdm.dequantize_mx4(sdm.Mx4(q.codes[s], q.scales[s], width)))
        del back
    del q, x, base
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m", [4, 64, 300])
@pytest.mark.parametrize("scale", [252, 253, 254])
def test_products_of_two_take_values_past_float32(m, scale):
    """4 times 2^125 to 2^127 by tokens of 2^-100 and 1: the products themselves, infinite only past float32's range."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    n, width = 64, 40
    codes = np.zeros((n, 32), np.uint8)
    codes[:, 0] = 6
    scales = np.full((n, 2), scale, np.uint8)
    tokens = np.zeros((m, 32), np.uint8)
    tokens[:, 0] = 2
    for exponent in (-100, 0):
        got = sdm.matmul_mx4(packed(tokens, np.full((m, 2), 127 + exponent, np.uint8), width, dev),
                             packed(codes, scales, width, dev), dtype=torch.float32)
        want = 4 * 2.0 ** (scale - 127 + exponent)
        want = want if want < 2.0 ** 128 else np.inf
        assert (host(got) == want).all()
