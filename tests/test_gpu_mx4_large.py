"""4-bit products of many tokens, where whole tiles are streamed: bit for bit
against float64 products on the device, on data whose float32 sums are exact."""

import numpy as np
import pytest
import torch

import mx4_ref as R
from helpers import need_gpu
from test_gpu_mx4 import TYPES, packed, small_matrix

pytestmark = pytest.mark.gpu

# rows and columns that tiles of 256 do not divide, widths of one to five copies of scales
SHAPES = [(4096, 4096, 512), (3700, 3900, 1024), (257, 60000, 512), (50001, 300, 1536), (4000, 3841, 2560), (3601, 4100, 256), (4096, 4096, 768),
          (8192, 2048, 1280)]


def values(codes, scales, width, dev):
    return torch.from_numpy(R.unpack(codes, scales, width)).to(dev)


def equal(got, ref, kind):
    want = ref.float().to(TYPES[kind])
    assert torch.equal(got, want), int((got != want).sum())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,width", SHAPES)
def test_matmul(kind, m, n, width):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, n, width])
    codes, scales = small_matrix(rng, n, width)
    w, wv = packed(codes, scales, width, dev), values(codes, scales, width, dev)
    g = torch.Generator(device=dev).manual_seed(m)
    x = torch.randint(-8, 9, (m, width + 8), device=dev, generator=g).to(TYPES[kind])[:, :width]
    base = torch.full((m, n + 3), 9.0, dtype=TYPES[kind], device=dev)
    sdm.matmul_mx4(x, w, out=base[:, 1:n + 1])
    equal(base[:, 1:n + 1], x.double() @ wv.t(), kind)
    assert (base[:, 0] == 9).all() and (base[:, n + 1:] == 9).all()
    if kind == "f16" and n < 5000:  # scales that float16 cannot hold, in one block
        scales[n // 2, width // 64] = 127 - 40
        w, wv = packed(codes, scales, width, dev), values(codes, scales, width, dev)
        equal(sdm.matmul_mx4(x, w), x.double() @ wv.t(), kind)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,width", [(m, w, n) for m, n, w in SHAPES])
def test_matmul_grad(kind, m, n, width):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, n, width, 1])
    codes, scales = small_matrix(rng, n, width)
    w, wv = packed(codes, scales, width, dev), values(codes, scales, width, dev)
    gen = torch.Generator(device=dev).manual_seed(n)
    g = torch.randint(-8, 9, (m, n), device=dev, generator=gen).to(TYPES[kind])
    equal(sdm.matmul_mx4_grad(g, w), g.double() @ wv, kind)
    if kind == "f16" and width < 5000:
        scales[n // 2, width // 64] = 127 - 40
        w, wv = packed(codes, scales, width, dev), values(codes, scales, width, dev)
        equal(sdm.matmul_mx4_grad(g, w), g.double() @ wv, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,width", SHAPES)
def test_matmul_of_two(kind, m, n, width):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, n, width, 2])
    a, sa = small_matrix(rng, m, width, -1, 1)
    b, sb = small_matrix(rng, n, width, -1, 1)
    got = sdm.matmul_mx4(packed(a, sa, width, dev), packed(b, sb, width, dev), dtype=TYPES[kind])
    equal(got, values(a, sa, width, dev) @ values(b, sb, width, dev).t(), kind)


def test_ordinary_values_and_repeats():
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    g = torch.Generator(device=dev).manual_seed(5)
    m, n, width = 3900, 4000, 1024
    w = sdm.quantize_mx4(torch.randn(n, width, device=dev, generator=g) / 32)
    wv = sdm.dequantize_mx4(w, torch.float32).double()
    for kind in ("bf16", "f16"):
        x = torch.randn(m, width, device=dev, generator=g).to(TYPES[kind])
        got = sdm.matmul_mx4(x, w)
        ref, size = x.double() @ wv.t(), x.double().abs() @ wv.abs().t()
        bound = R.product_bound(ref.cpu().numpy(), size.cpu().numpy(), width, kind)
        assert (np.abs((got.double() - ref).cpu().numpy()) <= bound).all()
        assert torch.equal(sdm.matmul_mx4(x, w), got)
        q = sdm.quantize_mx4(x)
        assert torch.equal(sdm.matmul_mx4(q, w), sdm.matmul_mx4(q, w))
