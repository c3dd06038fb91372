"""Streamed products of rows at every stride that they are taken for: 16 bytes more
than the row and up, not a number in the gaps."""

import numpy as np
import pytest
import torch

import mx4_ref as R
from helpers import need_gpu
from test_gpu_mx4 import TYPES, small_matrix, up

pytestmark = pytest.mark.gpu

M, N, K = 4096, 4096, 256


def apart(t, gap, fill):
    big = torch.full((t.shape[0], t.shape[1] + gap), fill, dtype=t.dtype, device=t.device)[:, :t.shape[1]]
    big.copy_(t)
    return big


def matrix(rng, n, width, gap, dev, low=-2, high=2):
    import sparse_dense_matmul_amd as sdm
    codes, scales = small_matrix(rng, n, width, low, high)
    w = sdm.Mx4(apart(up(codes, dev), 16 * gap, 0x77), apart(up(scales, dev), 4 * gap, 255), width)
    return w, torch.from_numpy(R.unpack(codes, scales, width)).to(dev)


@pytest.mark.parametrize("gap", [0, 1, 2, 3, 4, 5, 7])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_dense_rows(kind, gap):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(gap)
    g = torch.Generator(device=dev).manual_seed(gap)
    for n, width, k, product in ((N, K, K, sdm.matmul_mx4), (K, N, K, sdm.matmul_mx4_grad)):
        w, wv = matrix(rng, n, width, gap, dev)
        x = apart(torch.randint(-8, 9, (M, k), device=dev, generator=g).to(TYPES[kind]), 8 * gap, float("nan"))
        ref = x.double() @ (wv.t() if product is sdm.matmul_mx4 else wv)
        assert torch.equal(product(x, w), ref.float().to(TYPES[kind])), product


@pytest.mark.parametrize("gap", [0, 1, 2, 3, 4, 5, 7])
def test_both_sides(gap):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(gap)
    x, xv = matrix(rng, M, K, gap, dev, -1, 1)
    w, wv = matrix(rng, N, K, gap, dev, -1, 1)
    assert torch.equal(sdm.matmul_mx4(x, w, dtype=torch.float32), (xv @ wv.t()).float())
