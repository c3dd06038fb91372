"""One rounding rule in every instance of the selection products: a product or a
fused sum in float32, rounded to nearest even to the 16-bit type written, signs of
zero kept. Every finite float16 value goes through, by whole chunks and by single
elements (widths below 8), and equals torch's float32 product rounded by its cast."""

import pytest
import torch

from helpers import need_gpu
from test_gpu_selection import BF16, F16, F32, by_name, same_bits, sdm

pytestmark = pytest.mark.gpu

WIDTHS = [1, 7, 8, 9, 520]
SCALES = [1.0, -1.0, 0.0, 0.3, -3.7, 1e-3, 1e5, 2.0**-12]


def every_value(dtype, width, dev):
    """All finite values of a 16-bit type, in rows of the width (the last cut off
    and filled with zeros of both signs)."""
    x = torch.arange(65536, device=dev, dtype=torch.int32).to(torch.int16).view(dtype)
    x = x[x.isfinite()]
    tail = -x.numel() % width
    fill = torch.tensor([0.0, -0.0], device=dev).to(dtype).repeat(tail // 2 + 1)[:tail]
    return torch.cat([x, fill]).reshape(-1, width)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype", [F16, BF16], ids=by_name)
def test_lookup(dtype, width):
    dev = need_gpu()
    x = every_value(dtype, width, dev)
    ids = torch.arange(len(x), device=dev)
    many = ids.repeat(1 + (1 << 20) * 8 // x.numel() * (8 if width < 8 else 1))[:2_200_000]
    for scale in SCALES:
        want = (x.float() * torch.tensor(scale, device=dev)).to(dtype)
        assert same_bits(sdm().embedding(x, ids, scale), want), scale
        assert same_bits(sdm().embedding(x, many, scale), want[many]), scale


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype", [F16, BF16], ids=by_name)
def test_combine_and_its_gradient(dtype, width):
    dev = need_gpu()
    x = every_value(dtype, width, dev)
    t = len(x)
    pos = torch.arange(t - 1, -1, -1, device=dev, dtype=torch.int32)[:, None].contiguous()
    zero = torch.zeros((), device=dev)
    for scale in SCALES:
        w = torch.full((t, 1), scale, device=dev)
        want = x.float() * w
        grad_rows, _ = sdm().combine_grad(x, torch.ones_like(x), pos, w)
        assert same_bits(grad_rows.flip(0), want.to(dtype)), scale
        # a sum from +0 on: fma(w, y, 0) is the product, but for a zero's sign
        assert same_bits(sdm().combine(x.flip(0), pos, w), (want + zero).to(dtype)), scale


@pytest.mark.parametrize("gtype", [F16, F32], ids=by_name)
@pytest.mark.parametrize("width", WIDTHS)
def test_gradient(width, gtype):
    """One token a row, and a run over many segments whose other tokens are zeros:
    the sum is the one token's value, scaled."""
    dev = need_gpu()
    x = every_value(F16, width, dev)
    n = len(x)
    ids = torch.randperm(n, device=dev)
    zero = torch.zeros((), device=dev)
    run = torch.zeros((700, width), dtype=F16, device=dev)
    for scale in SCALES:
        want = ((x.float() + zero) * torch.tensor(scale, device=dev)).to(gtype)
        got = sdm().embedding_grad(x, ids, n, scale, dtype=gtype)
        assert same_bits(got[ids], want), scale
        for r in range(0, n, n // 5 + 1):
            run[345] = x[r]
            got = sdm().embedding_grad(run, torch.zeros(700, dtype=torch.int64, device=dev), 2, scale,
                                       dtype=gtype)
            assert same_bits(got[0], want[r]), (scale, r)


@pytest.mark.parametrize("width", WIDTHS)
def test_accumulated_gradient(width):
    """fma(sum, scale, old) in float32, then one rounding to float16. Values of
    2^-4 to 2^4 and scales of 24 bits: exact in float64 (lowest bit 2^-14 * 2^-25,
    highest 2^9), whose cast to float32 is the fused operation's rounding."""
    dev = need_gpu()
    x = every_value(F16, width, dev)
    x = torch.where((x.abs() >= 2.0**-4) & (x.abs() < 16), x, torch.ones((), dtype=F16, device=dev))
    n = len(x)
    old = x.reshape(-1)[torch.randperm(x.numel(), device=dev)].reshape(n, width)
    ids = torch.randperm(n, device=dev)
    for scale in (0.3, -3.7, 1.0):
        s = torch.tensor(scale, device=dev)
        want = (x.double() * s.double() + old[ids].double()).float().half()
        out = old.clone()
        sdm().embedding_grad(x, ids, n, scale, out=out, accumulate=True)
        assert same_bits(out[ids], want), scale
