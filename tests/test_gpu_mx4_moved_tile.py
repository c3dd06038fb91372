"""The last tile of a streamed product is moved to end with the matrix. Which
route a column of a float16 product takes depends on the scales of its own tile of
256 rows, whatever those of the rows that the moved tile shares with the one
before it: on ordinary values the routes differ in their last bits."""

import pytest
import torch

import mx4_ref as R
from helpers import need_gpu

pytestmark = pytest.mark.gpu

M, N, WIDTH = 3900, 4000, 1024
OWN = N // 256 * 256  # the first row of the last tile, which starts at N - 256


@pytest.mark.parametrize("row", [OWN + 3, N - 1, N - 200, OWN - 1, OWN - 256, N - 257])
@pytest.mark.parametrize("scale", [127 - 60, 127 + 20, 127 - 100, 255])
def test_columns_of_the_tile_before(row, scale):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    g = torch.Generator(device=dev).manual_seed(row)
    x = torch.randn(M, WIDTH, device=dev, generator=g).half()
    x[1, 5], x[2, 9] = float("inf"), float("nan")
    near = sdm.quantize_mx4(torch.randn(N, WIDTH, device=dev, generator=g) / 32)
    far = near._replace(scales=near.scales.clone())
    far.scales[row, 7] = scale

    def product(w):
        return sdm.matmul_mx4(x, w).view(torch.int16)
    a, b = product(near), product(far)
    for _ in range(3):
        assert torch.equal(product(far), b)
    # every tile but the one that owns the row as if nothing had happened
    own = slice(row // 256 * 256, min(row // 256 * 256 + 256, N))
    same = torch.ones(N, dtype=torch.bool, device=dev)
    same[own] = False
    assert torch.equal(a[:, same], b[:, same])
    # that one by the other route in all of its columns: as where the matrix ends with it, or near the exact result
    if own.stop <= OWN:
        part = product(sdm.Mx4(far.codes[:OWN], far.scales[:OWN], WIDTH))
        assert torch.equal(part[:, own], b[:, own])
    wv = sdm.dequantize_mx4(sdm.Mx4(far.codes[own], far.scales[own], WIDTH), torch.float32).double()
    ok = ~wv.isnan().any(1)
    ref, size = x[3:].double() @ wv[ok].t(), x[3:].double().abs() @ wv[ok].abs().t()
    got = b.view(torch.float16)[3:, own][:, ok].double()
    bound = torch.from_numpy(R.product_bound(ref.cpu().numpy(), size.cpu().numpy(), WIDTH, "f16")).to(dev)
    near_enough = (got - ref).abs() <= bound
    assert (near_enough | (ref.abs() > 65000)).all()
