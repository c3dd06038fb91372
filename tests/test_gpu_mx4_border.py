"""Dense tokens by 4-bit rows on either side of the border between the kernel for
few tokens and tiles, on data whose float32 sums are exact."""

import numpy as np
import pytest

from helpers import need_gpu
from test_gpu_mx4 import exact_case, rounded, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m,n", [(32, 9000), (33, 4095), (64, 4096), (33, 4097), (64, 4100), (65, 4096), (40, 9000)])
@pytest.mark.parametrize("width", [31, 100, 257])
def test_either_side(kind, m, n, width):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, n, width])
    x, xv, w, wv = exact_case(rng, m, n, width, kind, dev)
    same(sdm.matmul_mx4(x, w), rounded(xv @ wv.T, kind))
