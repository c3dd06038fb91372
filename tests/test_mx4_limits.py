"""The documented limits of the 4-bit products: sizes past one launch are refused
by the host or split over launches."""

import ctypes

import pytest
import torch

import sparse_dense_matmul_amd as sdm
from helpers import need_gpu
from test_mx4_refusals import BF16, D, UNSUPPORTED, caller, mx4

M, N = 2**30, 129  # 2^24 tiles of 128 x 128, of 256 threads each


def test_results_past_one_launch_are_refused():
    w = mx4()
    for name, n, width in (("vspmm_mx4_matmul", N, 8), ("vspmm_mx4_matmul_grad", 8, N)):
        call = caller(getattr(sdm.lib, name), [BF16, M, n, width, D, n if name.endswith("grad") else width,
                                               ctypes.byref(w), D, N, None])
        assert call() == UNSUPPORTED
        assert call(**{"_3" if name.endswith("grad") else "_2": 2**24, "_8": 2**24}) == UNSUPPORTED
    call = caller(sdm.lib.vspmm_mx4_matmul_mx4,
                  [BF16, M, N, 8, ctypes.byref(w), ctypes.byref(w), D, N, None])
    assert call() == UNSUPPORTED and call(_2=2**24, _7=2**24) == UNSUPPORTED


@pytest.mark.gpu
def test_transpose_past_one_launch():
    """2^24 columns of 16,384 equal values: 2^23 blocks of 512 threads, one more than a launch has."""
    dev = need_gpu()
    rows, width = 2**14, 2**24
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info(dev)[0] < 170 * 2**30:
        pytest.skip("needs 160 GB of device memory")
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(1, width, device=dev, generator=g).bfloat16()
    one = sdm.quantize_mx4(x.expand(32, width), transpose=True)
    got = sdm.quantize_mx4(x.expand(rows, width), transpose=True)
    assert got.codes.shape == (width, rows // 2) and got.scales.shape == (width, rows // 32)
    step = 2**19
    for at in range(0, width, step):
        part = slice(at, at + step)
        # sixteen equal bytes a block: as words of eight
        codes = got.codes[part].view(torch.int64)
        assert (codes == one.codes[part].view(torch.int64)[:, :1]).all()
        assert (got.scales[part] == one.scales[part]).all()
    del got, codes
    torch.cuda.empty_cache()
