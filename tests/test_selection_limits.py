"""The limits of the embedding's gradient as the header states them: up to 2^30
tokens and dout up to 2^40 bytes, whatever the width. The sizes are checked on
the host; one call past 2^24 pieces of work runs on the GPU."""

import ctypes

import pytest
import torch

import sparse_dense_matmul_amd as sdm
from helpers import need_gpu

UNSUPPORTED = 6
BYTES = {0: 4, 1: 8, 2: 2, 3: 2}


@pytest.mark.parametrize("elt", [0, 1, 2, 3])
def test_the_documented_limits_are_the_ones_checked(elt):
    """Rows of whole slices (64 chunks of 16 bytes), one element more and less,
    and rows narrower than a chunk: the longest list within the limits is served
    and one token more is not."""
    size, n = sdm.lib.vspmm_embed_grad_workspace_size, ctypes.c_size_t()
    per = 1024 // BYTES[elt]  # elements of a whole slice
    for width in (1, 3, 8, per - 1, per, per + 1, 2 * per + 1, 65 * per - 1, 65 * per + 7,
                  1_000_003, 2**24):
        most = min(2**30, 2**40 // (width * BYTES[elt]))
        assert size(elt, 100, width, most, ctypes.byref(n)) == 0, width
        assert size(elt, 100, width, most + 1, ctypes.byref(n)) == UNSUPPORTED, width


@pytest.mark.gpu
def test_more_than_2_24_pieces():
    """16,773,120 tokens of 16,388 float32, the longest list at this width: 262,080
    segments of 65 slices, more than 2^24 pieces, of a broadcast row. Counts stay
    below 2^24: exact."""
    dev = need_gpu()
    w, v = 64 * 64 * 4 + 4, 97
    n = 2**40 // (w * 4)
    assert -(-n // 64) * 65 > 2**24
    ids = torch.arange(n, device=dev, dtype=torch.int32) % (v + 1)  # v is outside
    row = (torch.arange(w, device=dev) % 5 - 2).float()
    grad = sdm.embedding_grad(row[None].expand(n, w), ids, v)
    count = torch.bincount(ids, minlength=v + 1)[:v].float()
    assert float(count.max()) * 2 < 2**24
    assert torch.equal(grad, count[:, None] * row[None])
