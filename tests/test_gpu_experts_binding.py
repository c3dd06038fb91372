"""The binding of the experts' layer: its refusals of things that are no matrices."""

import numpy as np
import pytest
import torch

from helpers import need_gpu

pytestmark = pytest.mark.gpu


def arguments(dev):
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    return dict(x=b(4, 16), experts=torch.zeros(4, 2, dtype=torch.int64, device=dev), weights=torch.zeros(4, 2, device=dev),
                gate=b(3, 32, 16), up=b(3, 32, 16), down=b(3, 16, 32))


@pytest.mark.parametrize("name", ["gate", "up", "down"])
def test_matrices_that_are_none(name):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    ok = arguments(dev)
    for bad in (None, [1.0], np.zeros((3, 32, 16)), sdm.Mx4(None, None, 16)):
        with pytest.raises(TypeError):
            sdm.expert_mlp(**{**ok, name: bad})
