"""Results and workspaces that share memory with an operand are refused before
anything is enqueued; views that interleave without sharing an element are
served. The geometry is checked on the host against sets of bytes."""

import numpy as np
import pytest
import torch

import sparse_dense_matmul_amd as sdm
from helpers import need_gpu
from sparse_dense_matmul_amd import selection


def bytes_of(region):
    start, rows, width, ld = region
    return {start + r * ld + i for r in range(rows) for i in range(width)}


def test_overlap_of_strided_rows_against_sets_of_bytes():
    rng = np.random.default_rng(1)
    seen = {True: 0, False: 0}
    for _ in range(20_000):
        regions = []
        for _ in range(2):
            rows, width = int(rng.integers(0, 6)), int(rng.integers(0, 7))
            ld = int(rng.integers(0, 14)) if rows > 1 else 0
            regions.append((int(rng.integers(0, 50)), rows, width, ld))
        if rng.random() < 0.5 and regions[0][1] > 1 and regions[1][1] > 1:
            regions[1] = regions[1][:3] + (regions[0][3],)
        want = bool(bytes_of(regions[0]) & bytes_of(regions[1]))
        seen[want] += 1
        assert selection._overlap(*regions) is want, regions
        assert selection._overlap(*regions[::-1]) is want, regions
    assert min(seen.values()) > 2000


def test_regions_of_tensors():
    t = torch.zeros(10, 12, dtype=torch.bfloat16)
    p = t.data_ptr()
    assert selection._region(t, 12) == (p, 10, 24, 24)
    assert selection._region(t[2:5, 3:8], 12) == (p + 54, 3, 10, 24)
    assert selection._region(t[:1].expand(6, 12), 0) == (p, 6, 24, 0)
    assert selection._region(t) == (p, 1, 240, 0)


@pytest.mark.gpu
def test_results_on_operands_are_refused():
    dev = need_gpu()
    S = sdm
    x = torch.ones((6, 8), device=dev)
    ids = torch.tensor([5, 4, 3, 2, 1, 0], device=dev)
    pos = torch.arange(6, dtype=torch.int32, device=dev)[:, None].contiguous()
    w = torch.full((6, 1), 2.0, device=dev)
    other = torch.ones((6, 8), device=dev)
    big = torch.ones((12, 8), device=dev)
    own_ids = torch.zeros(12, dtype=torch.int64, device=dev)
    ids_as_rows = own_ids.view(torch.float32).reshape(6, 4)
    ws = torch.zeros(S.embedding_grad_workspace(9, 8, 6, torch.float32) + 4096, dtype=torch.uint8,
                     device=dev)
    ws_as_rows = ws[256:256 + 192].view(torch.float32).reshape(6, 8)
    calls = [
        lambda: S.embedding(x, ids, out=x),
        lambda: S.embedding(big[:6], ids, out=big[5:11]),
        lambda: S.embedding(torch.ones((9, 4), device=dev), own_ids[:6], out=ids_as_rows),
        lambda: S.embedding_grad(x, ids, 6, out=x),
        lambda: S.embedding_grad(x, ids, 6, out=x, accumulate=True),
        lambda: S.embedding_grad(ws_as_rows, ids, 9, workspace=ws),
        lambda: S.embedding_grad(x, ids, 6, out=ws_as_rows, workspace=ws),
        lambda: S.embedding_grad(x, ws[:48].view(torch.int64), 9, workspace=ws),
        lambda: S.dispatch(x, pos, out=x),
        lambda: S.combine(x, pos, w, out=x),
        lambda: S.combine(other, pos, big.reshape(-1)[:6].reshape(6, 1), out=big[:6]),
        lambda: S.dispatch_grad(x, pos, out=x),
        lambda: S.combine_grad(x, other, pos, w, out=x),
        lambda: S.combine_grad(other, x, pos, w, out=x),
    ]
    for i, fn in enumerate(calls):
        with pytest.raises(ValueError, match="overlap"):
            fn()
    torch.cuda.synchronize()
    for t in (x, other, big):
        assert (t == 1).all()  # nothing was enqueued
    experts = torch.zeros((4096, 2), dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="overlap"):
        S.route(experts, 500, workspace=experts)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [3, 16, 37])
def test_interleaved_views_are_served(width):
    """Operand and result side by side in the rows of one buffer."""
    dev = need_gpu()
    rng = np.random.default_rng(width)
    buf = torch.from_numpy(rng.integers(-4, 5, (60, 2 * width + 1))).to(dev).float()
    left, right = buf[:, :width], buf[:, width:2 * width]
    ids = torch.from_numpy(rng.integers(-1, 60, 60)).to(dev)
    pos = torch.from_numpy(rng.permutation(60).astype(np.int32)).to(dev)[:, None]
    w = torch.from_numpy(rng.integers(-3, 4, (60, 1))).to(dev).float()
    ws = torch.empty(sdm.embedding_grad_workspace(60, width, 60, torch.float32), dtype=torch.uint8,
                     device=dev)
    for fn in (lambda a, o: sdm.embedding(a, ids, 2.0, out=o),
               lambda a, o: sdm.embedding_grad(a, ids, 60, out=o, workspace=ws),
               lambda a, o: sdm.dispatch(a, pos, out=o),
               lambda a, o: sdm.combine(a, pos, w, out=o),
               lambda a, o: sdm.dispatch_grad(a, pos, out=o),
               lambda a, o: sdm.combine_grad(a, a, pos, w, out=o)[0]):
        want = fn(left, None)
        before = left.clone()
        got = fn(left, right)
        assert got.data_ptr() == right.data_ptr() and torch.equal(right, want.reshape(60, width))
        assert torch.equal(left, before)
