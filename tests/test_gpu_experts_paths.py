"""The experts' layer on each path that its sizes choose: tokens staged or not,
units shared by one to eight waves, columns shared by several blocks, and lists."""

import numpy as np
import pytest
import torch

from helpers import need_gpu
from test_gpu_experts import check, layer
from test_gpu_mx4 import up

pytestmark = pytest.mark.gpu

CASES = [
    # tokens, top_k, experts, width, hidden, drop
    (16, 4, 6, 1600, 64, 0.0),     # few choices, tokens too wide to be staged
    (16, 4, 5, 2100, 50, 0.1),
    (3, 2, 5, 128, 130, 0.0),      # a wave to a run of units
    (3, 2, 5, 600, 70, 0.0),       # two
    (2, 3, 6, 1100, 90, 0.0),      # four
    (1, 3, 4, 2050, 33, 0.0),      # eight
    (16, 4, 9, 70, 600, 0.0),      # hidden values too many to be staged, columns shared by blocks
    (2, 8, 16, 48, 2100, 0.0),
    (16, 6, 12, 600, 300, 0.2),    # more choices than a wave has lanes
    (15, 8, 11, 2100, 260, 0.0),
    (40, 4, 12, 300, 700, 0.0),    # several tiles, columns shared by blocks
    (130, 3, 10, 100, 600, 0.1),   # two groups of tokens
    (48, 1, 1, 130, 90, 0.0),      # three tiles of one expert
    (40, 8, 260, 40, 1100, 0.0),   # several runs of units a block
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("kind,weights", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "mx4"), ("f16", "mx4")])
def test_paths(kind, weights, case):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    tokens, top_k, experts, width, hidden, drop = case
    rng = np.random.default_rng([*case[:5], len(weights), 1])
    x, xv, e, wt, mats, vals = layer(rng, kind, weights, tokens, top_k, experts, width, hidden, dev, drop)
    ids, w = up(e, dev), up(wt, dev)
    need = sdm.expert_mlp_workspace(tokens, top_k, experts, width, hidden)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=dev)
    got = sdm.expert_mlp(x, ids, w, *mats, workspace=ws[:need])
    check(got, xv, e, wt, vals, kind)
    assert (ws[need:] == 255).all()
    # again over what the first call left, and in memory of its own: the same bits
    assert torch.equal(sdm.expert_mlp(x, ids, w, *mats, workspace=ws[:need]), got)
    assert torch.equal(sdm.expert_mlp(x, ids, w, *mats), got)


@pytest.mark.parametrize("tokens", [3, 40])
def test_replays_with_columns_shared_by_blocks(tokens):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(tokens)
    x, xv, e, wt, mats, vals = layer(rng, "bf16", "bf16", tokens, 4, 12, 300, 700, dev)
    ids, w = up(e, dev), up(wt, dev)
    sdm.expert_mlp(x, ids, w, *mats)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sdm.expert_mlp(x, ids, w, *mats)
    for i in range(4):
        x.copy_(torch.randn(x.shape, device=dev))
        w.copy_(torch.rand(w.shape, device=dev))
        graph.replay()
        want = sdm.expert_mlp(x, ids, w, *mats)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_two_streams_at_once():
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(8)
    x, xv, e, wt, mats, vals = layer(rng, "f16", "f16", 20, 4, 12, 300, 700, dev)
    ids, w = up(e, dev), up(wt, dev)
    want = sdm.expert_mlp(x, ids, w, *mats)
    check(want, xv, e, wt, vals, "f16")
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(12):
        with torch.cuda.stream(streams[i % 2]):
            got.append(sdm.expert_mlp(x, ids, w, *mats))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
