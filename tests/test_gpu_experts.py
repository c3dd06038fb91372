"""The experts' layer on the GPU against numpy in 64 bits, within a bound that
follows each rounding through both products."""

import numpy as np
import pytest
import torch

import mx4_ref as R
from helpers import need_gpu
from test_gpu_mx4 import host, packed, typed, up

pytestmark = pytest.mark.gpu


def layer(rng, kind, weights, tokens, top_k, experts, width, hidden, dev, drop=0.0, ids=np.int64):
    import sparse_dense_matmul_amd as sdm
    x, xv = typed(rng.standard_normal((tokens, width)), kind, dev)
    mats, vals = [], []
    for n, k in ((hidden, width), (hidden, width), (width, hidden)):
        v = rng.standard_normal((experts, n, k)) / np.sqrt(k)
        if weights == "mx4":
            c, s = R.quantize(v.reshape(-1, k).astype(np.float32).astype(np.float64))
            c, s = c.reshape(experts, n, -1), s.reshape(experts, n, -1)
            mats.append(packed(c, s, k, dev))
            vals.append(R.unpack(c, s, k))
        else:
            t, tv = typed(v, kind, dev)
            mats.append(t)
            vals.append(tv)
    e = np.stack([rng.permutation(max(experts, top_k))[:top_k] for _ in range(tokens)]) if tokens else \
        np.zeros((0, top_k))
    e = np.where(rng.random(e.shape) < drop, -1, e).astype(ids)
    wt = rng.random((tokens, top_k)).astype(np.float32)
    assert sdm.expert_mlp
    return x, xv, e, wt, mats, vals


def check(got, xv, e, wt, vals, kind, act=R.silu):
    ref, off = R.expert_mlp(xv, e, wt.astype(np.float64), *vals, act=act)
    bound = R.EPS[kind] * (np.abs(ref) + off) + off + R.LEAST[kind]
    assert (np.abs(host(got) - ref) <= bound).all()


CASES = [
    # tokens, top_k, experts, width, hidden, drop
    (1, 1, 1, 32, 32, 0.0),
    (1, 8, 16, 512, 256, 0.0),
    (1, 2, 300, 130, 70, 0.0),
    (2, 6, 4, 100, 33, 0.2),
    (13, 6, 60, 101, 73, 0.25),
    (16, 4, 8, 257, 129, 0.0),
    (17, 2, 4, 64, 200, 0.0),
    (40, 3, 5, 96, 128, 0.5),
    (64, 8, 32, 128, 64, 0.0),
    (65, 1, 2, 33, 31, 0.0),
    (130, 2, 3, 40, 48, 0.1),
    (200, 1, 1, 16, 24, 0.0),
    (7, 3, 9, 1, 5, 0.0),
    (7, 3, 9, 5, 1, 0.0),
    (3, 5, 7, 1100, 1030, 0.9),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("kind,weights", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "mx4"), ("f16", "mx4")])
def test_layer(kind, weights, case):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    tokens, top_k, experts, width, hidden, drop = case
    rng = np.random.default_rng([*case[:5], len(weights)])
    x, xv, e, wt, mats, vals = layer(rng, kind, weights, tokens, top_k, experts, width, hidden, dev, drop,
                                     np.int32 if tokens % 2 else np.int64)
    check(sdm.expert_mlp(x, up(e, dev), up(wt, dev), *mats), xv, e, wt, vals, kind)


@pytest.mark.parametrize("tokens", [5, 50])
@pytest.mark.parametrize("weights", ["bf16", "mx4"])
def test_gelu(weights, tokens):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(31)
    x, xv, e, wt, mats, vals = layer(rng, "bf16", weights, tokens, 2, 6, 96, 80, dev)
    got = sdm.expert_mlp(x, up(e, dev), up(wt, dev), *mats, activation="gelu")
    check(got, xv, e, wt, vals, "bf16", R.gelu)


@pytest.mark.parametrize("tokens", [1, 16, 30, 300, 1024])
def test_all_tokens_to_one_expert(tokens):
    """Every token sent to one expert, some twice, some nowhere, and choices past every range."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(tokens)
    x, xv, e, wt, mats, vals = layer(rng, "bf16", "bf16", tokens, 3, 5, 48, 40, dev)
    e[:, 0] = 3
    e[:, 1] = np.where(np.arange(tokens) % 3 == 0, 3, -5)
    e[:, 2] = np.where(np.arange(tokens) % 2 == 0, 2 ** 40, 5)
    e[tokens // 2] = [-1, 5, 2 ** 33 + 1]
    got = sdm.expert_mlp(x, up(e, dev), up(wt, dev), *mats)
    check(got, xv, e, wt, vals, "bf16")
    assert (got[tokens // 2] == 0).all()


def test_no_choice_at_all():
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(2)
    x, _, e, wt, mats, _ = layer(rng, "bf16", "bf16", 9, 2, 5, 48, 40, dev, drop=1.0)
    out = torch.full((9, 60), 5.0, dtype=torch.bfloat16, device=dev)
    sdm.expert_mlp(x, up(e, dev), up(wt, dev), *mats, out=out[:, 4:52])
    assert (out[:, 4:52] == 0).all() and (out[:, :4] == 5).all() and (out[:, 52:] == 5).all()
    none = sdm.expert_mlp(x, up(e[:, :0], dev), up(wt[:, :0], dev), *mats)
    assert none.shape == (9, 48) and (none == 0).all()
    empty = [m[:0] for m in mats]
    assert (sdm.expert_mlp(x, up(e, dev), up(wt, dev), *empty) == 0).all()
    thin = [mats[0][:, :0], mats[1][:, :0], mats[2][:, :, :0]]
    assert (sdm.expert_mlp(x, up(e, dev), up(wt, dev), *thin) == 0).all()
    assert sdm.expert_mlp(x[:0], up(e[:0], dev), up(wt[:0], dev), *mats).shape == (0, 48)


@pytest.mark.parametrize("tokens", [6, 40])
@pytest.mark.parametrize("weights", ["bf16", "mx4"])
def test_nonfinite_weights_reach_only_their_tokens(weights, tokens):
    """Experts nobody chose may hold anything; one with NaN and infinities spoils its own tokens alone, and so does a
    token that is not a number."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(7)
    x, xv, e, wt, mats, vals = layer(rng, "bf16", weights, tokens, 2, 8, 70, 90, dev)
    e[e == 2] = 4
    e[0] = [1, 6]
    e[1:][e[1:] == 1] = 5
    for m in mats:
        for bad in (2, 1):
            if weights == "mx4":
                m.scales[bad] = 255
            else:
                m[bad] = float("nan") if bad == 2 else float("inf")
    x[3] = float("nan")
    got = sdm.expert_mlp(x, up(e, dev), up(wt, dev), *mats)
    assert got[0].isnan().all() and got[3].isnan().all()
    rest = [i for i in range(tokens) if i not in (0, 3)]
    check(got[rest], xv[rest], e[rest], wt[rest], vals, "bf16")


@pytest.mark.parametrize("weights", ["bf16", "mx4"])
def test_strided_weights(weights):
    """gate and up as halves of one array, rows and experts apart, at odd addresses."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(17)
    x, xv, e, wt, mats, vals = layer(rng, "bf16", weights, 5, 2, 6, 67, 45, dev)

    def apart(t, fill):
        n, r, k = t.shape
        big = torch.full((n, r + 3, k + 5), fill, dtype=t.dtype, device=dev)[:, 2:2 + r, 3:3 + k]
        big.copy_(t)
        return big
    if weights == "mx4":
        views = [sdm.Mx4(apart(m.codes, 255), apart(m.scales, 255), m.width) for m in mats]
        both = sdm.Mx4(torch.cat([mats[0].codes, mats[1].codes], 1), torch.cat([mats[0].scales, mats[1].scales], 1), 67)
        halves = [sdm.Mx4(both.codes[:, :45], both.scales[:, :45], 67),
                  sdm.Mx4(both.codes[:, 45:], both.scales[:, 45:], 67), mats[2]]
    else:
        views = [apart(m, float("nan")) for m in mats]
        both = torch.cat(mats[:2], 1)
        halves = [both[:, :45], both[:, 45:], mats[2].transpose(1, 2).contiguous().transpose(1, 2)]
    wide = torch.full((5, 80), float("nan"), dtype=torch.bfloat16, device=dev)[:, 9:76]
    wide.copy_(x)
    ref = sdm.expert_mlp(x, up(e, dev), up(wt, dev), *mats)
    check(ref, xv, e, wt, vals, "bf16")
    for m in (views, halves):
        assert torch.equal(sdm.expert_mlp(wide, up(e, dev), up(wt, dev), *m), ref)


def test_workspace_streams_and_graphs():
    """A given workspace, a stream that is behind, two graphs over one workspace replayed in turn on new inputs."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    g = torch.Generator(device=dev).manual_seed(3)
    n, hidden, width = 12, 96, 160
    gate, upm = (torch.randn(n, hidden, width, device=dev, generator=g).bfloat16() / 12 for _ in range(2))
    down = torch.randn(n, width, hidden, device=dev, generator=g).bfloat16() / 10
    sizes = (4, 33)
    sets = [[torch.randn(t, width, device=dev, generator=g).bfloat16(),
             torch.randint(-1, n, (t, 3), device=dev, generator=g),
             torch.rand(t, 3, device=dev, generator=g)] for t in sizes]
    ws = torch.empty(max(sdm.expert_mlp_workspace(t, 3, n, width, hidden) for t in sizes), dtype=torch.uint8, device=dev)
    ws.fill_(255)
    ref = [sdm.expert_mlp(*s, gate, upm, down) for s in sets]
    for s, r in zip(sets, ref):
        assert torch.equal(sdm.expert_mlp(*s, gate, upm, down, workspace=ws), r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        late = [sdm.expert_mlp(*s, gate, upm, down, workspace=ws) for s in sets]
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(late, ref):
        assert torch.equal(a, b)
    graphs, held = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(sdm.expert_mlp(*s, gate, upm, down, workspace=ws))
        graphs.append(graph)
    for turn in range(3):
        for x, e, w in sets:
            x.copy_(torch.randn(x.shape, device=dev, generator=g))
            e.copy_(torch.randint(-1, n, e.shape, device=dev, generator=g))
            w.copy_(torch.rand(w.shape, device=dev, generator=g))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for s, h in zip(sets, held):
            assert torch.equal(sdm.expert_mlp(*s, gate, upm, down), h), turn


def test_decoding_step_together():
    """Tokens embedded, through the experts' layer, and to logits by a 4-bit product, against the same steps through
    route, dispatch, a product per expert and combine."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(23)
    vocab, t, k, n, width, hidden = 500, 10, 2, 6, 128, 96
    _, _, e, wt, mats, vals = layer(rng, "bf16", "bf16", t, k, n, width, hidden, dev)
    table, _ = typed(rng.standard_normal((vocab, width)), "bf16", dev)
    head = sdm.quantize_mx4(table)
    ids = torch.from_numpy(rng.integers(0, vocab, t)).to(dev)
    experts, weights = up(e, dev), up(wt, dev)
    x = sdm.embedding(table, ids)
    y = sdm.expert_mlp(x, experts, weights, *mats)
    logits = sdm.matmul_mx4(y, head)
    r = sdm.route(experts, n)
    rows = sdm.dispatch(x, r.position).float()
    res = torch.zeros_like(rows)
    for i in range(n):
        a, b = int(r.offsets[i]), int(r.offsets[i + 1])
        gate, upm, down = (m[i].float() for m in mats)
        inner = rows[a:b] @ gate.t()
        res[a:b] = (inner * torch.sigmoid(inner) * (rows[a:b] @ upm.t())) @ down.t()
    other = sdm.combine(res, r.position, weights)
    check(y, host(x), e, wt, vals, "bf16")
    # both within the same bound of the exact result
    ref, off = R.expert_mlp(host(x), e, wt.astype(np.float64), *vals)
    assert (np.abs(host(other) - ref) <= off + 2.0 ** -20 * np.abs(ref)).all()
    hv = R.unpack(*R.quantize(host(table)), width)
    ref, size = host(y) @ hv.T, np.abs(host(y)) @ np.abs(hv).T
    assert (np.abs(host(logits) - ref) <= R.product_bound(ref, size, width, "bf16")).all()
