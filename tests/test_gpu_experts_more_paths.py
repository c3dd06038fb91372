"""The experts' layer where other tests do not go: float16 tokens over 4-bit
weights that float16 cannot hold, tokens and weights that are not finite, and
weights past 2^31 elements."""

import numpy as np
import pytest
import torch

import mx4_ref as R
from helpers import need_gpu
from test_gpu_experts import check, layer
from test_gpu_experts_infinite import layer_of
from test_gpu_mx4 import host, rounded, typed, up

pytestmark = pytest.mark.gpu

CASES = [
    # tokens, top_k, experts, width, hidden
    (1, 8, 16, 512, 256),
    (5, 2, 6, 100, 33),
    (13, 6, 60, 1101, 173),    # more choices than a wave has lanes
    (16, 4, 5, 2100, 50),      # tokens too wide to be staged
    (40, 3, 5, 300, 128),
    (130, 2, 3, 140, 248),
]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_far_scales(kind, case):
    """Blocks of gate 2^-40 and of up 2^18 times as large as the others, down 2^-18: results of ordinary size."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    tokens, top_k, experts, width, hidden = case
    rng = np.random.default_rng([*case, 6])
    x, xv, e, wt, mats, vals = layer(rng, kind, "mx4", tokens, top_k, experts, width, hidden, dev)
    # zero blocks keep their scale of 2^-127
    for i, (by, share) in enumerate(((-40, 0.3), (18, 0.3), (-18, 1.0))):
        s = mats[i].scales.cpu().numpy().astype(int)
        s = np.where((s > 50) & (rng.random(s.shape) < share), s + by, s).astype(np.uint8)
        vals[i] = R.unpack(mats[i].codes.cpu().numpy(), s, mats[i].width)
        mats[i] = mats[i]._replace(scales=up(s, dev))
    check(sdm.expert_mlp(x, up(e, dev), up(wt, dev), *mats), xv, e, wt, vals, kind)


@pytest.mark.parametrize("kind,weights", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "mx4"), ("f16", "mx4")])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_tokens_that_are_not_finite(kind, weights, case):
    """An element of a token that gate takes once, beside 128, and up s times: infinite or NaN it makes the token's hidden
    values infinite (of s's sign; NaN where the activation's argument is minus infinity) and no other's."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    tokens, top_k, experts, width, hidden = case
    rng = np.random.default_rng([*case, len(weights), 7])
    x = np.zeros((tokens, width))
    x[:, 0], x[:, 33] = 1, rng.choice([1, 2, np.inf, -np.inf, np.nan], tokens)
    x[0, 33] = np.inf
    gate, upm = np.zeros((2, experts, hidden, width))
    s = rng.integers(-3, 4, (experts, hidden)).astype(float)
    s[s == 0] = 1
    gate[..., 0], gate[..., 33], upm[..., 33] = 128, 1, s
    down = np.zeros((experts, width, hidden))
    sign = np.where(rng.random(width) < 0.5, -1, 1)  # three columns of four agree on the sign of what they add
    agree = np.where(np.arange(width) % 4, sign, 0)[None, :, None]
    down[:] = rng.integers(1, 4, down.shape) * np.where(agree != 0, agree * np.sign(s)[:, None, :],
                                                        rng.choice([-1, 1], down.shape))
    mats = []
    for m in (gate, upm, down):
        if weights == "mx4":
            c, b = R.quantize(m.reshape(-1, m.shape[2]))
            mats.append(sdm.Mx4(up(c.reshape(*m.shape[:2], -1), dev), up(b.reshape(*m.shape[:2], -1), dev), m.shape[2]))
        else:
            mats.append(typed(m, kind, dev)[0])
    e = np.stack([rng.permutation(max(experts, top_k))[:top_k] for _ in range(tokens)])
    ones = np.ones((tokens, top_k), np.float32)
    want = np.zeros((tokens, width))
    for t in range(tokens):  # silu of 129 and 130 is they themselves in float32
        act = np.nan if x[t, 33] == -np.inf else 128 + x[t, 33]
        want[t] = layer_of(e[t:t + 1], ones[:1], act * (s * x[t, 33]), down)[0]
    got = sdm.expert_mlp(typed(x, kind, dev)[0], up(e, dev), up(ones, dev), *mats)
    np.testing.assert_array_equal(host(got), rounded(want, kind))


@pytest.mark.parametrize("weights", ["bf16", "mx4"])
@pytest.mark.parametrize("tokens", [3, 40])
def test_experts_far_apart(weights, tokens):
    """Experts 2^30 elements from one another, rows 2^20, in one array past 2^31."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(tokens)
    x, xv, e, wt, mats, vals = layer(rng, "bf16", weights, tokens, 2, 3, 200, 150, dev)
    size = 2**31 + 2**29
    space = torch.empty(size, dtype=torch.uint8 if weights == "mx4" else torch.bfloat16, device=dev)
    at = 0

    def far(t):
        nonlocal at
        view = space.as_strided(t.shape, (2**30 + 8, 2**20 + 8, 1), at)
        at += 1000
        view.copy_(t)
        return view
    views = [sdm.Mx4(far(m.codes), far(m.scales), m.width) if weights == "mx4" else far(m) for m in mats]
    ids, w = up(e, dev), up(wt, dev)
    got = sdm.expert_mlp(x, ids, w, *views)
    check(got, xv, e, wt, vals, "bf16")
    assert torch.equal(got, sdm.expert_mlp(x, ids, w, *mats))
