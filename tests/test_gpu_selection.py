"""The selection products on the GPU against their definitions in float64
(tests/selection_ref.py, which also derives the bounds): every element type
and both index types, widths around the 16-byte chunks and the lane groups,
no tokens and one token, padding and ids past 32 bits, strided and offset
rows with guards around what is written, runs of equal ids from one to
thousands, experts from one to 4,096, dropped slots (with NaN behind them),
other streams, captured graphs, repeated bits, and a layer of experts run
forward and backward."""

import numpy as np
import pytest
import torch

import selection_ref as R
from helpers import need_gpu

pytestmark = pytest.mark.gpu

F32, F64, BF16, F16 = torch.float32, torch.float64, torch.bfloat16, torch.float16
TYPES = [F32, F64, BF16, F16]
NAMES = {F32: "f32", F64: "f64", BF16: "bf16", F16: "f16"}
WIDTHS = [1, 2, 3, 7, 8, 9, 16, 31, 64, 65, 127, 128, 129, 255, 513, 1000, 1024, 4099]


def by_name(t):
    return NAMES.get(t, str(t))


def sdm():
    import sparse_dense_matmul_amd

    return sparse_dense_matmul_amd


def normal(rng, shape, dtype, dev):
    return torch.from_numpy(rng.standard_normal(shape)).to(dtype).to(dev)


def ints(rng, shape, dtype, dev, high=4):
    return torch.from_numpy(rng.integers(-high, high + 1, shape)).to(dtype).to(dev)


def same_bits(a, b):
    v = {8: torch.int64, 4: torch.int32, 2: torch.int16}[a.element_size()]
    return torch.equal(a.contiguous().view(v), b.contiguous().view(v))


def guarded(rows, width, dtype, dev, left=3, right=5):
    """A strided, unaligned (rows x width) view inside a buffer of 7s."""
    buf = torch.full((rows + 2, left + width + right), 7.0, dtype=dtype, device=dev)
    return buf, buf[1:rows + 1, left:left + width]


def guards_kept(buf, width, left=3):
    inside = torch.zeros_like(buf, dtype=torch.bool)
    inside[1:-1, left:left + width] = True
    return bool((buf[~inside] == 7.0).all())


# --------------------------------------------------------------- embedding


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES, ids=by_name)
def test_embedding(dtype, width):
    dev = need_gpu()
    rng = np.random.default_rng(width)
    for n, index in ((1, torch.int64), (3, torch.int32), (65, torch.int64), (300, torch.int32)):
        table = normal(rng, (50, width), dtype, dev)
        ids = rng.integers(0, 50, n)
        ids[rng.random(n) < 0.2] = -1
        if index == torch.int64 and n > 3:
            ids[:4] = [2**40 + 3, -2**40, 50, 2**32]  # the low 32 bits of the last are a row
        dids = torch.from_numpy(ids).to(index).to(dev)
        out = sdm().embedding(table, dids, scale=1.5)
        want, mag = R.embedding(R.f64(table), ids, 1.5)
        R.check(out, want, 1, mag, dtype, (n, width))
        assert same_bits(sdm().embedding(table, dids), torch.where(
            ((dids >= 0) & (dids < 50))[:, None], table[dids.clamp(0, 49).long()],
            torch.zeros((), dtype=dtype, device=dev)))  # scale 1 copies the rows


@pytest.mark.parametrize("dtype", TYPES, ids=by_name)
def test_embedding_strided(dtype):
    """Rows inside a wider buffer, at odd offsets; a transposed table (copied);
    ids of two dimensions."""
    dev = need_gpu()
    rng = np.random.default_rng(5)
    wide = normal(rng, (40, 150), dtype, dev)
    ids = rng.integers(-2, 42, (6, 7))
    dids = torch.from_numpy(ids).to(dev)
    for table in (wide[:, 5:138], wide[3:, :8], wide.t()[:, 1:34]):
        want, mag = R.embedding(R.f64(table), ids, 0.5)
        w = table.shape[1]
        out = sdm().embedding(table, dids, 0.5)
        assert out.shape == (6, 7, w)
        R.check(out.reshape(-1, w), want, 1, mag, dtype)
        buf, view = guarded(ids.size, w, dtype, dev)
        sdm().embedding(table, dids, 0.5, out=view)
        assert same_bits(view, out.reshape(-1, w)) and guards_kept(buf, w)


def test_embedding_empty():
    dev = need_gpu()
    table = torch.ones((5, 8), device=dev)
    none = torch.zeros(0, dtype=torch.int64, device=dev)
    assert sdm().embedding(table, none).shape == (0, 8)
    assert sdm().embedding(table[:, :0], torch.zeros(3, dtype=torch.int32, device=dev)).shape == (3, 0)
    out = sdm().embedding(table[:0], torch.zeros(3, dtype=torch.int32, device=dev))
    assert out.shape == (3, 8) and not out.any()


def test_embedding_of_one_id_without_dimensions():
    dev = need_gpu()
    table = torch.arange(12.0, device=dev).reshape(4, 3)
    one = torch.tensor(2, device=dev)
    assert sdm().embedding(table, one).tolist() == [6, 7, 8]
    grad = sdm().embedding_grad(torch.ones(3, device=dev), one, 4)
    assert grad.tolist() == [[0, 0, 0], [0, 0, 0], [1, 1, 1], [0, 0, 0]]


def test_embedding_nonfinite():
    """Non-finite entries reach the tokens that select them and no other."""
    dev = need_gpu()
    table = torch.ones((4, 33), dtype=BF16, device=dev)
    table[1] = float("nan")
    table[2] = float("inf")
    out = sdm().embedding(table, torch.tensor([0, 1, 2, 3, -1], device=dev), 2.0)
    assert (out[0] == 2).all() and out[1].isnan().all() and (out[2] == float("inf")).all()
    assert (out[3] == 2).all() and not out[4].any()


def test_embedding_past_2_31_elements():
    """A table of more than 2^31 elements: its last rows, forward and back."""
    dev = need_gpu()
    v, w = 600_011, 4096
    table = torch.zeros((v, w), dtype=BF16, device=dev)
    ids = torch.tensor([v - 1, 0, v - 2, 524_288, v - 1], device=dev)
    for i, row in enumerate((v - 1, 0, v - 2, 524_288)):
        table[row] = i + 1
    out = sdm().embedding(table, ids)
    assert out[:, 0].tolist() == [1, 2, 3, 4, 1] and (out == out[:, :1]).all()
    grad = sdm().embedding_grad(out, ids, v, out=table)
    assert grad[ids, 0].tolist() == [2, 2, 3, 4, 2]
    assert [int(x) for x in grad.count_nonzero(dim=1)[[v - 1, 0, v - 2, 524_288, 1, 524_287]]] == \
        [w, w, w, w, 0, 0]
    assert int(grad.any(dim=1).sum()) == 4


def test_embedding_of_more_chunks_than_a_launch_takes():
    """300,000 x 65,536 bf16 (39 GB) out: 2.4e9 chunks, two launches, the second
    from row 262,016 on."""
    dev = need_gpu()
    n, w = 300_000, 65_536
    table = torch.arange(1, 6, device=dev).to(BF16)[:, None].expand(5, w).contiguous()
    ids = torch.arange(n, device=dev) % 6  # 5 is outside
    out = sdm().embedding(table, ids)
    want = torch.where(ids < 5, ids + 1, 0).to(BF16)
    for a, b in ((0, 50), (262_000, 262_050), (n - 50, n)):
        assert torch.equal(out[a:b], want[a:b, None].expand(b - a, w)), a
    assert torch.equal(out[:, w - 1], want) and torch.equal(out[:, 0], want)


# ---------------------------------------------------------- embedding grad


def token_ids(kind, n, v, rng):
    if kind == "uniform":
        ids = rng.integers(0, v, n)
    elif kind == "same":
        ids = np.full(n, v // 2)
    elif kind == "zipf":
        ids = np.minimum(rng.zipf(1.3, n) - 1, v - 1) * 7 % v
    elif kind == "hot":  # one long run among single tokens
        ids = np.where(rng.random(n) < 0.7, v - 1, rng.integers(0, v, n))
    elif kind == "none":
        ids = np.where(rng.random(n) < 0.5, -1, v)
    else:  # padded
        ids = np.where(rng.random(n) < 0.4, -1, rng.integers(0, v, n))
    return ids.astype(np.int64)


KINDS = ["uniform", "same", "zipf", "hot", "none", "padded"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,gtype", [(F32, F32), (F64, F64), (BF16, BF16), (BF16, F32),
                                         (F16, F16), (F16, F32)], ids=by_name)
def test_embedding_grad(dtype, gtype, kind):
    dev = need_gpu()
    for n, v, w in ((1, 1, 1), (2, 9, 130), (65, 40, 7), (200, 1000, 64), (1537, 33, 200),
                    (700, 5000, 515), (5000, 300, 24)):
        rng = np.random.default_rng(n + w)
        dout = normal(rng, (n, w), dtype, dev)
        ids = token_ids(kind, n, v, rng)
        dids = torch.from_numpy(ids).to(torch.int32 if n % 2 else torch.int64).to(dev)
        grad = sdm().embedding_grad(dout, dids, v, scale=0.75, dtype=gtype)
        assert grad.dtype == gtype
        want, terms, mag = R.embedding_grad(R.f64(dout), ids, v, 0.75)
        R.check(grad, want, terms, mag, dtype, (kind, n, v, w))
        again = sdm().embedding_grad(dout, dids, v, scale=0.75, dtype=gtype)
        assert same_bits(grad, again), (kind, n, v, w)


@pytest.mark.parametrize("dtype,gtype", [(F32, F32), (F64, F64), (BF16, BF16), (BF16, F32),
                                         (F16, F32)], ids=by_name)
def test_embedding_grad_accumulates(dtype, gtype):
    """Adds to the rows selected, in a strided buffer, and touches no other."""
    dev = need_gpu()
    rng = np.random.default_rng(3)
    for n, v, w in ((1, 30, 40), (3000, 64, 133), (400, 900, 1030)):
        ids = token_ids("padded", n, v, rng)
        dout = normal(rng, (n, w), dtype, dev)
        buf, view = guarded(v, w, gtype, dev)
        view.copy_(normal(rng, (v, w), gtype, dev))
        untouched = ~np.isin(np.arange(v), ids)
        view[torch.from_numpy(untouched).to(dev)] = float("nan")
        old = view.clone()
        sdm().embedding_grad(dout, torch.from_numpy(ids).to(dev), v, scale=2.0, out=view,
                             accumulate=True)
        assert guards_kept(buf, w)
        rows = torch.from_numpy(untouched).to(dev)
        assert same_bits(view[rows], old[rows])
        want, terms, mag = R.embedding_grad(R.f64(dout), ids, v, 2.0,
                                            np.where(untouched[:, None], 0.0, R.f64(old)))
        R.check(torch.where(rows[:, None], 0.0, view), want, terms, mag, dtype, (n, v, w))


def test_embedding_grad_strided_and_shaped():
    """A gradient of ids.shape + (width,), rows of stride zero (a broadcast
    gradient), rows inside a wider buffer, and a strided result."""
    dev = need_gpu()
    rng = np.random.default_rng(8)
    ids = rng.integers(-1, 21, (5, 13))
    dids = torch.from_numpy(ids).to(dev)
    one = normal(rng, (1, 97), BF16, dev)
    wide = normal(rng, (65, 120), BF16, dev)
    for dout in (one.expand(65, 97), wide[:, 11:108], wide[:, 11:108].reshape(5, 13, 97),
                 normal(rng, (97, 65), BF16, dev).t()):
        want, terms, mag = R.embedding_grad(R.f64(dout.reshape(65, 97)), ids, 20, 1.0)
        buf, view = guarded(20, 97, F32, dev)
        sdm().embedding_grad(dout, dids, 20, out=view)
        R.check(view, want, terms, mag, F32)
        assert guards_kept(buf, 97)


def test_embedding_grad_exact_on_integers():
    """Integer data: every sum is exact, whatever the pieces; a table of two
    and of three sort passes, tokens of more than one tile."""
    dev = need_gpu()
    rng = np.random.default_rng(11)
    for n, v, w in ((30_000, 3_000, 8), (70_001, 131_072, 4), (9_000, 5_000_000, 3),
                    (600_000, 400, 1)):
        ids = token_ids("zipf", n, v, rng)
        dout = ints(rng, (n, w), F32, dev)
        dids = torch.from_numpy(ids).to(dev)
        grad = sdm().embedding_grad(dout, dids, v)
        want = np.stack([np.bincount(ids, weights=col, minlength=v) for col in R.f64(dout).T], axis=1)
        assert np.array_equal(R.f64(grad), want), (n, v, w)


@pytest.mark.parametrize("n", [8191, 8192, 8193, 16384, 16385, 32769, 65536, 65537, 131_071, 131_072, 300_000])
@pytest.mark.parametrize("kind", ["uniform", "same", "zipf", "hot", "padded"])
def test_embedding_grad_sort_paths(n, kind):
    """Lists on both sides of every length where the sort's kind changes, in
    tables of one, two and three digits: exact on integers, every row (a sum of
    at most 300,000 products of at most 3 stays below 2^24)."""
    dev = need_gpu()
    rng = np.random.default_rng(n)
    for v, w in ((7, 5), (50_021, 2), (5_000_000, 1)):
        ids = token_ids(kind, n, v, rng)
        dout = ints(rng, (n, w), F32, dev, high=3)
        dids = torch.from_numpy(ids).to(dev)
        grad = sdm().embedding_grad(dout, dids, v)
        real = (ids >= 0) & (ids < v)
        want = np.stack([np.bincount(ids[real], weights=col[real], minlength=v)
                         for col in R.f64(dout).T], axis=1)
        assert np.array_equal(R.f64(grad), want), (v, w)


@pytest.mark.parametrize("dtype,w", [(F32, 130), (F64, 5), (BF16, 600)])
@pytest.mark.parametrize("kind", ["same", "hot", "zipf", "padded"])
def test_embedding_grad_long_lists(kind, dtype, w):
    """Lists long enough that a run's partial rows are folded before their join,
    with runs that start and end anywhere in a block of folded segments: exact
    on ones and zeros (counts below 2^24 in the float32 and float64 results)."""
    dev = need_gpu()
    n, v = 300_001, 2000
    rng = np.random.default_rng(w)
    ids = token_ids(kind, n, v, rng)
    if kind == "padded":  # two long runs of odd lengths between short ones
        ids[1000:150_777] = 900
        ids[160_000:260_123] = 901
    on = rng.integers(0, 2, n)
    dout = torch.from_numpy(on).to(dev).to(dtype)[:, None].expand(n, w)
    grad = sdm().embedding_grad(dout, torch.from_numpy(ids).to(dev), v,
                                dtype=F64 if dtype == F64 else F32)
    real = ids >= 0
    want = np.bincount(ids[real], weights=on[real], minlength=v)
    assert torch.equal(grad, torch.from_numpy(want).to(dev).to(grad.dtype)[:, None].expand(v, w))


def test_embedding_grad_nonfinite():
    """A token's non-finite gradient reaches its own row of the table alone,
    whatever stands beside it in the sorted list, and a dropped token's none."""
    dev = need_gpu()
    rng = np.random.default_rng(14)
    for n, w in ((40, 33), (3000, 520)):
        ids = np.sort(rng.integers(0, 200, n))[rng.permutation(n)]
        ids[:3] = [5, 6, -1]
        ids[3:][(ids[3:] == 5) | (ids[3:] == 6)] = 7
        dout = torch.ones((n, w), dtype=BF16, device=dev)
        dout[0], dout[1], dout[2] = float("nan"), float("inf"), float("nan")
        grad = sdm().embedding_grad(dout, torch.from_numpy(ids).to(dev), 200)
        assert grad[5].isnan().all() and (grad[6] == float("inf")).all()
        rest = torch.cat([grad[:5], grad[7:]])
        count = np.bincount(ids[3:], minlength=200)
        want = torch.from_numpy(np.delete(count, [5, 6])).to(dev).to(BF16)
        assert torch.equal(rest, want[:, None].expand(198, w))


def test_embedding_grad_empty():
    dev = need_gpu()
    none = torch.zeros(0, dtype=torch.int64, device=dev)
    grad = sdm().embedding_grad(torch.zeros((0, 6), device=dev), none, 4)
    assert grad.shape == (4, 6) and not grad.any()
    keep = torch.full((4, 6), 3.0, device=dev)
    sdm().embedding_grad(torch.zeros((0, 6), device=dev), none, 4, out=keep, accumulate=True)
    assert (keep == 3).all()
    ids = torch.zeros(3, dtype=torch.int64, device=dev)
    assert sdm().embedding_grad(torch.ones((3, 6), device=dev), ids, 0).shape == (0, 6)
    assert sdm().embedding_grad(torch.ones((3, 0), device=dev), ids, 4).shape == (4, 0)


def test_embedding_gradient_against_differences():
    """<embedding(table + e), g> - <embedding(table), g> = <e, gradient>, which
    is exact for a linear map in float64 up to rounding."""
    dev = need_gpu()
    rng = np.random.default_rng(12)
    table, e = normal(rng, (60, 37), F64, dev), normal(rng, (60, 37), F64, dev)
    ids = torch.from_numpy(rng.integers(-1, 61, 500)).to(dev)
    g = normal(rng, (500, 37), F64, dev)
    grad = sdm().embedding_grad(g, ids, 60, scale=1.25)
    up = (sdm().embedding(table + e, ids, 1.25) * g).sum()
    down = (sdm().embedding(table - e, ids, 1.25) * g).sum()
    # the two sums hold 18,500 products of size ~2: errors of ~1e-11 at most
    assert abs(float(up - down) / 2 - float((grad * e).sum())) < 1e-9


# ------------------------------------------------------------------ routing


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("t,k,e", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (64, 8, 128), (257, 3, 7),
                                   (1000, 1, 4096), (4096, 2, 8), (5001, 6, 60), (16384, 8, 256),
                                   (70_000, 9, 500), (2000, 4, 0), (100_000, 1, 3000)])
def test_route(t, k, e, index):
    dev = need_gpu()
    rng = np.random.default_rng(t + k + e)
    for kind in ("uniform", "skew", "dropped", "all"):
        if kind == "uniform":
            x = rng.integers(0, max(e, 1), (t, k))
        elif kind == "skew":
            x = np.minimum(rng.geometric(0.5, (t, k)) - 1, max(e - 1, 0))
        elif kind == "dropped":
            x = rng.integers(-e - 1, 2 * e + 1, (t, k))
        else:
            x = np.full((t, k), e if t % 2 else -1)
        got = sdm().route(torch.from_numpy(x).to(index).to(dev), e)
        want = R.route(x, e)
        for name, a, b in zip(got._fields, got, want):
            assert a.dtype == torch.int32
            assert np.array_equal(a.cpu().numpy(), b), (kind, name)


def test_route_wide_ids():
    """int64 experts whose low 32 bits are in range are still outside."""
    dev = need_gpu()
    x = np.array([[2**32 + 1, 1], [-2**40, 0], [3, 2**63 - 1]])
    got = sdm().route(torch.from_numpy(x).to(dev), 4)
    for a, b in zip(got, R.route(x, 4)):
        assert np.array_equal(a.cpu().numpy(), b)


def test_route_empty():
    dev = need_gpu()
    for shape in ((0, 4), (4, 0)):
        r = sdm().route(torch.zeros(shape, dtype=torch.int32, device=dev), 9)
        assert r.order.numel() == 0 and r.position.shape == shape
        assert r.offsets.tolist() == [0] * 10
        x = torch.ones((shape[0], 8), device=dev)
        rows = sdm().dispatch(x, r.position)
        assert rows.shape == (0, 8)
        out = sdm().combine(rows, r.position, torch.ones(shape, device=dev))
        assert out.shape == (shape[0], 8) and not out.any()
        gr, gw = sdm().combine_grad(x, rows, r.position, torch.ones(shape, device=dev))
        assert gr.shape == (0, 8) and gw.shape == shape


def routed(t, k, e, drop, rng, dev):
    x = np.argsort(rng.random((t, max(e, k))), axis=1)[:, :k] % max(e, 1)
    x = np.where(rng.random((t, k)) < drop, -1, x)
    r = sdm().route(torch.from_numpy(x).to(dev), e)
    return r, r.position.cpu().numpy()


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES, ids=by_name)
def test_dispatch_combine_and_gradients(dtype, width):
    dev = need_gpu()
    for t, k, e, drop in ((1, 1, 4, 0.0), (1, 8, 16, 0.4), (33, 4, 8, 0.0), (50, 9, 12, 0.3),
                          (7, 17, 40, 0.0), (9, 2, 3, 1.0), (10, 3, 5, 0.1), (11, 5, 9, 0.2),
                          (8, 6, 8, 0.25), (6, 7, 9, 0.0)):
        rng = np.random.default_rng(t + width)
        r, pos = routed(t, k, e, drop, rng, dev)
        n = t * k
        wtype = R.acc(dtype)
        x, dout = normal(rng, (t, width), dtype, dev), normal(rng, (t, width), dtype, dev)
        rows, drows = normal(rng, (n, width), dtype, dev), normal(rng, (n, width), dtype, dev)
        weights = normal(rng, (t, k), wtype, dev)
        where = (t, k, width)
        # a dropped slot's row and weight take no part, not even as NaN
        live = int(r.offsets[-1])
        rows[live:] = float("nan")
        drows[live:] = float("nan")
        weights[r.position < 0] = float("nan")

        out = sdm().dispatch(x, r.position)
        assert np.array_equal(R.f64(out), R.dispatch(R.f64(x), pos)), where
        got = sdm().combine(rows, r.position, weights)
        want, mag = R.combine(R.f64(rows), pos, R.f64(weights))
        R.check(got, want, k + 1, mag, dtype, where)
        got = sdm().dispatch_grad(drows, r.position)
        want, mag = R.combine(R.f64(drows), pos, np.ones((t, k)))
        R.check(got, want, k + 1, mag, dtype, where)
        gr, gw = sdm().combine_grad(dout, rows, r.position, weights)
        want_gr, want_gw, mag = R.combine_grad(R.f64(dout), R.f64(rows), pos, R.f64(weights))
        R.check(gr, want_gr, 1, np.abs(want_gr), dtype, where)
        assert gw.dtype == wtype
        R.check(gw, want_gw, width + 1, mag, dtype, where)
        # the same bits again
        gr2, gw2 = sdm().combine_grad(dout, rows, r.position, weights)
        assert same_bits(gr, gr2) and same_bits(gw, gw2)


def test_combine_grad_of_more_tokens_than_a_launch_takes():
    """5,000,000 tokens of one expert each, in two launches."""
    dev = need_gpu()
    t = 5_000_000
    pos = torch.arange(t - 1, -1, -1, device=dev, dtype=torch.int32)[:, None].contiguous()
    rows = (torch.arange(t, device=dev) % 1000).float()[:, None].expand(t, 4).contiguous()
    dout = (torch.arange(t, device=dev) % 7).float()[:, None].expand(t, 4)
    gr, gw = sdm().combine_grad(dout, rows, pos, torch.full((t, 1), 2.0, device=dev))
    assert torch.equal(gr, 2 * dout.flip(0))
    assert torch.equal(gw[:, 0], 4 * dout[:, 0] * rows[:, 0].flip(0))


@pytest.mark.parametrize("dtype", TYPES, ids=by_name)
def test_routing_strided(dtype):
    """Operands and results inside wider buffers at odd offsets."""
    dev = need_gpu()
    rng = np.random.default_rng(21)
    t, k, e, w = 37, 3, 6, 133
    r, pos = routed(t, k, e, 0.2, rng, dev)
    wide = normal(rng, (t * k + 9, 160), dtype, dev)
    x, rows, dout = wide[2:2 + t, 5:5 + w], wide[9:, 17:17 + w], wide[4:4 + t, 1:1 + w]
    weights = normal(rng, (k, t), R.acc(dtype), dev).t()
    for fn, shape in ((lambda o: sdm().dispatch(x, r.position, out=o), (t * k, w)),
                      (lambda o: sdm().combine(rows, r.position, weights, out=o), (t, w)),
                      (lambda o: sdm().dispatch_grad(rows, r.position, out=o), (t, w)),
                      (lambda o: sdm().combine_grad(dout, rows, r.position, weights, out=o)[0],
                       (t * k, w))):
        buf, view = guarded(*shape, dtype, dev)
        plain = fn(None)
        fn(view)
        assert same_bits(view, plain) and guards_kept(buf, w)
    want, mag = R.combine(R.f64(rows), pos, R.f64(weights))
    R.check(sdm().combine(rows, r.position, weights), want, k + 1, mag, dtype)


def test_positions_out_of_range():
    """Entries that name no row are passed over: nothing is read or written
    outside the operands."""
    dev = need_gpu()
    pos = torch.tensor([[0, 9], [2**31 - 1, 1], [-2**31, -6]], dtype=torch.int32, device=dev)
    x = torch.arange(1.0, 4.0, device=dev)[:, None].expand(3, 40)
    buf, rows = guarded(6, 40, F32, dev)
    sdm().dispatch(x, pos, out=rows)
    assert guards_kept(buf, 40)
    assert rows[:, 0].tolist() == [1, 2, 7, 7, 7, 0]  # ~(-6) = 5, a dropped slot's row
    out = sdm().combine(torch.ones((6, 40), device=dev), pos, torch.ones((3, 2), device=dev))
    assert out[:, 0].tolist() == [1, 1, 0]
    buf, rows = guarded(6, 40, F32, dev)
    _, gw = sdm().combine_grad(x, torch.ones((6, 40), device=dev), pos,
                               torch.full((3, 2), 2.0, device=dev), out=rows)
    assert guards_kept(buf, 40)
    assert rows[:, 0].tolist() == [2, 4, 7, 7, 7, 0]
    assert gw.tolist() == [[40, 0], [0, 80], [0, 0]]


def test_combine_is_the_csr_product():
    """combine equals the CSR product whose rows hold a token's slots, and
    dispatch_grad the product with unit values; integer data, exact."""
    dev = need_gpu()
    rng = np.random.default_rng(31)
    t, k, w = 200, 4, 48
    r, _ = routed(t, k, 16, 0.0, rng, dev)
    rows, weights = ints(rng, (t * k, w), F32, dev), ints(rng, (t, k), F32, dev)
    ptr = torch.arange(0, t * k + 1, k, dtype=torch.int32, device=dev)
    A = sdm().CsrMatrix.from_arrays((t, t * k), ptr, r.position.reshape(-1), weights.reshape(-1))
    assert torch.equal(A @ rows, sdm().combine(rows, r.position, weights))
    x = ints(rng, (t, w), F32, dev)
    ones = sdm().CsrMatrix.from_arrays((t, t * k), ptr, r.position.reshape(-1),
                                       torch.ones(t * k, device=dev))
    assert torch.equal(ones.spmm(x, "BA"), sdm().dispatch(x, r.position))


def test_the_same_expert_twice_and_one_expert_for_all():
    """Equal experts of one token are separate slots; one expert holding every
    slot keeps their order."""
    dev = need_gpu()
    x = np.array([[3, 3], [1, 3], [3, 3]])
    r = sdm().route(torch.from_numpy(x).to(dev), 5)
    assert r.order.tolist() == [2, 0, 1, 3, 4, 5] and r.offsets.tolist() == [0, 0, 1, 1, 6, 6]
    rows = torch.ones((6, 9), device=dev)
    out = sdm().combine(rows, r.position, torch.tensor([[1.0, 2], [3, 4], [5, 6]], device=dev))
    assert out[:, 0].tolist() == [3, 7, 11]


# ------------------------------------------------- streams, graphs, refusals


def test_on_another_stream():
    """Calls on a side stream while the default stream is busy: results only
    depend on the side stream's order."""
    dev = need_gpu()
    rng = np.random.default_rng(41)
    table = normal(rng, (3000, 515), BF16, dev)
    ids = torch.from_numpy(token_ids("zipf", 4000, 3000, rng)).to(dev)
    want = sdm().embedding(table, ids, 2.0)
    want_grad = sdm().embedding_grad(want, ids, 3000)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.zeros((4096, 4096), device=dev)
    for _ in range(20):
        busy = busy + 1
    with torch.cuda.stream(side):
        out = sdm().embedding(table, ids, 2.0)
        grad = sdm().embedding_grad(out, ids, 3000)
    side.synchronize()
    assert same_bits(out, want) and same_bits(grad, want_grad)


@pytest.mark.parametrize("t,e", [(16, 12), (1500, 12), (9000, 3000)])
def test_captured_graph(t, e):
    """One training step's calls in a graph, replayed on new inputs: every
    replay gives the eager bits."""
    dev = need_gpu()
    rng = np.random.default_rng(t)
    v, w, k = 700, 260, 4
    table = normal(rng, (v, w), BF16, dev)
    ids = torch.zeros(t, dtype=torch.int64, device=dev)
    experts = torch.zeros((t, k), dtype=torch.int64, device=dev)
    weights = torch.zeros((t, k), device=dev)

    def step():
        x = sdm().embedding(table, ids, 1.5)
        r = sdm().route(experts, e)
        rows = sdm().dispatch(x, r.position)
        out = sdm().combine(rows, r.position, weights)
        gr, gw = sdm().combine_grad(out, rows, r.position, weights)
        gx = sdm().dispatch_grad(gr, r.position)
        return (*r, rows, out, gr, gw, gx, sdm().embedding_grad(gx, ids, v, 1.5))

    def fresh():
        ids.copy_(torch.from_numpy(token_ids("zipf", t, v, rng)))
        experts.copy_(torch.from_numpy(rng.integers(-1, e, (t, k))))
        weights.copy_(torch.from_numpy(rng.random((t, k))))

    fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(4):
        fresh()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, step()):
            assert same_bits(a, b)


def test_calls_on_two_streams_at_once():
    """The same operators on two streams, each with its own workspace, while
    both run: the bits of one after the other."""
    dev = need_gpu()
    rng = np.random.default_rng(61)
    ids = [torch.from_numpy(token_ids("zipf", 20_000, 5000, rng)).to(dev) for _ in range(2)]
    dout = [normal(rng, (20_000, 256), BF16, dev) for _ in range(2)]
    experts = [torch.from_numpy(rng.integers(0, 64, (20_000, 2))).to(dev) for _ in range(2)]

    def work(i):
        r = sdm().route(experts[i], 64)
        rows = sdm().dispatch(dout[i], r.position)
        return sdm().embedding_grad(dout[i], ids[i], 5000), r.position, rows

    want = [work(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(work(i))
    torch.cuda.synchronize()
    for i in range(2):
        for result in got[i]:
            for a, b in zip(result, want[i]):
                assert same_bits(a, b)


def test_workspace_given():
    """A caller's workspace, filled with ones before each call, serves calls of
    any smaller size after one another."""
    dev = need_gpu()
    rng = np.random.default_rng(62)
    ws = torch.empty(sdm().embedding_grad_workspace(400, 300, 9000, BF16), dtype=torch.uint8,
                     device=dev)
    for n in (9000, 8000, 100, 8500):
        ids = torch.from_numpy(token_ids("hot", n, 400, rng)).to(dev)
        dout = normal(rng, (n, 300), BF16, dev)
        ws.fill_(255)
        got = sdm().embedding_grad(dout, ids, 400, workspace=ws)
        assert same_bits(got, sdm().embedding_grad(dout, ids, 400)), n


def test_refusals_on_the_device():
    dev = need_gpu()
    S = sdm()
    x = torch.zeros((4, 8), device=dev)
    ids = torch.zeros(4, dtype=torch.int64, device=dev)
    pos = torch.zeros((4, 2), dtype=torch.int32, device=dev)
    w = torch.zeros((4, 2), device=dev)
    rows = torch.zeros((8, 8), device=dev)
    for error, fn in [
        (TypeError, lambda: S.embedding(x, ids.float())),
        (ValueError, lambda: S.embedding(x, ids.cpu())),
        (ValueError, lambda: S.embedding(x[0], ids)),
        (ValueError, lambda: S.embedding(x, ids, out=torch.zeros((4, 9), device=dev))),
        (ValueError, lambda: S.embedding(x, ids, out=torch.zeros((8, 4), device=dev).t())),
        (ValueError, lambda: S.embedding(x, ids, out=torch.zeros((1, 8), device=dev).expand(4, 8))),
        (TypeError, lambda: S.embedding(x, ids, out=x.double())),
        (ValueError, lambda: S.embedding_grad(x[:3], ids, 9)),
        (ValueError, lambda: S.embedding_grad(x, ids, 9, accumulate=True)),
        (TypeError, lambda: S.embedding_grad(x, ids, 9, dtype=torch.int32)),
        (S.VspmmError, lambda: S.embedding_grad(x, ids, 9, dtype=F64)),
        (S.VspmmError, lambda: S.embedding_grad(x, ids, -1)),
        (S.VspmmError, lambda: S.embedding_grad(
            x, ids, 9, workspace=torch.zeros(1, dtype=torch.uint8, device=dev))),
        (ValueError, lambda: S.route(ids, 4)),
        (S.VspmmError, lambda: S.route(pos, 4097)),
        (S.VspmmError, lambda: S.route(pos, -1)),
        (TypeError, lambda: S.route(w, 4)),
        (TypeError, lambda: S.dispatch(x, pos.long())),
        (ValueError, lambda: S.dispatch(x[:3], pos)),
        (ValueError, lambda: S.combine(rows[:7], pos, w)),
        (TypeError, lambda: S.combine(rows, pos, w.double())),
        (TypeError, lambda: S.combine(rows.to(BF16), pos, w.to(BF16))),
        (ValueError, lambda: S.combine(rows, pos, w[:, :1])),
        (ValueError, lambda: S.combine_grad(x[:3], rows, pos, w)),
        (TypeError, lambda: S.combine_grad(x.double(), rows, pos, w)),
    ]:
        with pytest.raises(error):
            fn()


# ------------------------------------------------------------ used together


def test_a_layer_of_experts_forward_and_backward():
    """Tokens embedded, routed, passed through their experts' matrices and
    brought back with the router's weights; then every gradient back to the
    table, against the same layer written with dense torch operations on the
    host in float64 and its autograd."""
    dev = need_gpu()
    rng = np.random.default_rng(51)
    v, t, w, e, k = 90, 120, 24, 6, 2
    table, mats = normal(rng, (v, w), F64, dev), normal(rng, (e, w, w), F64, dev)
    ids = torch.from_numpy(rng.integers(-1, v, t)).to(dev)
    experts = torch.from_numpy(np.argsort(rng.random((t, e)), axis=1)[:, :k]).to(dev)
    weights = torch.from_numpy(rng.random((t, k))).to(dev)
    target = normal(rng, (t, w), F64, dev)

    x = sdm().embedding(table, ids, 3.0)
    r = sdm().route(experts, e)
    rows = sdm().dispatch(x, r.position)
    offs = r.offsets.tolist()
    ys = torch.cat([rows[offs[i]:offs[i + 1]] @ mats[i] for i in range(e)])
    out = sdm().combine(ys, r.position, weights)
    dout = out - target
    dys, dweights = sdm().combine_grad(dout, ys, r.position, weights)
    drows = torch.cat([dys[offs[i]:offs[i + 1]] @ mats[i].t() for i in range(e)])
    dx = sdm().dispatch_grad(drows, r.position)
    dtable = sdm().embedding_grad(dx, ids, v, 3.0)

    ct, cm, cw = (a.cpu().clone().requires_grad_(True) for a in (table, mats, weights))
    cids = ids.cpu()
    cx = torch.where((cids >= 0)[:, None], 3.0 * ct[cids.clamp(0)], 0.0)
    every = (cx[:, None, None, :] @ cm[experts.cpu()]).squeeze(2)
    cout = (cw[:, :, None] * every).sum(1)
    ((cout - target.cpu())**2 / 2).sum().backward()
    # products and sums of at most 24 and some hundred terms of size up to ~1e3
    for got, want in ((out, cout.detach()), (dweights, cw.grad), (dtable, ct.grad)):
        scale = float(want.abs().max())
        assert float((got.cpu() - want).abs().max()) < 1e-12 * scale
