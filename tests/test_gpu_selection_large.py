"""The selection products where their size picks another path: rows beyond the
last-level cache (read and written nontemporally), lookups of four chunks a
lane, arrays past 2^31 elements and launches' worth of chunks, zeroing that goes
around its grid; and calls on a stream that is behind the host. Data are small
integers (sums and products exact in every type used), so results are compared
whole and for equality; a lookup's one product and rounding are torch's own."""

import pytest
import torch

from helpers import need_gpu
from test_gpu_selection import BF16, F16, F32, F64, TYPES, by_name, guarded, guards_kept, sdm, same_bits

pytestmark = pytest.mark.gpu


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def ints(shape, high, dtype, g):
    return torch.randint(-high, high + 1, shape, generator=g, device=g.device).to(dtype)


def weighted_sum(rows, pos, weights):
    """sum over k of weights[t, k] * rows[pos[t, k]], live slots only"""
    out = torch.zeros((pos.shape[0], rows.shape[1]), device=rows.device,
                      dtype=F64 if rows.dtype == F64 else F32)
    for k in range(pos.shape[1]):
        live = (pos[:, k] >= 0)[:, None]
        picked = rows[pos[:, k].clamp(min=0).long()].to(out.dtype)
        out += torch.where(live, weights[:, k, None] * picked, 0.0)
    return out.to(rows.dtype)


# Rows of more than 256 MB. The widths give combine_grad's one, two and four
# waves a token, rows of whole chunks and cut ones, and top_k of one batch, of a
# padded one and of two.
@pytest.mark.parametrize("dtype,width,k", [
    (BF16, 509, 6), (BF16, 1000, 3), (BF16, 4099, 8), (F16, 513, 9), (F16, 1024, 1),
    (F32, 250, 5), (F32, 511, 8), (F32, 1001, 6), (F64, 127, 7), (F64, 200, 2), (F64, 515, 4),
    (F32, 3, 8), (BF16, 7, 4)], ids=by_name)
def test_rows_beyond_the_caches(dtype, width, k):
    dev = need_gpu()
    g = gen(dev, width)
    size = torch.empty(0, dtype=dtype).element_size()
    t = 300_000_000 // (k * width * size)
    assert t * k * width * size > 1 << 28
    experts = torch.randint(0, 60, (t, k), generator=g, device=dev)
    experts[torch.rand((t, k), generator=g, device=dev) < 0.2] = -1
    r = sdm().route(experts, 60)
    pos, live = r.position, int(r.offsets[-1])
    assert 0 < live < t * k
    acc = F64 if dtype == F64 else F32
    weights = ints((t, k), 3, acc, g)
    rows, dout = ints((t * k, width), 4, dtype, g), ints((t, width), 4, dtype, g)
    rows[live:] = float("nan")  # behind dropped slots
    weights[pos < 0] = float("nan")

    for fn, want in (
            (lambda o: sdm().combine(rows, pos, weights, out=o), weighted_sum(rows, pos, weights)),
            (lambda o: sdm().dispatch_grad(rows, pos, out=o),
             weighted_sum(rows, pos, torch.ones_like(weights)))):
        assert torch.equal(fn(None), want)
        buf, view = guarded(t, width, dtype, dev)
        assert torch.equal(fn(view), want) and guards_kept(buf, width)

    want_rows, want_weights = torch.zeros_like(rows), torch.zeros_like(weights)
    for j in range(k):
        on = pos[:, j] >= 0
        at = pos[on, j].long()
        want_rows[at] = (weights[on, j, None] * dout[on].to(acc)).to(dtype)
        want_weights[on, j] = (dout[on].to(acc) * rows[at].to(acc)).sum(1)
    grad_rows, grad_weights = sdm().combine_grad(dout, rows, pos, weights)
    assert torch.equal(grad_rows, want_rows) and torch.equal(grad_weights, want_weights)
    buf, view = guarded(t * k, width, dtype, dev)
    _, grad_weights = sdm().combine_grad(dout, rows, pos, weights, out=view)
    assert torch.equal(view, want_rows) and torch.equal(grad_weights, want_weights)
    assert guards_kept(buf, width)


# 2^20 chunks or more, no multiple of the 1,024 that a block takes
@pytest.mark.parametrize("dtype,n,width,chunk", [
    (F32, 5003, 1023, 4), (F32, 700_001, 3, 1), (BF16, 1_300_001, 9, 8), (BF16, 300_001, 7, 1),
    (BF16, 5001, 2048, 8), (F16, 150_001, 57, 8), (F64, 600_003, 3, 2), (F64, 9001, 250, 2)],
    ids=by_name)
@pytest.mark.parametrize("index", [torch.int32, torch.int64], ids=str)
def test_lookup_of_four_chunks_a_lane(dtype, n, width, chunk, index):
    dev = need_gpu()
    chunks = n * -(-width // chunk)
    assert chunks >= 1 << 20 and chunks % 1024
    g = gen(dev, n)
    v = 3001
    wide = torch.randn((v, width + 13), generator=g, device=dev, dtype=F64).to(dtype)
    table = wide[:, 5:5 + width]
    ids = torch.randint(-300, v + 300, (n,), generator=g, device=dev).to(index)
    scale = torch.tensor(0.3, dtype=F64 if dtype == F64 else F32, device=dev)
    real = ((ids >= 0) & (ids < v))[:, None]
    want = (table[ids.clamp(0, v - 1).long()].to(scale.dtype) * scale).to(dtype)
    want = torch.where(real, want, torch.zeros((), dtype=dtype, device=dev))
    assert same_bits(sdm().embedding(table, ids, 0.3), want)
    buf, view = guarded(n, width, dtype, dev)
    sdm().embedding(table, ids, 0.3, out=view)
    assert same_bits(view, want) and guards_kept(buf, width)


def test_routing_past_one_launch():
    """307,000,000 tokens of 7 bf16 to two rows each: 2.149e9 chunks (elements)
    on the tokens' side, two launches, and 4.3e9 elements of rows."""
    dev = need_gpu()
    t, k, w = 307_000_000, 2, 7
    assert t * w > 2**31
    x = (torch.arange(t, device=dev) % 101).to(BF16)[:, None].repeat(1, w)
    x += torch.arange(w, device=dev).to(BF16)
    pos = torch.arange(t * k - 1, -1, -1, device=dev, dtype=torch.int32).reshape(t, k)
    pieces = [(a, min(a + 50_000_000, t)) for a in range(0, t, 50_000_000)]
    rows = sdm().dispatch(x, pos)
    for a, b in pieces:
        back = rows[k * (t - b):k * (t - a)].flip(0).reshape(b - a, k, w)
        for j in range(k):
            assert torch.equal(back[:, j], x[a:b]), (a, j)
    weights = (torch.arange(t * k, device=dev) % 3 - 1).float().reshape(t, k)
    out = sdm().combine(rows, pos, weights)
    for a, b in pieces:
        assert torch.equal(out[a:b], x[a:b] * weights[a:b].sum(1, keepdim=True).to(BF16)), a
    out = sdm().dispatch_grad(rows, pos, out=out)
    for a, b in pieces:
        assert torch.equal(out[a:b], x[a:b] * 2), a


def test_wide_rows_past_2_31_elements():
    """70,000 tokens of 4,096 bf16 to eight rows each: 2.29e9 elements of rows,
    an eighth of the slots dropped."""
    dev = need_gpu()
    t, k, w = 70_000, 8, 4096
    g = gen(dev, 7)
    assert t * k * w > 2**31
    x = ints((t, w), 4, BF16, g)
    experts = torch.randint(0, 128, (t, k), generator=g, device=dev)
    experts[torch.rand((t, k), generator=g, device=dev) < 0.125] = -1
    r = sdm().route(experts, 128)
    live = r.position >= 0
    rows = sdm().dispatch(x, r.position)
    where = torch.where(live, r.position, ~r.position).long()
    for j in range(k):
        assert torch.equal(rows[where[:, j]], torch.where(live[:, j, None], x, 0.0))
    weights = torch.where(live, ints((t, k), 3, F32, g), 0.0)
    assert torch.equal(sdm().combine(rows, r.position, weights),
                       (x.float() * weights.sum(1, keepdim=True)).to(BF16))
    dout = ints((t, w), 4, BF16, g)
    grad_rows, grad_weights = sdm().combine_grad(dout, rows, r.position, weights)
    dot = (dout.float() * x.float()).sum(1, keepdim=True)
    assert torch.equal(grad_weights, torch.where(live, dot, 0.0))
    for j in range(k):
        assert torch.equal(grad_rows[where[:, j]], (dout.float() * weights[:, j, None]).to(BF16))


# tables larger than the launch that zeroes them reaches at once: 2^21 blocks of
# 1,024, 256 and 512 threads (one sort each) or 256 (no tokens), 16 bytes a thread
@pytest.mark.parametrize("n,v,gap", [(100, 8_500_000, 0), (100, 8_500_000, 4), (9000, 2_200_000, 0),
                                     (9000, 2_200_000, 4), (70_000, 4_300_000, 4),
                                     (0, 2_200_000, 0), (0, 2_200_000, 4)])
def test_zeroing_goes_around_its_grid(n, v, gap):
    dev = need_gpu()
    w = 1024
    threads = 256 if n == 0 or 8192 < n <= 65_536 else 1024 if n <= 8192 else 512
    assert v * w * 4 > (1 << 21) * threads * 16
    buf = torch.full((v, w + gap), 7.0, device=dev)
    grad = buf[:, :w]
    ids = torch.arange(n, device=dev) * 7919 % v  # distinct: 7919 is prime and divides no v here
    if n:
        ids[0], ids[1] = v - 1, 0
    ids = torch.unique(ids)
    ids = ids[torch.randperm(len(ids), device=dev)]
    rows = (torch.arange(len(ids), device=dev) % 9 + 1).float()[:, None]
    sdm().embedding_grad(rows.expand(-1, w), ids, v, out=grad)
    assert torch.equal(grad[ids], rows.expand(-1, w))
    grad[ids] = 0.0
    for a in range(0, v, 500_000):
        assert int(grad[a:a + 500_000].count_nonzero()) == 0, a
        assert bool((buf[a:a + 500_000, w:] == 7.0).all()), a


def test_a_stream_that_is_behind():
    """Operands that get their values on a side stream, behind work that is still
    running when the calls are made: every call must wait its turn there. On
    any other stream it would read what the operands held before."""
    dev = need_gpu()
    g = gen(dev, 41)
    v, t, w, k, e = 3000, 4000, 515, 3, 40
    names = dict(table=torch.randn((v, w), generator=g, device=dev).to(BF16),
                 ids=torch.randint(0, v, (t,), generator=g, device=dev),
                 experts=torch.randint(0, e, (t, k), generator=g, device=dev),
                 weights=torch.rand((t, k), generator=g, device=dev),
                 position=None)
    names["position"] = sdm().route(names["experts"], e).position
    used = {name: torch.zeros_like(x) for name, x in names.items()}
    used["position"].copy_(torch.arange(t * k, device=dev).reshape(t, k))

    def calls(a):
        x = sdm().embedding(a["table"], a["ids"], 2.0)
        r = sdm().route(a["experts"], e)
        rows = sdm().dispatch(x, a["position"])
        some = torch.ones((t, w), dtype=BF16, device=dev)
        many = (torch.arange(t * k, device=dev) % 7).to(BF16)[:, None].repeat(1, w)
        return (x, *r, rows, sdm().combine(many, a["position"], a["weights"]),
                *sdm().combine_grad(some, many, a["position"], a["weights"]),
                sdm().dispatch_grad(rows, a["position"]),
                sdm().embedding_grad(some, a["ids"], v, 2.0),
                sdm().embedding_grad(x, a["ids"], v, dtype=F32))

    want = calls(names)
    stale = calls(used)
    assert not any(same_bits(a, b) for a, b in zip(want, stale))
    busy = torch.zeros((8192, 8192), device=dev)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls(used)  # its memory is there before the busy work
        side.synchronize()
        for _ in range(300):  # 0.5 GB moved each: some 30 ms
            busy += 1
        for name, x in names.items():
            used[name].copy_(x)
        set_right = torch.cuda.Event()
        set_right.record(side)
        got = calls(used)
        behind = not set_right.query()
        got = [x.clone() for x in got]
    side.synchronize()
    assert behind, "the stream was not behind: nothing was tested"
    for a, b in zip(got, want):
        assert same_bits(a, b)
