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


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


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


def test_the_widest_rows():
    """2^24 elements a row, and one element less: every operator. Ones and zeros:
    sums below 2^24, exact."""
    dev = need_gpu()
    g = gen(dev, 3)
    for w in (2**24, 2**24 - 1):
        table = torch.randint(0, 2, (5, w), generator=g, device=dev).to(BF16)
        ids = torch.tensor([4, 0, -1, 4, 2], device=dev)
        out = sdm().embedding(table, ids, 3.0)
        for t, i in enumerate(ids.tolist()):
            assert torch.equal(out[t], table[i] * 3 if i >= 0 else torch.zeros_like(out[t]))
        same = torch.full((150,), 2, device=dev)  # three segments, joined
        grad = sdm().embedding_grad(table[:1].expand(150, w), same, 3, dtype=F32)
        assert torch.equal(grad[2], table[0].float() * 150) and not grad[:2].any()
        pos = torch.tensor([[1, 3], [~4, 0], [2, ~5]], dtype=torch.int32, device=dev)
        rows = sdm().dispatch(table[:3], pos)
        for row, want in enumerate((table[1], table[0], table[2], table[0], None, None)):
            assert torch.equal(rows[row], torch.zeros_like(table[0]) if want is None else want)
        weights = torch.tensor([[2.0, 3], [5, 7], [1, 4]], device=dev)
        out = sdm().combine(rows, pos, weights)
        for t, s in enumerate((5, 7, 1)):
            assert torch.equal(out[t], table[t] * s)
        dout = table[2:]
        grad_rows, grad_weights = sdm().combine_grad(dout, rows, pos, weights)
        for (t, k), p in ((x, int(pos[x])) for x in ((0, 0), (0, 1), (1, 1), (2, 0))):
            assert torch.equal(grad_rows[p], dout[t] * weights[t, k].to(BF16))
            dot = (dout[t].float() * table[t].float()).sum(dtype=F64)
            assert float(grad_weights[t, k]) == float(dot)
        assert not grad_rows[4:].any() and grad_weights[1, 0] == 0 and grad_weights[2, 1] == 0


def test_row_strides_past_2_31_elements():
    dev = need_gpu()
    ld, w = 2**31 + 5, 37
    buf = torch.full((2 * ld + w,), 7.0, dtype=BF16, device=dev)
    far = buf.as_strided((3, w), (ld, 1))
    x = ints((3, w), 4, BF16, gen(dev, 9))
    ids = torch.tensor([2, 0, 1], device=dev)
    pos = ids.int()[:, None]
    w2 = torch.full((3, 1), 2.0, device=dev)
    back = torch.argsort(ids)
    for fn, want in ((lambda a, o: sdm().embedding(a, ids, out=o), x[ids]),
                     (lambda a, o: sdm().embedding_grad(a, ids, 3, out=o), x[back]),
                     (lambda a, o: sdm().dispatch(a, pos, out=o), x[back]),
                     (lambda a, o: sdm().combine(a, pos, w2, out=o), 2 * x[ids]),
                     (lambda a, o: sdm().dispatch_grad(a, pos, out=o), x[ids]),
                     (lambda a, o: sdm().combine_grad(a, a, pos, w2, out=o)[0], 2 * x[back])):
        far.fill_(7.0)
        assert torch.equal(fn(x, far), want)
        far.copy_(x)
        assert torch.equal(fn(far, None), want)
    far.fill_(7.0)
    for a in range(0, buf.numel(), 2**30):
        assert bool((buf[a:a + 2**30] == 7.0).all())


def test_the_longest_lookup():
    """2^31 - 1 tokens of one element, two launches."""
    dev = need_gpu()
    n = 2**31 - 1
    table = (torch.arange(100, device=dev) + 1).to(F16)[:, None]
    ids = torch.empty(n, dtype=torch.int32, device=dev)
    pieces = [(a, min(a + 2**28, n)) for a in range(0, n, 2**28)]
    for a, b in pieces:
        ids[a:b] = torch.arange(a, b, device=dev) % 101  # 100 is outside
    out = sdm().embedding(table, ids)
    for a, b in pieces:
        want = torch.where(ids[a:b] < 100, ids[a:b] + 1, 0).to(F16)
        assert torch.equal(out[a:b, 0], want), a


def test_the_longest_list_of_the_gradient():
    """2^30 tokens of one element: two sort passes of 256 tiles, 2^24 segments,
    their partial rows folded. Ones and zeros, at most 1.2e6 of a row: exact."""
    dev = need_gpu()
    n, v = 2**30, 5000
    ids = torch.empty(n, dtype=torch.int32, device=dev)
    dout = torch.empty((n, 1), dtype=BF16, device=dev)
    want = torch.zeros(v, dtype=torch.int64, device=dev)
    for a in range(0, n, 2**27):
        i = torch.arange(a, a + 2**27, device=dev)
        some = (i * 2654435761) % 1_000_003
        # a fifth of the tokens outside, row 4,999 several times the others
        part = torch.where(some < 800_000, some % v, v)
        part = torch.where(some % 1000 == 7, v - 1, part)
        on = (i // 3) % 2
        ids[a:a + 2**27], dout[a:a + 2**27, 0] = part.int(), on.to(BF16)
        want += torch.bincount(part[on == 1], minlength=v + 1)[:v]
    assert int(want.max()) < 2**24
    grad = sdm().embedding_grad(dout, ids, v, dtype=F32)
    assert torch.equal(grad[:, 0], want.float())


@pytest.mark.parametrize("t,k,e", [(2**31 - 1, 1, 61), (238_000_000, 9, 4096)])
def test_the_longest_routing(t, k, e):
    """2^31 - 1 slots, and 2.142e9 over the most experts: the order is sorted, stable
    and a permutation, position its inverse, and offsets where the experts start."""
    dev = need_gpu()
    n = t * k
    experts = torch.empty(n, dtype=torch.int32, device=dev)
    pieces = [(a, min(a + 2**27, n)) for a in range(0, n, 2**27)]
    counts = torch.zeros(e + 1, dtype=torch.int64, device=dev)
    for a, b in pieces:
        i = torch.arange(a, b, device=dev)
        experts[a:b] = ((i * 2654435761) % 1_000_003 % (e + 3)).int() - 1  # -1, e, e + 1: outside
        x = experts[a:b]
        counts += torch.bincount(torch.where((x >= 0) & (x < e), x, e), minlength=e + 1)
    order, position, offsets = sdm().route(experts.reshape(t, k), e)
    want = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), counts[:e].cumsum(0)])
    assert torch.equal(offsets.long(), want)
    position = position.reshape(-1)
    last = torch.full((2,), -1, dtype=torch.int64, device=dev)  # the piece before's last key, slot
    for a, b in pieces:
        slot = order[a:b].long()
        assert int(slot.min()) >= 0 and int(slot.max()) < n
        x = experts[slot]
        live = (x >= 0) & (x < e)
        key = torch.where(live, x, e).long()
        row = torch.arange(a, b, device=dev)
        assert torch.equal(position[slot].long(), torch.where(live, row, ~row))
        key, slot = torch.cat([last[:1], key]), torch.cat([last[1:], slot])
        assert bool(((key[1:] > key[:-1]) | ((key[1:] == key[:-1]) & (slot[1:] > slot[:-1]))).all())
        last = torch.stack([key[-1], slot[-1]])


@pytest.mark.parametrize("n,v", [(70_000, 50_021), (300_001, 400), (300_001, 5_000_000)])
def test_captured_gradient_of_long_lists(n, v):
    """The sort by digits, the fold and the join in a graph, replayed on new tokens
    between eager calls: the eager bits, accumulated ones too."""
    dev = need_gpu()
    g = gen(dev, n)
    w = 12
    ids = torch.zeros(n, dtype=torch.int64, device=dev)
    dout = torch.zeros((n, w), dtype=BF16, device=dev)
    total = torch.zeros((v, w), device=dev)

    def fresh():
        u = torch.rand(n, generator=g, device=dev, dtype=F64)
        ids.copy_((u**6 * (v + 3)).long() - 1)  # row 0 and its neighbours often, some outside
        dout.copy_(torch.randn((n, w), generator=g, device=dev))

    def step(out):
        grad = sdm().embedding_grad(dout, ids, v, 0.5)
        sdm().embedding_grad(dout, ids, v, 0.5, out=out, accumulate=True)
        return grad

    fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(total)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(total)
    for _ in range(4):
        fresh()
        eager = total.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(captured, step(eager)) and same_bits(total, eager)
