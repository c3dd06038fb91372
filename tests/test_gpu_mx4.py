"""Microscaled 4-bit matrices on the GPU against numpy in 64 bits: quantisation
code by code, products bit for bit on data whose sums float32 holds exactly and
within a bound derived from the arithmetic on other data."""

import numpy as np
import pytest
import torch

import mx4_ref as R
from helpers import need_gpu

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def up(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def typed(a, kind, dev):
    """a rounded to the type, on the device, and the values it then holds."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[kind])
    return t.to(dev), t.double().numpy()


def host(t):
    return t.double().cpu().numpy()


def packed(codes, scales, width, dev):
    import sparse_dense_matmul_amd as sdm
    return sdm.Mx4(up(codes, dev), up(scales, dev), width)


def small_matrix(rng, n, width, low=-2, high=2):
    """Random codes and scales 2^low .. 2^high: every value a multiple of 2^(low - 1)."""
    b = R.blocks(width)
    c = rng.integers(0, 16, (n, 32 * b)).astype(np.uint8)
    c[:, width:] = 0
    codes = c[:, 0::2] | (c[:, 1::2] << 4)
    return codes, rng.integers(127 + low, 128 + high, (n, b)).astype(np.uint8)


def rounded(ref, kind):
    return torch.from_numpy(ref).to(torch.float32).to(TYPES[kind]).double().numpy()


def same(got, want):
    np.testing.assert_array_equal(host(got), want)


# ------------------------------------------------------------- quantisation

def values(rng, n, width):
    """Normal values over many exponents, ties and borders of codes among them,
    zeros of both signs, and blocks of zeros."""
    x = rng.standard_normal((n, width)) * np.exp2(rng.integers(-12, 12, (n, width)))
    tie = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5, 0.0, -0.0])
    at = rng.random((n, width)) < 0.4
    x[at] = (rng.choice(tie, (n, width)) * np.where(rng.random((n, width)) < 0.5, -1, 1) * 4.0)[at]
    x[rng.random(n) < 0.1] = 0
    return x


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("shape", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 100), (33, 65), (257, 130),
                                   (64, 256), (300, 1023), (1, 4096), (513, 7)])
def test_quantize_gives_every_code(kind, transpose, shape):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([shape[0], shape[1], transpose])
    x, v = typed(values(rng, *shape), kind, dev)
    got = sdm.quantize_mx4(x, transpose=transpose)
    codes, scales = R.quantize(v.T if transpose else v)
    assert got.width == (shape[0] if transpose else shape[1])
    np.testing.assert_array_equal(got.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(got.codes.cpu().numpy(), codes)
    same(sdm.dequantize_mx4(got, torch.float32), R.unpack(codes, scales, got.width))


@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_extremes(transpose):
    """Subnormal blocks, the largest numbers, infinities and NaN, one block each."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(3)
    x = np.zeros((9, 64))
    x[0, :32] = rng.integers(-9, 10, 32) * 2.0 ** -149
    x[1, :32] = rng.standard_normal(32) * 2.0 ** -126
    x[2, :32] = rng.uniform(-1, 1, 32) * 3.4e38
    x[3, 5], x[3, 40] = np.inf, 1.0
    x[4, 40] = np.nan
    x[5, 0], x[5, 63] = -np.inf, np.nan
    x[6] = 2.0 ** -127
    x[7] = rng.standard_normal(64) * np.exp2(rng.integers(-140, 120, 64))
    x[8, 3] = -0.0
    t = torch.from_numpy(x).float()
    v = t.double().numpy()
    got = sdm.quantize_mx4((t.t().contiguous() if transpose else t).to(dev), transpose=transpose)
    codes, scales = R.quantize(v)
    np.testing.assert_array_equal(got.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(got.codes.cpu().numpy(), codes)
    same(sdm.dequantize_mx4(got, torch.float32), R.unpack(codes, scales, 64))


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_dequantize_every_code_and_scale(kind):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8), 16)[:, None]
    for width in (32, 27):
        ref = torch.from_numpy(R.unpack(codes, scales, width)).to(torch.float32)
        got = sdm.dequantize_mx4(packed(codes, scales, width, dev), TYPES[kind]).cpu()
        np.testing.assert_array_equal(got.double().numpy(), ref.to(TYPES[kind]).double().numpy())


def test_quantize_strided_views():
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(5)
    big, v = typed(values(rng, 70, 200), "bf16", dev)
    for transpose in (False, True):
        for view, ref in ((big[3:60:2, 7:150], v[3:60:2, 7:150]), (big[:, ::3], v[:, ::3]),
                          (big[4:5].expand(40, 200), np.repeat(v[4:5], 40, 0)), (big.t(), v.T)):
            got = sdm.quantize_mx4(view, transpose=transpose)
            codes, scales = R.quantize(ref.T if transpose else ref)
            np.testing.assert_array_equal(got.codes.cpu().numpy(), codes)
            np.testing.assert_array_equal(got.scales.cpu().numpy(), scales)
    # rows of a matrix of more rows, as strided codes and scales
    q = sdm.quantize_mx4(big)
    part = sdm.Mx4(q.codes[1::3], q.scales[1::3], q.width)
    out = torch.full((24, 250), 7.0, dtype=torch.float32, device=dev)[:23, 20:220]
    sdm.dequantize_mx4(part, out=out)
    same(out, host(sdm.dequantize_mx4(q, torch.float32))[1::3])


# ----------------------------------------------------------------- products

MS = [1, 2, 15, 16, 17, 33, 48, 64, 65, 100, 129, 260]


def exact_case(rng, m, n, width, kind, dev):
    """Tokens of small integers and a matrix of small values: float32 sums are exact."""
    x, xv = typed(rng.integers(-8, 9, (m, width)), kind, dev)
    codes, scales = small_matrix(rng, n, width)
    return x, xv, packed(codes, scales, width, dev), R.unpack(codes, scales, width)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m", MS)
def test_matmul_is_exact(kind, m):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, kind == "f16"])
    for n, width in ((1, 1), (15, 31), (16, 32), (17, 33), (100, 64), (257, 65), (31, 127), (64, 128), (33, 129),
                     (300, 1000), (128, 2048), (1000, 257), (7, 4100)):
        x, xv, w, wv = exact_case(rng, m, n, width, kind, dev)
        same(sdm.matmul_mx4(x, w), rounded(xv @ wv.T, kind))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m", MS)
def test_matmul_grad_is_exact(kind, m):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, kind == "f16", 1])
    for n, width in ((1, 1), (15, 31), (16, 32), (17, 33), (100, 64), (257, 65), (31, 127), (64, 128), (33, 129),
                     (300, 1000), (128, 2048), (1000, 257), (4100, 7)):
        g, gv = typed(rng.integers(-8, 9, (m, n)), kind, dev)
        codes, scales = small_matrix(rng, n, width)
        got = sdm.matmul_mx4_grad(g, packed(codes, scales, width, dev))
        same(got, rounded(gv @ R.unpack(codes, scales, width), kind))


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m", MS)
def test_matmul_of_two_is_exact(kind, m):
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, len(kind), 2])
    for n, width in ((1, 1), (15, 31), (16, 32), (17, 33), (100, 64), (257, 65), (31, 127), (64, 128), (33, 129),
                     (300, 1000), (128, 2048), (1000, 257), (7, 4100), (65, 255), (65, 256), (65, 289)):
        a, sa = small_matrix(rng, m, width, -1, 1)
        b, sb = small_matrix(rng, n, width, -1, 1)
        got = sdm.matmul_mx4(packed(a, sa, width, dev), packed(b, sb, width, dev), dtype=TYPES[kind])
        same(got, rounded(R.unpack(a, sa, width) @ R.unpack(b, sb, width).T, kind))


@pytest.mark.parametrize("m,n,width", [(1, 512, 4096), (37, 1003, 1001), (64, 257, 8192), (200, 300, 999),
                                       (515, 1111, 2049), (1024, 2048, 512), (3000, 3001, 100)])
def test_products_within_their_bound(m, n, width):
    """Ordinary values, every path: the bound counts each addition and the rounding."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, n, width])
    w = rng.standard_normal((n, width)) / np.sqrt(width)
    codes, scales = R.quantize(w.astype(np.float32).astype(np.float64))
    wq, wv = packed(codes, scales, width, dev), R.unpack(codes, scales, width)
    for kind in ("bf16", "f16"):
        x, xv = typed(rng.standard_normal((m, width)) * np.exp(rng.standard_normal(width)), kind, dev)
        ref, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
        assert (np.abs(host(sdm.matmul_mx4(x, wq)) - ref) <= R.product_bound(ref, size, width, kind)).all()
        g, gv = typed(rng.standard_normal((m, n)), kind, dev)
        ref, size = gv @ wv, np.abs(gv) @ np.abs(wv)
        assert (np.abs(host(sdm.matmul_mx4_grad(g, wq)) - ref) <= R.product_bound(ref, size, n, kind)).all()
        c, s = R.quantize(xv)
        v = R.unpack(c, s, width)
        ref, size = v @ wv.T, np.abs(v) @ np.abs(wv).T
        got = sdm.matmul_mx4(sdm.quantize_mx4(x), wq, dtype=TYPES[kind])
        assert (np.abs(host(got) - ref) <= R.product_bound(ref, size, width, kind)).all()


@pytest.mark.parametrize("m", [1, 40, 64, 65, 200])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_far_scales(kind, m):
    """Scales from 2^-100 to 2^60 in one row: float16 cannot hold these weights, the products are right all the same."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, 9])
    n, width = 70, 320
    codes, scales = small_matrix(rng, n, width)
    scales[:, :] = 127 + rng.choice([-100, -60, -24, -23, -10, 0], scales.shape).astype(np.int64)
    scales[5, 3] = 127 + 13
    scales[6, 3] = 127 + 14
    scales[7, 1] = 0
    x, xv = typed(rng.standard_normal((m, width)), kind, dev)
    w, wv = packed(codes, scales, width, dev), R.unpack(codes, scales, width)
    ref, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    ok = np.abs(ref) < 60000
    got = host(sdm.matmul_mx4(x, w))
    assert (np.abs(got - ref)[ok] <= R.product_bound(ref, size, width, kind)[ok]).all()
    # only small ones: what float16 flushes must not be lost before the sum is scaled up by the tokens
    scales[:] = 127 - 30
    x, xv = typed(rng.integers(-8, 9, (m, width)) * 2048, kind, dev)
    wv = R.unpack(codes, scales, width)
    same(sdm.matmul_mx4(x, packed(codes, scales, width, dev)), rounded(xv @ wv.T, kind))
    g, gv = typed(rng.integers(-8, 9, (m, n)) * 2048, kind, dev)
    same(sdm.matmul_mx4_grad(g, packed(codes, scales, width, dev)), rounded(gv @ wv, kind))


@pytest.mark.parametrize("m", [3, 50, 130])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_nonfinite_values_stay_in_their_rows(kind, m):
    """An infinity or NaN of a token, and a NaN block of the matrix, reach the results that multiply them alone."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, 4])
    n, width = 90, 200
    x = rng.integers(1, 9, (m, width)).astype(float)
    x[0, 70], x[1, 199], x[2, 3] = np.inf, np.nan, -np.inf
    xt, xv = typed(x, kind, dev)
    codes, scales = small_matrix(rng, n, width)
    codes = (codes & 0x77) | 0x11  # positive, none zero
    codes[:, (width + 1) // 2:] = 0
    scales[17, 2] = 255
    w, wv = packed(codes, scales, width, dev), R.unpack(codes, scales, width)
    with np.errstate(invalid="ignore"):
        same(sdm.matmul_mx4(xt, w), rounded(xv @ wv.T, kind))
        g = rng.integers(1, 9, (m, n)).astype(float)
        g[0, 5], g[1, 60], g[2, 89] = np.inf, np.nan, -np.inf
        gt, gv = typed(g, kind, dev)
        same(sdm.matmul_mx4_grad(gt, w), rounded(gv @ wv, kind))
        q, s = R.quantize(xv)
        got = sdm.matmul_mx4(sdm.quantize_mx4(xt), w, dtype=TYPES[kind])
        same(got, rounded(R.unpack(q, s, width) @ wv.T, kind))


@pytest.mark.parametrize("m", [2, 40, 64, 70, 300])
def test_strides_and_alignment(m):
    """Rows of any stride and alignment, NaN between them; out's gaps stay."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng([m, 6])
    n, width = 75, 163
    for kind in ("bf16", "f16"):
        codes, scales = small_matrix(rng, n, width)
        wv = R.unpack(codes, scales, width)
        # codes and scales in rows of larger arrays, at odd addresses
        c = torch.full((n, codes.shape[1] + 19), 255, dtype=torch.uint8, device=dev)[:, 3:3 + codes.shape[1]]
        s = torch.full((n, scales.shape[1] + 3), 255, dtype=torch.uint8, device=dev)[:, 1:1 + scales.shape[1]]
        c.copy_(up(codes, dev))
        s.copy_(up(scales, dev))
        w = sdm.Mx4(c, s, width)
        for rows, k in ((m, width), (m, n)):
            v = rng.integers(-8, 9, (rows, k)).astype(float)
            x = torch.full((rows, k + 9), float("nan"), dtype=TYPES[kind], device=dev)[:, 5:5 + k]
            x.copy_(up(v, dev))
            grad = k == n
            ref = rounded(v @ (wv if grad else wv.T), kind)
            base = torch.full((rows, ref.shape[1] + 4), 3.0, dtype=TYPES[kind], device=dev)
            out = base[:, 1:-3]
            got = (sdm.matmul_mx4_grad if grad else sdm.matmul_mx4)(x, w, out=out)
            assert got.data_ptr() == out.data_ptr()
            same(out, ref)
            assert (base[:, 0] == 3).all() and (base[:, -3:] == 3).all()
            # one row for all, and columns apart (copied)
            one = x[:1].expand(rows, k)
            same((sdm.matmul_mx4_grad if grad else sdm.matmul_mx4)(one, w), np.repeat(
                rounded(v[:1] @ (wv if grad else wv.T), kind), rows, 0))
            wide = torch.zeros(rows, 2 * k, dtype=TYPES[kind], device=dev)
            wide[:, ::2] = x
            same((sdm.matmul_mx4_grad if grad else sdm.matmul_mx4)(wide[:, ::2], w), ref)
        a, sa = small_matrix(rng, m, width, -1, 1)
        ac = torch.zeros(m, a.shape[1] + 5, dtype=torch.uint8, device=dev)[:, 5:]
        ac.copy_(up(a, dev))
        sc = torch.zeros(m, sa.shape[1] + 7, dtype=torch.uint8, device=dev)[:, 7:]
        sc.copy_(up(sa, dev))
        same(sdm.matmul_mx4(sdm.Mx4(ac, sc, width), w), rounded(R.unpack(a, sa, width) @ wv.T, "bf16"))


def test_empty_extents():
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    for t in (False, True):
        for shape in ((0, 5), (5, 0), (0, 0)):
            q = sdm.quantize_mx4(z(*shape), transpose=t)
            assert sdm.dequantize_mx4(q).shape == (shape[::-1] if t else shape)
    w = sdm.quantize_mx4(z(6, 40))
    assert sdm.matmul_mx4(z(0, 40), w).shape == (0, 6)
    assert sdm.matmul_mx4_grad(z(0, 6), w).shape == (0, 40)
    assert sdm.matmul_mx4(z(3, 40), sdm.quantize_mx4(z(0, 40))).shape == (3, 0)
    none = sdm.quantize_mx4(z(6, 0))
    for got in (sdm.matmul_mx4(z(3, 0), none), sdm.matmul_mx4(sdm.quantize_mx4(z(3, 0)), none)):
        assert got.shape == (3, 6) and (got == 0).all()
    got = sdm.matmul_mx4_grad(z(3, 0), sdm.quantize_mx4(z(0, 40)))
    assert got.shape == (3, 40) and (got == 0).all()
    assert sdm.matmul_mx4_grad(z(3, 6), none).shape == (3, 0)


def test_gradient_is_that_of_differences():
    """The product is linear in x: on data whose sums are exact, the change of the
    result along a step equals the gradient's product with it, to the last bit."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(8)
    for m in (4, 90):
        n, width = 60, 130
        codes, scales = small_matrix(rng, n, width, 0, 0)  # values to 6 in halves
        codes &= np.uint8(0x33)  # to 1.5: results stay in bfloat16's eight bits on two entries a token
        w = packed(codes, scales, width, dev)
        x = np.zeros((m, width))
        x[np.arange(m), rng.integers(0, width, m)] = 1
        step = np.zeros((m, width))
        step[np.arange(m), rng.integers(0, width, m)] = 2
        g, gv = typed(rng.integers(-3, 4, (m, n)), "bf16", dev)
        before = host(sdm.matmul_mx4(typed(x, "bf16", dev)[0], w))
        after = host(sdm.matmul_mx4(typed(x + step, "bf16", dev)[0], w))
        change = ((after - before) * gv).sum(1)
        grad = host(sdm.matmul_mx4_grad(g, w))
        ref = gv @ R.unpack(codes, scales, width)
        np.testing.assert_array_equal(grad, rounded(ref, "bf16"))
        np.testing.assert_array_equal(change, (ref * step).sum(1))


def test_training_step_in_four_bits():
    """A linear layer's forward and backward products with both sides in 4 bits,
    each quantised along what it contracts, as one run."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    rng = np.random.default_rng(12)
    m, n, k = 300, 190, 270
    x, xv = typed(rng.standard_normal((m, k)), "bf16", dev)
    w, wv = typed(rng.standard_normal((n, k)) / 16, "bf16", dev)
    y = sdm.matmul_mx4(sdm.quantize_mx4(x), sdm.quantize_mx4(w))
    grad_y = (y * 0.01).to(torch.bfloat16)
    gv = host(grad_y)
    grad_x = sdm.matmul_mx4(sdm.quantize_mx4(grad_y), sdm.quantize_mx4(w, transpose=True))
    grad_w = sdm.matmul_mx4(sdm.quantize_mx4(grad_y, transpose=True), sdm.quantize_mx4(x, transpose=True),
                            dtype=torch.float32)

    def q(v):
        return R.unpack(*R.quantize(v), v.shape[1])
    for got, a, b, kind in ((y, q(xv), q(wv), "bf16"), (grad_x, q(gv), q(wv.T), "bf16"),
                            (grad_w, q(gv.T), q(xv.T), "f32")):
        ref, size = a @ b.T, np.abs(a) @ np.abs(b).T
        assert (np.abs(host(got) - ref) <= R.product_bound(ref, size, a.shape[1], kind)).all()


def test_repeats_and_graphs():
    """Equal bits from call to call, on a stream that is behind, and from a graph
    replayed on new inputs with eager work between."""
    dev = need_gpu()
    import sparse_dense_matmul_amd as sdm
    g = torch.Generator(device=dev).manual_seed(1)
    w = sdm.quantize_mx4(torch.randn(500, 700, device=dev, generator=g))
    xs = [torch.randn(m, 700, device=dev, generator=g).bfloat16() for m in (3, 150)]

    def all_of():
        out = []
        for x in xs:
            y = sdm.matmul_mx4(x, w)
            q = sdm.quantize_mx4(x)
            out += [y, sdm.matmul_mx4_grad(y, w), sdm.matmul_mx4(q, w), sdm.dequantize_mx4(q),
                    sdm.quantize_mx4(y, transpose=True).codes]
        return out
    ref = [t.clone() for t in all_of()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        late = all_of()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(ref, late):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of()
    for turn in range(3):
        for x in xs:
            x.copy_(torch.randn(x.shape, device=dev, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, all_of()):
            assert torch.equal(a, b), turn
