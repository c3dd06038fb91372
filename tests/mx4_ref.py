"""Microscaled 4-bit matrices and the experts' layer in numpy, in 64 bits, from
their definitions; and the bounds that the tests hold the kernels to."""

import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # a rounding's relative error
LEAST = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}  # and the absolute one of subnormals


def blocks(width):
    return -(-width // 32)


def unpack(codes, scales, width):
    """Values of uint8 codes [.., 16 * blocks] and scales [.., blocks]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * LEVELS[c & 7]
    s = scales.astype(np.float64)
    s = np.where(s == 255, np.nan, np.exp2(s - 127))
    return (v * np.repeat(s, 32, -1))[..., :width]


def quantize(x):
    """Codes and scales of x's rows (float64 holding the input's values)."""
    n, width = x.shape
    v = np.zeros((n, blocks(width) * 32))
    v[:, :width] = x
    v = v.reshape(n, -1, 32)
    most = np.abs(v).max(2) if v.shape[1] else np.zeros((n, 0))
    ok = np.isfinite(most)
    _, e = np.frexp(np.where(ok, most, 1.0))
    e = np.where(most > 0, e - 1 - 2, -127)
    e = np.maximum(e, -127)
    a = np.ldexp(np.where(ok[..., None], np.abs(v), 0.0), -e[..., None])
    code = np.zeros(a.shape, np.uint8)
    for i in range(7):  # halfway to the next level: up only if that level's code is even
        half = (LEVELS[i] + LEVELS[i + 1]) / 2
        code[(a > half) | ((a == half) & (i % 2 == 1))] = i + 1
    code |= np.where(np.signbit(v) & ok[..., None], 8, 0).astype(np.uint8)
    code = code.reshape(n, -1, 2)
    return code[..., 0] | (code[..., 1] << 4), np.where(ok, e + 127, 255).astype(np.uint8)


def product_bound(ref, scale, k, kind):
    """What a sum of k exact products in float32 (each of at most k additions off
    by 2^-23 of the sum of magnitudes so far, if the matrix cores truncate),
    rounded once, may be off by."""
    return EPS[kind] * np.abs(ref) * (1 + 2 ** -8) + 1.01 * (k + 1) * 2.0 ** -23 * scale + LEAST[kind]


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def gelu(g):
    from scipy.special import erf

    return 0.5 * g * (1 + erf(g / np.sqrt(2)))


def expert_mlp(x, experts, weights, gate, up, down, act=silu):
    """The layer's result, and a bound of its float32 arithmetic: sums as in
    product_bound, an activation within 2^-20 of itself (and 2^-20 of its argument
    for gelu's cancellation) and of slope at most 1.2, a hidden value held to
    2^-17, and 2^-17 for products of both second parts left out."""
    t, width = x.shape
    hidden = gate.shape[1]
    out, off = np.zeros((t, width)), np.zeros((t, width))
    size = np.zeros((t, width))
    for i in range(t):
        for k in range(experts.shape[1]):
            e = experts[i, k]
            if not 0 <= e < len(gate):
                continue
            g, u = gate[e] @ x[i], up[e] @ x[i]
            dg = (width + 1) * 2.0 ** -23 * (np.abs(gate[e]) @ np.abs(x[i]))
            du = (width + 1) * 2.0 ** -23 * (np.abs(up[e]) @ np.abs(x[i]))
            a, w = act(g), float(weights[i, k])
            da = 1.2 * dg + 2.0 ** -20 * (np.abs(a) + np.abs(g))
            h = w * a * u
            dh = abs(w) * (np.abs(a) * du + np.abs(u) * da + da * du) + 2.0 ** -16 * np.abs(h)
            out[i] += down[e] @ h
            off[i] += np.abs(down[e]) @ dh
            size[i] += np.abs(down[e]) @ (np.abs(h) + dh)
    off += (2.0 ** -17 + (hidden * experts.shape[1] + 17) * 2.0 ** -23) * size
    return out, off
