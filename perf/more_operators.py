"""Microscaled 4-bit matrices measured: quantisation and back, products with them and the gradient, and a whole
mixture-of-experts layer for a few tokens over 16-bit or 4-bit weights.

A microscaled 4-bit matrix holds every value as a 4-bit float (sign, two exponent bits, one mantissa bit: 0, 0.5, 1,
1.5, 2, 3, 4, 6), two to a byte, and one power of two for each 32 values of a row.

Each case is one operator at one size. ``run`` computes it in plain torch operations, or, where ``own`` is true,
through the framework's entry points. ``exact`` gives the same from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IDS = {"i32": torch.int32, "i64": torch.int64}


def listed():
    return [
        # the activations of one decoding step of 32 sequences, quantised and back
        dict(name="quantize_step", op="quantize", rows=32, width=4096, transpose=False, type="bf16"),
        # a training step's activations quantised along the tokens, for the weights' gradient, and back
        dict(name="quantize_batch", op="quantize", rows=16384, width=8192, transpose=True, type="bf16"),
        # one token through one layer's 4-bit weights: latency
        dict(name="matmul_token", op="matmul", rows=1, n=4096, width=4096, type="bf16"),
        # a few sequences' tokens, sizes no block divides
        dict(name="matmul_odd", op="matmul", rows=37, n=5003, width=4001, type="f16"),
        # a prompt of 4,096 tokens
        dict(name="matmul_prompt", op="matmul", rows=4096, n=8192, width=8192, type="bf16"),
        # fine-tuning over frozen 4-bit weights: the gradient of the layer's input
        dict(name="matmul_grad_batch", op="matmul_grad", rows=4096, n=8192, width=4096, type="bf16"),
        # the same for a short batch, sizes no block divides
        dict(name="matmul_grad_odd", op="matmul_grad", rows=515, n=1111, width=2049, type="f16"),
        # a decoding step of 64 sequences with its activations in 4 bits too
        dict(name="matmul_both_step", op="matmul_both", rows=64, n=8192, width=4096, type="bf16"),
        # a training step's product with both sides in 4 bits
        dict(name="matmul_both_batch", op="matmul_both", rows=8192, n=8192, width=8192, type="bf16"),
        # one token through the experts' layer, weights in 4 bits
        dict(name="experts_token", op="experts", tokens=1, top_k=8, experts=128, width=4096, hidden=1024, type="bf16",
             weights="mx4", ids="i64", drop=0.0),
        # a decoding step of 64 sequences
        dict(name="experts_step", op="experts", tokens=64, top_k=8, experts=128, width=4096, hidden=1024, type="bf16",
             weights="bf16", ids="i64", drop=0.0),
        # a device that holds three quarters of the experts, sizes no vector divides
        dict(name="experts_odd", op="experts", tokens=13, top_k=6, experts=60, width=1001, hidden=733, type="f16",
             weights="f16", ids="i32", drop=0.25),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def _size(rng, low, high):
    n = _log_int(rng, low, high)
    return n | 1 if rng.random() < 0.35 else max(32, n // 32 * 32)


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul_grad", "matmul_both", "experts"])
    if op == "quantize":
        width = _size(rng, 64, 16384)
        return dict(op=op, rows=_log_int(rng, 1, min(32768, 2 ** 26 // width)), width=width,
                    transpose=rng.random() < 0.5, type=rng.choice(["bf16", "f16", "f32"]))
    if op == "experts":
        kind = rng.choice(["bf16", "f16", "mx4", "mx4"])
        case = dict(op=op, tokens=_log_int(rng, 1, 128), top_k=rng.choice([1, 2, 4, 6, 8]),
                    width=_size(rng, 256, 8192), hidden=_size(rng, 128, 8192),
                    type=kind if kind != "mx4" else rng.choice(["bf16", "f16"]), weights=kind,
                    ids=rng.choice(["i32", "i64"]), drop=rng.choice([0.0, 0.0, 0.25, 0.75]))
        case["experts"] = _log_int(rng, 8, max(8, min(256, 2 ** 28 // (case["width"] * case["hidden"]))))
        return case
    case = dict(op=op, n=_size(rng, 64, 16384), width=_size(rng, 64, 16384), type=rng.choice(["bf16", "f16"]))
    case["rows"] = _log_int(rng, 1, min(8192, 2 ** 36 // (case["n"] * case["width"])))
    return case


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, kind, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(TYPES[kind])


def _activations(rows, width, kind, g):
    """Activations: normal, some columns a good deal larger than the others."""
    scale = torch.exp(torch.randn(width, generator=g, device="cuda"))
    return (torch.randn(rows, width, generator=g, device="cuda") * scale).to(TYPES[kind])


def _blocks(width):
    return (width + 31) // 32


def _packed_normal(n, width, g):
    """A weight matrix of entries of size 1 / sqrt(width) as its 4-bit codes and scales."""
    return _plain_quantize(torch.randn(n, width, generator=g, device="cuda") / math.sqrt(width))


def _packed_experts(experts, n, width, g):
    codes = torch.empty(experts, n, 16 * _blocks(width), dtype=torch.uint8, device="cuda")
    scales = torch.empty(experts, n, _blocks(width), dtype=torch.uint8, device="cuda")
    step = max(1, 2 ** 26 // (n * width))
    for e in range(0, experts, step):
        count = min(step, experts - e)
        c, s = _packed_normal(count * n, width, g)
        codes[e:e + count], scales[e:e + count] = c.view(count, n, -1), s.view(count, n, -1)
    return codes, scales


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    op = case["op"]
    if op == "quantize":
        s["x"] = _activations(case["rows"], case["width"], case["type"], g)
    elif op == "experts":
        tokens, width, hidden = case["tokens"], case["width"], case["hidden"]
        s["x"] = _normal((tokens, width), case["type"], g)
        score = torch.randn(tokens, case["experts"], generator=g, device="cuda")
        top, ids = torch.topk(score, case["top_k"], dim=1)
        weights = torch.exp(top - top[:, :1])
        s["router"] = weights / weights.sum(1, keepdim=True)
        away = torch.rand(ids.shape, generator=g, device="cuda") < case["drop"]
        s["ids"] = torch.where(away, -1, ids).to(IDS[case["ids"]])
        for name, n, k in (("gate", hidden, width), ("up", hidden, width), ("down", width, hidden)):
            if case["weights"] == "mx4":
                s[name] = _packed_experts(case["experts"], n, k, g)
            else:
                s[name] = _normal((case["experts"], n, k), case["weights"], g)
                s[name] *= 1 / math.sqrt(k)
    else:
        s["codes"], s["scales"] = _packed_normal(case["n"], case["width"], g)
        if op == "matmul_grad":
            s["grad_out"] = _normal((case["rows"], case["n"]), case["type"], g)
        else:
            s["x"] = _activations(case["rows"], case["width"], case["type"], g)
    return s


def _power(exponent):
    """2^exponent in float32, for whole numbers from -127 to 127."""
    exponent = exponent.int()
    return torch.where(exponent > -127, (exponent + 127) << 23, 1 << 22).view(torch.float32)


def _plain_quantize(x):
    """Codes [rows, 16 * blocks] (value 2 j of a row in the low half of byte j) and scales [rows, blocks] of the rows'
    blocks of 32: the scale 2^(b - 127) has the largest magnitude's exponent less 2, a value over its scale is rounded
    to the nearest of the eight magnitudes (ties to the even code), those past 6 to 6."""
    rows, width = x.shape
    v = torch.zeros(rows, _blocks(width) * 32, device=x.device)
    v[:, :width] = x
    v = v.view(rows, -1, 32)
    most = v.abs().amax(2)
    exponent = torch.where(most > 0, torch.frexp(most)[1] - 3, -127).clamp(min=-127)
    # over the scale in two steps, each a power of two that float32 holds
    half = -(exponent // 2)
    a = v.abs() * _power(half)[..., None] * _power(-exponent - half)[..., None]
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6)
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code + torch.signbit(v) * 8).to(torch.uint8).view(rows, -1, 2)
    return code[..., 0] | (code[..., 1] << 4), (exponent + 127).to(torch.uint8)


def _plain_values(codes, scales, width):
    """The values of codes and scales in float32."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(*scales.shape, 32)
    v = table[c.int()] * _power(scales.int() - 127)[..., None]
    return v.reshape(*scales.shape[:-1], -1)[..., :width]


def _plain_expert(s, e):
    """The three matrices of expert e (a number, or an index of one element) in float32."""
    out = []
    for name, k in (("gate", s["width"]), ("up", s["width"]), ("down", s["hidden"])):
        pick = (lambda t: t[e]) if isinstance(e, int) else (lambda t: t.index_select(0, e)[0])
        if s["weights"] == "mx4":
            out.append(_plain_values(pick(s[name][0]), pick(s[name][1]), k))
        else:
            out.append(pick(s[name]).float())
    return out


def _plain_mlp(x, gate, up, down):
    g = x @ gate.t()
    return (g / (1 + torch.exp(-g)) * (x @ up.t())) @ down.t()


def _plain_experts(s):
    x, ids, router = s["x"].float(), s["ids"].long(), s["router"]
    out = torch.zeros_like(x)
    live = (ids >= 0) & (ids < s["experts"])
    if ids.numel() <= s["experts"]:
        for t in range(ids.shape[0]):
            for k in range(ids.shape[1]):
                y = _plain_mlp(x[t:t + 1], *_plain_expert(s, torch.where(live, ids, 0)[t, k:k + 1]))
                out[t:t + 1] += torch.where(live[t, k], router[t, k] * y, 0.0)
    else:
        for e in range(s["experts"]):
            here = ids == e
            weight = torch.where(here, router, 0.0).sum(1, keepdim=True)
            out += torch.where(here.any(1, keepdim=True), weight * _plain_mlp(x, *_plain_expert(s, e)), 0.0)
    return out.to(s["x"].dtype)


def run(s):
    op = s["op"]
    if own:
        import sparse_dense_matmul_amd as sdm

        if op == "quantize":
            return sdm.dequantize_mx4(sdm.quantize_mx4(s["x"], transpose=s["transpose"]), s["x"].dtype)
        if op == "experts":
            matrices = [sdm.Mx4(*s[name], k) if s["weights"] == "mx4" else s[name]
                        for name, k in (("gate", s["width"]), ("up", s["width"]), ("down", s["hidden"]))]
            return sdm.expert_mlp(s["x"], s["ids"], s["router"], *matrices)
        w = sdm.Mx4(s["codes"], s["scales"], s["width"])
        if op == "matmul":
            return sdm.matmul_mx4(s["x"], w)
        if op == "matmul_grad":
            return sdm.matmul_mx4_grad(s["grad_out"], w)
        return sdm.matmul_mx4(sdm.quantize_mx4(s["x"]), w, dtype=s["x"].dtype)
    if op == "quantize":
        x = s["x"].float()
        x = x.t() if s["transpose"] else x
        return _plain_values(*_plain_quantize(x), x.shape[1]).to(s["x"].dtype)
    if op == "experts":
        return _plain_experts(s)
    w = _plain_values(s["codes"], s["scales"], s["width"])
    if op == "matmul":
        return (s["x"].float() @ w.t()).to(s["x"].dtype)
    if op == "matmul_grad":
        return (s["grad_out"].float() @ w).to(s["grad_out"].dtype)
    x = _plain_values(*_plain_quantize(s["x"].float()), s["width"])
    return (x @ w.t()).to(s["x"].dtype)


def _packed_bytes(n, width):
    return n * 17 * _blocks(width)


def work(case):
    size = 4 if case["type"] == "f32" else 2
    op, width = case["op"], case["width"]
    if op == "quantize":
        n, k = (width, case["rows"]) if case["transpose"] else (case["rows"], width)
        # both calls: values read, codes written and read again, values written
        return {"bytes": 2 * n * k * size + 2 * _packed_bytes(n, k), "flops": 2 * n * k}
    if op == "experts":
        tokens, hidden, top_k, experts = case["tokens"], case["hidden"], case["top_k"], case["experts"]
        # experts that at least one token is sent to
        share = top_k * (1 - case["drop"]) / experts
        distinct = experts * (1 - (1 - share) ** tokens)
        if case["weights"] == "mx4":
            expert = 2 * _packed_bytes(hidden, width) + _packed_bytes(width, hidden)
        else:
            expert = 3 * 2 * width * hidden
        slots = tokens * top_k
        return {"bytes": distinct * expert + 4 * tokens * width + slots * (4 + (4 if case["ids"] == "i32" else 8)),
                "flops": 6 * slots * (1 - case["drop"]) * width * hidden}
    rows, n = case["rows"], case["n"]
    return {"bytes": _packed_bytes(n, width) + rows * (n + width) * size, "flops": 2 * rows * n * width}


def _exact_values(codes, scales, width):
    """The values from the codes' bits: sign, two bits of exponent, one of mantissa."""
    c = torch.empty(*codes.shape, 2, dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        bits = (codes.int() >> (4 * half)) & 15
        exponent, mantissa = (bits >> 1) & 3, (bits & 1).double()
        size = torch.where(exponent == 0, mantissa / 2,
                           (1 + mantissa / 2) * torch.pow(2.0, (exponent - 1).double()))
        c[..., half] = torch.where(bits >= 8, -size, size)
    c = c.flatten(-2)
    scale = torch.pow(2.0, scales.double() - 127).repeat_interleave(32, dim=-1)
    return (c * scale)[..., :width]


def _exact_rounded(x):
    """The value that quantisation along the rows gives each element, found by the borders between magnitudes."""
    rows, width = x.shape
    x = x.double()
    out = torch.empty_like(x)
    for c in range(0, width, 32):
        part = x[:, c:c + 32]
        most = part.abs().amax(1, keepdim=True)
        _, exponent = np.frexp(most.cpu().numpy())
        exponent = np.where(most.cpu().numpy() > 0, exponent - 3, -127).clip(-127)
        scale = torch.from_numpy(np.ldexp(1.0, exponent)).to(x.device)
        a = part.abs() / scale
        level = ((a > 0.25).double() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + 2 * (a > 2.5) + 2 * (a >= 3.5)
                 + 4 * (a > 5)) / 2
        out[:, c:c + 32] = torch.sign(part) * level * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, width = case["op"], case["width"]
    if op == "quantize":
        return _exact_rounded(s["x"].t().contiguous() if case["transpose"] else s["x"])
    if op == "experts":
        ids = s["ids"].cpu().numpy()
        out = torch.zeros(case["tokens"], width, dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            token, slot = np.nonzero(ids == e)
            if not len(token):
                continue
            at = torch.from_numpy(token).cuda()
            if case["weights"] == "mx4":
                gate, up, down = (_exact_values(s[m][0][e], s[m][1][e], k)
                                  for m, k in (("gate", width), ("up", width), ("down", case["hidden"])))
            else:
                gate, up, down = (s[m][e].double() for m in ("gate", "up", "down"))
            x = s["x"][at].double()
            inner = torch.matmul(x, gate.t())
            hidden = inner * torch.sigmoid(inner) * torch.matmul(x, up.t())
            y = torch.matmul(hidden, down.t()) * s["router"][at, torch.from_numpy(slot).cuda()].double()[:, None]
            out.index_add_(0, at, y)
        return out
    w = _exact_values(s["codes"], s["scales"], width)
    if op == "matmul":
        return torch.matmul(s["x"].double(), w.t())
    if op == "matmul_grad":
        return torch.matmul(s["grad_out"].double(), w)
    return torch.matmul(_exact_rounded(s["x"]), w.t())
