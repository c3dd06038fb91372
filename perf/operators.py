"""The selection products measured: embedding lookup and its gradient, tokens sorted by expert and back with
weights, and the routing's gradients.

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
        # one decoding step of 32 sequences: a handful of rows out of a large table, latency only
        dict(name="embed_step", op="embed", tokens=32, vocab=131072, width=4096, type="bf16", ids="i64", pad=0.0),
        # a prompt of 16,384 tokens
        dict(name="embed_prompt", op="embed", tokens=16384, vocab=131072, width=4096, type="bf16", ids="i64", pad=0.0),
        # a padded batch of a small float32 model with a width no vector divides
        dict(name="embed_odd", op="embed", tokens=5003, vocab=50021, width=1023, type="f32", ids="i32", pad=0.1),
        # the table's gradient in a small fine-tuning step
        dict(name="embed_grad_small", op="embed_grad", tokens=2048, vocab=32000, width=1024, type="f32", ids="i64",
             pad=0.0),
        # the table's gradient in a pre-training step: 65,536 tokens, the common ones thousands of times
        dict(name="embed_grad_batch", op="embed_grad", tokens=65536, vocab=131072, width=4096, type="bf16", ids="i64",
             pad=0.0),
        # the same on a padded batch, sizes no vector divides
        dict(name="embed_grad_odd", op="embed_grad", tokens=12289, vocab=50021, width=1001, type="f16", ids="i32",
             pad=0.2),
        # one decoding step of 64 sequences sorted over 128 experts
        dict(name="dispatch_step", op="dispatch", tokens=64, top_k=8, experts=128, width=4096, type="bf16", ids="i64",
             drop=0.0),
        # a training step's tokens sorted over 128 experts
        dict(name="dispatch_batch", op="dispatch", tokens=16384, top_k=8, experts=128, width=4096, type="bf16",
             ids="i64", drop=0.0),
        # the experts' rows of a decoding step back to its tokens
        dict(name="combine_step", op="combine", tokens=64, top_k=8, experts=128, width=4096, type="bf16", ids="i64",
             drop=0.0),
        # the experts' rows of a training step back to its tokens
        dict(name="combine_batch", op="combine", tokens=16384, top_k=8, experts=128, width=4096, type="bf16",
             ids="i64", drop=0.0),
        # the gradients of both sides of the experts in a training step
        dict(name="route_grad_batch", op="route_grad", tokens=16384, top_k=8, experts=64, width=2048, type="bf16",
             ids="i64", drop=0.0),
        # the same on a device that holds three quarters of the experts, sizes no vector divides
        dict(name="route_grad_odd", op="route_grad", tokens=3001, top_k=6, experts=60, width=1001, type="f32",
             ids="i32", drop=0.25),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def _width(rng, low, high):
    w = _log_int(rng, low, high)
    return w | 1 if rng.random() < 0.35 else max(8, w // 8 * 8)


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "dispatch", "combine", "route_grad"])
    case = dict(op=op, type=rng.choice(["bf16", "bf16", "f16", "f32"]), ids=rng.choice(["i32", "i64"]))
    size = 4 if case["type"] == "f32" else 2
    if op in ("embed", "embed_grad"):
        case["width"] = _width(rng, 64, 8192)
        case["vocab"] = _log_int(rng, 1000, min(131072, 2 ** 30 // (case["width"] * size)))
        most = min(65536 if op == "embed_grad" else 32768, 2 ** 29 // (case["width"] * size))
        case["tokens"] = _log_int(rng, 1, most)
        case["pad"] = rng.choice([0.0, 0.0, 0.1, 0.4])
    else:
        case["width"] = _width(rng, 64, 8192)
        case["top_k"] = rng.choice([1, 2, 4, 6, 8])
        case["experts"] = _log_int(rng, 8, 512)
        row = case["width"] * size * (3 * case["top_k"] + 2 if op == "route_grad" else case["top_k"] + 1)
        case["tokens"] = _log_int(rng, 1, min(32768, 3 * 2 ** 29 // row))
        case["drop"] = rng.choice([0.0, 0.0, 0.25, 0.75])
    return case


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _token_ids(case, g):
    """Token ids with frequencies that fall as 1 / rank, the ranks spread over the table; padding is -1."""
    n, vocab = case["tokens"], case["vocab"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)).long() - 1).clamp(0, vocab - 1)
    step = next(a for a in range(vocab // 2 + 1, 2 * vocab + 2) if math.gcd(a, vocab) == 1)
    ids = rank * step % vocab
    pad = torch.rand(n, generator=g, device="cuda") < case["pad"]
    return torch.where(pad, -1, ids).to(IDS[case["ids"]])


def _distinct(case):
    """The expected number of different ids among a case's tokens."""
    vocab = case["vocab"]
    r = np.arange(vocab, dtype=np.float64)
    p = np.log((r + 2) / (r + 1)) / math.log(vocab + 1)
    return float(np.sum(-np.expm1(case["tokens"] * (1 - case["pad"]) * np.log1p(-np.minimum(p, 1 - 1e-12)))))


def _expert_ids(case, g):
    """Each token's top_k experts by a router's scores (some experts liked more), and their softmax weights; experts
    of other devices are -1."""
    score = torch.randn(case["tokens"], case["experts"], generator=g, device="cuda")
    score = score + 0.5 * torch.randn(case["experts"], generator=g, device="cuda")
    top, ids = torch.topk(score, case["top_k"], dim=1)
    weights = torch.exp(top - top[:, :1])
    weights = weights / weights.sum(1, keepdim=True)
    away = torch.rand(ids.shape, generator=g, device="cuda") < case["drop"]
    return torch.where(away, -1, ids).to(IDS[case["ids"]]), weights


def _normal(shape, case, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(TYPES[case["type"]])


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    width = case["width"]
    if case["op"] in ("embed", "embed_grad"):
        s["ids"] = _token_ids(case, g)
        s["scale"] = math.sqrt(width)
        rows = case["vocab"] if case["op"] == "embed" else case["tokens"]
        # a table's entries are of size 1 / sqrt(width), a gradient's of size 1 / tokens
        s["x"] = _normal((rows, width), case, g)
        s["x"] *= 1 / math.sqrt(width)
        return s
    s["ids"], s["weights"] = _expert_ids(case, g)
    slots = case["tokens"] * case["top_k"]
    if case["op"] == "dispatch":
        s["x"] = _normal((case["tokens"], width), case, g)
        return s
    s["position"] = _plain_route(s["ids"], case["experts"])[1]
    s["rows"] = _normal((slots, width), case, g)
    if case["op"] == "route_grad":
        s["grad_out"] = _normal((case["tokens"], width), case, g)
        s["grad_rows"] = _normal((slots, width), case, g)
    return s


def _plain_embed(table, ids, scale):
    real = (ids >= 0) & (ids < table.shape[0])
    rows = table[torch.where(real, ids, 0).long()].float() * scale
    return torch.where(real[:, None], rows, 0.0).to(table.dtype)


def _plain_embed_grad(grad_out, ids, vocab, scale):
    real = (ids >= 0) & (ids < vocab)
    grad = torch.zeros(vocab + 1, grad_out.shape[1], device=ids.device)
    grad.index_add_(0, torch.where(real, ids, vocab).long(), grad_out.float())
    return (grad[:vocab] * scale).to(grad_out.dtype)


def _plain_route(ids, experts):
    key = ids.reshape(-1).long()
    key = torch.where((key >= 0) & (key < experts), key, experts)
    sorted_key, order = torch.sort(key, stable=True)
    row = torch.arange(key.numel(), device=ids.device)
    position = torch.empty_like(row)
    position[order] = row
    position = torch.where(key < experts, position, -1 - position)  # a dropped slot's row is one of the last
    bounds = torch.arange(experts + 1, device=ids.device)
    offsets = (sorted_key[None, :] < bounds[:, None]).sum(1)
    return order.int(), position.int().reshape(ids.shape), offsets.int()


def _plain_dispatch(x, position):
    live = position.reshape(-1) >= 0
    row = torch.where(live, position.reshape(-1), -1 - position.reshape(-1)).long()
    out = torch.empty(position.numel(), x.shape[1], dtype=x.dtype, device=x.device)
    picked = x[:, None, :].expand(-1, position.shape[1], -1).reshape(out.shape)
    out[row] = torch.where(live[:, None], picked, torch.zeros((), dtype=x.dtype, device=x.device))
    return out


def _plain_combine(rows, position, weights):
    live = position >= 0
    picked = rows[torch.where(live, position, 0).long()].float() * weights[:, :, None]
    return torch.where(live[:, :, None], picked, 0.0).sum(1).to(rows.dtype)


def _plain_route_grad(grad_out, rows, grad_rows, position, weights):
    live = position >= 0
    row = torch.where(live, position, -1 - position).long()
    spread = grad_out.float()[:, None, :]
    to_rows = torch.empty_like(rows)
    to_rows[row] = torch.where(live[:, :, None], spread * weights[:, :, None], 0.0).to(rows.dtype)
    to_weights = torch.where(live, (spread * rows[row].float()).sum(2), 0.0)
    to_x = torch.where(live[:, :, None], grad_rows[row].float(), 0.0).sum(1).to(rows.dtype)
    return to_rows, to_weights, to_x


def run(s):
    op = s["op"]
    if own:
        import sparse_dense_matmul_amd as sdm

        if op == "embed":
            return sdm.embedding(s["x"], s["ids"], scale=s["scale"])
        if op == "embed_grad":
            return sdm.embedding_grad(s["x"], s["ids"], s["vocab"], scale=s["scale"])
        if op == "dispatch":
            order, position, offsets = sdm.route(s["ids"], s["experts"])
            return sdm.dispatch(s["x"], position), order, position, offsets
        if op == "combine":
            return sdm.combine(s["rows"], s["position"], s["weights"])
        to_rows, to_weights = sdm.combine_grad(s["grad_out"], s["rows"], s["position"], s["weights"])
        return to_rows, to_weights, sdm.dispatch_grad(s["grad_rows"], s["position"])
    if op == "embed":
        return _plain_embed(s["x"], s["ids"], s["scale"])
    if op == "embed_grad":
        return _plain_embed_grad(s["x"], s["ids"], s["vocab"], s["scale"])
    if op == "dispatch":
        order, position, offsets = _plain_route(s["ids"], s["experts"])
        return _plain_dispatch(s["x"], position), order, position, offsets
    if op == "combine":
        return _plain_combine(s["rows"], s["position"], s["weights"])
    return _plain_route_grad(s["grad_out"], s["rows"], s["grad_rows"], s["position"], s["weights"])


def work(case):
    size = 4 if case["type"] == "f32" else 2
    id_size = 4 if case["ids"] == "i32" else 8
    row = case["width"] * size
    n = case["tokens"]
    if case["op"] == "embed":
        return {"bytes": n * id_size + _distinct(case) * row + n * row, "flops": n * case["width"]}
    if case["op"] == "embed_grad":
        live = n * (1 - case["pad"])
        return {"bytes": n * id_size + live * row + case["vocab"] * row, "flops": live * case["width"]}
    slots = n * case["top_k"]
    live = slots * (1 - case["drop"])
    if case["op"] == "dispatch":
        return {"bytes": slots * (id_size + 8) + 4 * (case["experts"] + 1) + (n + slots) * row, "flops": slots}
    if case["op"] == "combine":
        return {"bytes": 8 * slots + (live + n) * row, "flops": 2 * live * case["width"]}
    return {"bytes": 12 * slots + (2 * n + 2 * live + slots) * row, "flops": 4 * live * case["width"]}


def exact(case, seed):
    s = prepare(case, seed)
    op, width = case["op"], case["width"]
    ids = s["ids"].cpu().numpy().astype(np.int64)
    if op == "embed":
        table = s["x"].double()
        out = torch.zeros(case["tokens"], width, dtype=torch.float64, device="cuda")
        at = np.flatnonzero((ids >= 0) & (ids < case["vocab"]))
        out[torch.from_numpy(at).cuda()] = s["scale"] * table.index_select(0, torch.from_numpy(ids[at]).cuda())
        return out
    if op == "embed_grad":
        # runs of equal ids as differences of a running sum over the sorted tokens, in blocks of columns
        at = np.flatnonzero((ids >= 0) & (ids < case["vocab"]))
        at = at[np.argsort(ids[at], kind="stable")]
        found, first = np.unique(ids[at], return_index=True)
        ends = torch.from_numpy(np.append(first[1:], len(at))).cuda()
        starts, found = torch.from_numpy(first).cuda(), torch.from_numpy(found).cuda()
        out = torch.zeros(case["vocab"], width, dtype=torch.float64, device="cuda")
        for c in range(0, width, 512):
            part = s["x"][:, c:c + 512].double().index_select(0, torch.from_numpy(at).cuda())
            run_sum = torch.cat([torch.zeros_like(part[:1]), part.cumsum(0)]) if len(at) else None
            if len(at):
                out[found, c:c + 512] = s["scale"] * (run_sum[ends] - run_sum[starts])
        return out
    tokens, top_k = ids.shape
    key = np.where((ids >= 0) & (ids < case["experts"]), ids, case["experts"]).reshape(-1)
    if op == "dispatch":
        order = np.argsort(key, kind="stable")
        position = np.empty(key.size, np.int64)
        position[order] = np.arange(key.size)
        offsets = np.searchsorted(key[order], np.arange(case["experts"] + 1))
        live = int(offsets[-1])
        out = torch.zeros(key.size, width, dtype=torch.float64, device="cuda")
        out[:live] = s["x"].double()[torch.from_numpy(order[:live] // top_k).cuda()]
        position[order[live:]] = -1 - position[order[live:]]
        return out, order, position.reshape(tokens, top_k), offsets
    position = s["position"].long()
    if op == "combine":
        out = torch.zeros(tokens, width, dtype=torch.float64, device="cuda")
        for k in range(top_k):
            at = torch.nonzero(position[:, k] >= 0)[:, 0]
            out[at] += s["weights"][at, k, None].double() * s["rows"][position[at, k]].double()
        return out
    to_rows = torch.zeros(tokens * top_k, width, dtype=torch.float64, device="cuda")
    to_weights = torch.zeros(tokens, top_k, dtype=torch.float64, device="cuda")
    to_x = torch.zeros(tokens, width, dtype=torch.float64, device="cuda")
    for k in range(top_k):
        at = torch.nonzero(position[:, k] >= 0)[:, 0]
        row, grad = position[at, k], s["grad_out"][at].double()
        to_rows[row] = s["weights"][at, k, None].double() * grad
        to_weights[at, k] = (grad * s["rows"][row].double()).sum(1)
        to_x[at] += s["grad_rows"][row].double()
    return to_rows, to_weights, to_x
