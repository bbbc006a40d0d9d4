"""Cases of the token-level operators and of the 8-bit layers, in their plain form and as the package's calls.

Four operators, named by a case's ``"op"``:

* ``lookup``  -- rows of an embedding table by token id, times a scale, with a padding id whose rows are zero;
* ``grad``    -- the gradient of that lookup (and of sum-pooled bags of L ids) with respect to the table;
* ``norm``    -- root-mean-square norm of ``x + residual`` rows, rounded to 8-bit integers with one scale for each row;
* ``linear``  -- a layer on 8-bit integers: ``act((x_q w_q^T) * x_scale * w_scale + bias)``.

``run`` computes them with elementary torch operations where ``own`` is false and with the package's kernels where it is
true; both start from the same state.
"""
from __future__ import annotations

import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_EPS = 1e-6


def listed():
    return [
        # the tiny configuration's ids as one token list: latency alone
        dict(name="lookup_64x16", op="lookup", tokens=64, rows=1000, dim=16, type="f32", skew=0.0, pad=False),
        # a batch of long histories over a wide table in bf16, row length not a power of two, with padding
        dict(name="lookup_16383x1000_bf16", op="lookup", tokens=16383, rows=50000, dim=1000, type="bf16", skew=1.05, pad=True),
        # one table of the largest configuration, every id of the batch unpooled
        dict(name="lookup_1310720x128", op="lookup", tokens=65536 * 20, rows=4_000_000, dim=128, type="f32", skew=1.2, pad=False),
        # the gradient of the tiny lookup: latency alone
        dict(name="grad_64x16", op="grad", tokens=64, bag=1, rows=1000, dim=16, type="f32", skew=0.0, pad=False),
        # one table of the 32-table configuration: bags of 16 ids, a dense gradient much larger than what reaches it
        dict(name="grad_bags_32768x64", op="grad", tokens=2048 * 16, bag=16, rows=1_000_000, dim=64, type="f32", skew=1.05, pad=False),
        # the histories' gradient, bf16 in and out: some rows get thousands of tokens, padding is skipped
        dict(name="grad_16383x1000_bf16", op="grad", tokens=16383, bag=1, rows=50000, dim=1000, type="bf16", skew=1.05, pad=True),
        # one table of the largest configuration, unpooled: more gradient bytes come in than go out for hot rows
        dict(name="grad_1310720x128", op="grad", tokens=65536 * 20, bag=1, rows=1_000_000, dim=128, type="f32", skew=1.2, pad=False),
        # one token through a wide layer's norm
        dict(name="norm_1x4096_bf16", op="norm", rows=1, dim=4096, type="bf16", residual=True),
        # a large batch through the same norm
        dict(name="norm_16384x4096_bf16", op="norm", rows=16384, dim=4096, type="bf16", residual=True),
        # one token through a wide layer: bound by reading the weights
        dict(name="linear_1x4096x4096", op="linear", rows=1, inner=4096, cols=4096, type="bf16", act="none", bias=False),
        # the top MLP's first layer at the benchmark batch: 64 dense and 528 interaction columns
        dict(name="linear_2048x592x512", op="linear", rows=2048, inner=592, cols=512, type="f32", act="relu", bias=True),
        # a large batch through wide layers: bound by the tensor cores
        dict(name="linear_8192x8192x8192", op="linear", rows=8192, inner=8192, cols=8192, type="bf16", act="none", bias=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lookup", "grad", "norm", "linear"])
    kind = rng.choice(["f32", "bf16"])
    if op in ("lookup", "grad"):
        dim = _spread(rng, 8, 2048)
        rows = min(_spread(rng, 100, 4_000_000), 250_000_000 // dim)
        tokens = min(_spread(rng, 1, 1_310_720), 160_000_000 // dim)
        case = dict(op=op, tokens=tokens, rows=rows, dim=dim, type=kind, skew=rng.choice([0.0, 1.05, 1.2]), pad=rng.random() < 0.5 and tokens >= 32)
        if op == "grad":
            bag = rng.choice([1, 1, 4, 20])
            case["bag"] = bag
            case["tokens"] = max(1, tokens // bag) * bag
            case["rows"] = min(rows, 120_000_000 // dim)
        return case
    if op == "norm":
        dim = _spread(rng, 16, 16384)
        return dict(op=op, rows=min(_spread(rng, 1, 65536), 60_000_000 // dim), dim=dim, type=kind, residual=rng.random() < 0.7)
    return dict(op=op, rows=_spread(rng, 1, 8192), inner=_spread(rng, 16, 8192), cols=_spread(rng, 1, 8192), type=kind,
                act=rng.choice(["none", "relu", "sigmoid"]), bias=rng.random() < 0.5)


def _ids(case, g):
    """Token ids: even over the rows, or a bounded power law whose frequent rows are scattered over the table."""
    n, rows = case["tokens"], case["rows"]
    if case["skew"] == 0.0:
        return torch.randint(0, rows, (n,), device="cuda", generator=g, dtype=torch.int64).to(torch.int32)
    weight = torch.arange(1, rows + 1, device="cuda", dtype=torch.float64) ** -case["skew"]
    edge = torch.cumsum(weight, 0)
    u = torch.rand(n, device="cuda", dtype=torch.float64, generator=g) * edge[-1]
    rank = torch.searchsorted(edge, u, right=True).clamp_(max=rows - 1)
    place = torch.randperm(rows, device="cuda", generator=g)
    return place[rank].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dev = case["op"], "cuda"
    kind = _TYPES[case["type"]]
    s = dict(case=case, op=op, kind=kind)
    if op in ("lookup", "grad"):
        s["ids"] = _ids(case, g)
        # the padding id is the most frequent one of the list: a batch of short histories
        s["pad"] = int(torch.mode(s["ids"]).values) if case["pad"] else None
        s["scale"] = math.sqrt(case["dim"])
    if op == "lookup":
        s["table"] = torch.empty((case["rows"], case["dim"]), device=dev, dtype=kind).normal_(0, 0.1, generator=g)
    elif op == "grad":
        s["grad"] = torch.empty((case["tokens"] // case["bag"], case["dim"]), device=dev, dtype=kind).normal_(0, 1, generator=g)
    elif op == "norm":
        m, k = case["rows"], case["dim"]
        s["x"] = torch.empty((m, k), device=dev, dtype=kind).normal_(0, 1, generator=g)
        # the running sum of a deep stack: larger than what a layer adds, with rows of different sizes
        size = torch.empty((m, 1), device=dev).uniform_(0.5, 8, generator=g)
        s["residual"] = (torch.empty((m, k), device=dev).normal_(0, 1, generator=g) * size).to(kind) if case["residual"] else None
        s["weight"] = torch.empty(k, device=dev).normal_(1, 0.2, generator=g)
    else:
        m, k, n = case["rows"], case["inner"], case["cols"]
        pitch = (k + 15) // 16 * 16  # rows of 8-bit integers start on 16 bytes
        for name, r in (("x", m), ("w", n)):
            v = torch.empty((r, k), device=dev).normal_(0, 1, generator=g)
            top = v.abs().amax(1)
            buf = torch.zeros((r, pitch), device=dev, dtype=torch.int8)
            buf[:, :k] = torch.round(v * (127.0 / top)[:, None]).to(torch.int8)
            s[name + "_q"] = buf[:, :k]
            s[name + "_scale"] = top / 127.0 * (1.0 if name == "x" else k ** -0.5)
        s["bias"] = torch.empty(n, device=dev).normal_(0, 0.5, generator=g) if case["bias"] else None
        s["act"] = case["act"]
    return s


def _plain(s):
    op, kind, case = s["op"], s["kind"], s["case"]
    if op == "lookup":
        y = s["table"][s["ids"].long()].float() * s["scale"]
        if s["pad"] is not None:
            y = torch.where((s["ids"] == s["pad"])[:, None], torch.zeros((), device=y.device), y)
        return y.to(kind)
    if op == "grad":
        rows = s["grad"].float() * s["scale"]
        if case["bag"] > 1:
            rows = rows.repeat_interleave(case["bag"], 0)
        if s["pad"] is not None:
            rows = torch.where((s["ids"] == s["pad"])[:, None], torch.zeros((), device=rows.device), rows)
        out = torch.zeros((case["rows"], case["dim"]), device=rows.device)
        return out.index_add_(0, s["ids"].long(), rows).to(kind)
    if op == "norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        y = h * s["weight"]
        top = y.abs().amax(1)
        q = torch.round(y * torch.where(top > 0, 127.0 / top, torch.zeros_like(top))[:, None])
        scale = torch.rsqrt(h.square().mean(1) + _EPS) * top / 127.0
        values = (q * scale[:, None]).to(torch.bfloat16)
        return (values, scale) if s["residual"] is None else (values, scale, h.to(kind))
    y = (s["x_q"].float() @ s["w_q"].float().T) * s["x_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["act"] == "relu":
        y = torch.clamp(y, min=0.0)
    elif s["act"] == "sigmoid":
        y = 1.0 / (1.0 + torch.exp(-y))
    return y.to(kind)


def run(state):
    if not own:
        return _plain(state)
    s = state
    if s["op"] == "lookup":
        from dlrm_embedding_bag_b200 import tokens
        return tokens.embedding_lookup(s["table"], s["ids"], scale=s["scale"], padding_idx=s["pad"])
    if s["op"] == "grad":
        from dlrm_embedding_bag_b200 import tokens
        return tokens.embedding_grad(s["grad"], s["ids"], s["case"]["rows"], L=s["case"]["bag"], scale=s["scale"],
                                     padding_idx=s["pad"], dtype=s["kind"])
    from dlrm_embedding_bag_b200 import int8
    if s["op"] == "norm":
        q, scale, h = int8.rms_norm_int8(s["x"], s["weight"], residual=s["residual"], eps=_EPS)
        # the 8-bit integers as the values that they stand for
        values = int8.dequantize_rows(q, scale, dtype=torch.bfloat16)
        return (values, scale) if h is None else (values, scale, h)
    return int8.linear_int8(s["x_q"], s["x_scale"], s["w_q"], s["w_scale"], s["bias"], s["act"], out_dtype=s["kind"])


def work(case):
    size = 4 if case["type"] == "f32" else 2
    op = case["op"]
    if op == "lookup":
        t, d = case["tokens"], case["dim"]
        return dict(bytes=4 * t + size * d * (min(t, case["rows"]) + t), flops=t * d)
    if op == "grad":
        t, d = case["tokens"], case["dim"]
        return dict(bytes=4 * t + size * d * (t // case["bag"] + case["rows"]), flops=2 * t * d)
    if op == "norm":
        m, k = case["rows"], case["dim"]
        streams = 3 if case["residual"] else 1  # x, residual, and the sum that goes back
        return dict(bytes=m * k * (size * streams + 1) + 4 * m + 4 * k, flops=8 * m * k)
    m, k, n = case["rows"], case["inner"], case["cols"]
    return dict(bytes=m * k + n * k + size * m * n + 4 * (m + n) + (4 * n if case["bias"] else 0), flops=2 * m * k * n)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        live = torch.ones(case["tokens"], device="cuda", dtype=torch.float64)
        if s["pad"] is not None:
            live[s["ids"] == s["pad"]] = 0.0
        picked = torch.index_select(s["table"], 0, s["ids"]).double()
        return picked.mul_((live * s["scale"])[:, None])
    if op == "grad":
        # running sums over the tokens in the order of their ids; a row's gradient is the difference at its borders
        order = torch.argsort(s["ids"], stable=True)
        near = s["ids"][order].long()
        edge = torch.searchsorted(near, torch.arange(case["rows"] + 1, device="cuda"))
        out = torch.empty((case["rows"], case["dim"]), device="cuda", dtype=torch.float64)
        for c in range(0, case["dim"], 32):
            part = s["grad"][:, c:c + 32].double()[order // case["bag"]]
            total = torch.zeros((case["tokens"] + 1, part.shape[1]), device="cuda", dtype=torch.float64)
            torch.cumsum(part, 0, out=total[1:])
            out[:, c:c + 32] = (total[edge[1:]] - total[edge[:-1]]) * s["scale"]
        if s["pad"] is not None:
            out[s["pad"]] = 0.0
        # rows that no token names have nothing left over from the running sums
        out[edge[1:] == edge[:-1]] = 0.0
        return out
    if op == "norm":
        outs = []
        step = max(1, (1 << 24) // case["dim"])
        for m in range(0, case["rows"], step):
            h = s["x"][m:m + step].double()
            if s["residual"] is not None:
                h = h + s["residual"][m:m + step].double()
            y = h / torch.sqrt(torch.linalg.vecdot(h, h)[:, None] / case["dim"] + _EPS) * s["weight"].double()
            scale = torch.linalg.vector_norm(y, math.inf, dim=1) / 127.0
            levels = torch.round(y / scale.clamp(min=1e-300)[:, None])
            outs.append((levels * scale[:, None], scale, h))
        values, scale, h = (torch.cat(v) for v in zip(*outs))
        return (values, scale) if s["residual"] is None else (values, scale, h)
    y = torch.einsum("mk,nk->mn", s["x_q"].double(), s["w_q"].double())
    y = torch.einsum("mn,m,n->mn", y, s["x_scale"].double(), s["w_scale"].double())
    if s["bias"] is not None:
        y += s["bias"].double()
    if s["act"] == "relu":
        y = torch.maximum(y, torch.zeros_like(y))
    elif s["act"] == "sigmoid":
        y = torch.reciprocal(torch.exp(-y) + 1.0)
    return y
