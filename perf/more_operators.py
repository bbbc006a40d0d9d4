"""Cases of the optimiser step and of the 4-bit layers, in their plain form and as the package's calls.

Three operators, named by a case's ``"op"``:

* ``adamw``    -- one AdamW step over many tensors at once, moments in 32 or in 8 bits, weights in f32 or bf16 (with or without
  f32 masters);
* ``quantize`` -- rows rounded to 4-bit floating point (e2m1) with one power of two for each 32 elements, returned as the values
  that they stand for;
* ``linear``   -- a layer on such numbers: ``act(x w^T + bias)``.

``run`` computes them with elementary torch operations where ``own`` is false and with the package's kernels where it is true;
both start from the same state.

Moments live in one flat buffer, a tensor's elements from a multiple of 256 on. In 8 bits the first moment is e4m3 and the root
of the second has four bits of exponent and four of mantissa, each with one f32 scale for 256 elements; they are rounded up or
down at random, in proportion, with bits that the seed, the step and the element's place give. So are bf16 weights without
masters. 4-bit matrices are packed two to a byte, the even column low; scales are bytes in tiles of 128 rows x 4 blocks.
"""
from __future__ import annotations

import math
import random

import torch
import torch.nn.functional as F

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_BETAS, _EPS, _LR, _DECAY, _SEED = (0.9, 0.999), 1e-8, 1e-3, 0.01, 7
_STEPS = 1000  # taken before the measured one
# the layers of the forward for 13 dense features, 32 tables and 64 columns
_MLP = [(512, 13), (256, 512), (64, 256), (512, 592), (256, 512), (1, 256)]


def listed():
    return [
        # both MLPs of the forward in f32: twelve small tensors, latency alone
        dict(name="adamw_mlp_f32", op="adamw", kind="mlp", type="f32", bits=32, master=False, clip=False),
        # the same layers as the package holds them (bf16 weights, f32 biases), with masters and 8-bit moments
        dict(name="adamw_mlp_mixed_8bit", op="adamw", kind="mlp", type="mixed", bits=8, master=True, clip=True),
        # sixty tensors of any length from one element up, bf16 without masters, 8-bit moments, clipped gradients
        dict(name="adamw_ragged_bf16_8bit", op="adamw", kind="ragged", count=60, most=4_000_000, mix=5, type="bf16", bits=8, master=False, clip=True),
        # one table of the 32-table configuration: most rows have no gradient in a batch
        dict(name="adamw_table_f32", op="adamw", kind="tables", count=1, rows=1_000_000, dim=64, type="f32", bits=32, master=False, clip=False),
        # four such tables, their moments in a quarter of the room
        dict(name="adamw_tables_8bit", op="adamw", kind="tables", count=4, rows=1_000_000, dim=64, type="f32", bits=8, master=False, clip=False),
        # one token in front of a wide layer: latency alone
        dict(name="quantize_1x4096_bf16", op="quantize", rows=1, dim=4096, type="bf16"),
        # the top MLP's input at the benchmark batch: 64 dense and 528 interaction columns
        dict(name="quantize_2048x592_f32", op="quantize", rows=2048, dim=592, type="f32"),
        # a large batch of wide rows
        dict(name="quantize_16384x4096_bf16", op="quantize", rows=16384, dim=4096, type="bf16"),
        # one token through a wide layer: bound by reading the weights
        dict(name="linear_1x4096x4096", op="linear", rows=1, inner=4096, cols=4096, type="bf16", act="none", bias=False),
        # the top MLP's first layer at the benchmark batch
        dict(name="linear_2048x592x512", op="linear", rows=2048, inner=592, cols=512, type="f32", act="relu", bias=True),
        # odd sizes: no side a multiple of a tile or of a block
        dict(name="linear_777x1001x1234", op="linear", rows=777, inner=1001, cols=1234, type="bf16", act="sigmoid", bias=True),
        # a large batch through wide layers: bound by the tensor cores
        dict(name="linear_8192x8192x8192", op="linear", rows=8192, inner=8192, cols=8192, type="bf16", act="none", bias=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "quantize", "linear", "linear"])
    if op == "adamw":
        kind = rng.choice(["ragged", "ragged", "tables"])
        case = dict(op=op, kind=kind, type=rng.choice(["f32", "bf16", "mixed"]), bits=rng.choice([8, 32]), clip=rng.random() < 0.5)
        case["master"] = case["type"] != "f32" and rng.random() < 0.5
        if kind == "ragged":
            case.update(count=_spread(rng, 1, 60), most=_spread(rng, 100, 3_000_000), mix=rng.randrange(1 << 20))
        else:
            dim, rows = _spread(rng, 8, 512), _spread(rng, 100, 1_000_000)
            rows = min(rows, 64_000_000 // dim)
            case.update(count=rng.choice([1, 2]), rows=rows, dim=dim)
        return case
    kind = rng.choice(["f32", "bf16"])
    if op == "quantize":
        dim = _spread(rng, 16, 16384)
        return dict(op=op, rows=min(_spread(rng, 1, 65536), 60_000_000 // dim), dim=dim, type=kind)
    return dict(op=op, rows=_spread(rng, 1, 8192), inner=_spread(rng, 16, 8192), cols=_spread(rng, 1, 8192), type=kind,
                act=rng.choice(["none", "relu", "sigmoid"]), bias=rng.random() < 0.5)


# ---- AdamW: shapes, and the moments' 8-bit forms -----------------------------------------------------------------------------


def _shapes(case):
    if case["kind"] == "mlp":
        return [s for n, k in _MLP for s in ((n, k), (n,))]
    if case["kind"] == "tables":
        return [(case["rows"], case["dim"])] * case["count"]
    r = random.Random(case["mix"])
    sizes = [_spread(r, 1, case["most"]) for _ in range(case["count"])]
    # matrices and vectors
    return [(n // 8, 8) if n >= 4096 and r.random() < 0.5 else (n,) for n in sizes]


def _dtype(case, shape):
    if case["type"] == "mixed":
        return torch.bfloat16 if len(shape) == 2 else torch.float32
    return _TYPES[case["type"]]


def _room(n):
    return (n + 255) // 256 * 256


def _mixed(x):
    """32 bits that look random from 32 that do not (held in 64-bit integers)."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random(block0, n, step, device):
    """Random 32-bit words of the n elements (a multiple of 256) from block block0 on, at that step (a tensor)."""
    key = _mixed(_mixed(torch.full((), _SEED + 0x9E3779B9, dtype=torch.int64, device=device)) ^ step)
    block = torch.arange(block0, block0 + n // 256, device=device, dtype=torch.int64)
    word = _mixed(key ^ block)[:, None] + torch.arange(256, device=device, dtype=torch.int64) * 0x9E3779B9
    return _mixed(word & 0xFFFFFFFF).reshape(-1)


def _codes(x, frac, least, top, chance=None):
    """x >= 0 as a number of `frac` mantissa bits whose least normal power is 2^least, rounded by 16 random bits or to nearest."""
    small = x < 2.0 ** least
    bits = torch.where(small, x + 2.0 ** least, x).contiguous().view(torch.int32).to(torch.int64)
    bits = bits + (chance << (7 - frac) if chance is not None else 1 << (22 - frac))
    code = (bits >> (23 - frac)) - (torch.where(small, 127 + least, 126 + least) << frac)
    return code.clamp(0, top)


def _first_values(codes, scale):
    return (codes.float().view(-1, 256) * scale[:, None]).view(-1)


def _root_values(codes, scale):
    c = codes.to(torch.int64)
    e, f = c >> 4, (c & 15).float() / 16
    r = torch.where(e > 0, (1 + f) * torch.exp2((e - 15).float()), f * 2.0 ** -14)
    return (r.view(-1, 256) * scale[:, None]).view(-1)


def _first_codes(m, chance=None):
    top = m.view(-1, 256).abs().amax(1)
    scale = top / 448.0
    live = scale >= 2.0 ** -126
    inv = torch.where(live, 448.0 / top, torch.zeros_like(top))
    c = _codes((m.view(-1, 256) * inv[:, None]).abs(), 3, -6, 126, chance if chance is None else chance.view(-1, 256))
    c = torch.where((m.view(-1, 256) < 0) & (c > 0), c | 128, c)
    return c.to(torch.uint8).view(-1).view(torch.float8_e4m3fn), torch.where(live, scale, torch.zeros_like(scale))


def _root_codes(r, chance=None):
    top = r.view(-1, 256).amax(1)
    scale = top / 1.9375
    inv = torch.where(top > 0, 1.9375 / top, torch.zeros_like(top))
    c = _codes(r.view(-1, 256) * inv[:, None], 4, -14, 255, chance if chance is None else chance.view(-1, 256))
    c = torch.where((r.view(-1, 256) > 0) & (c == 0), 1, c)  # what is not zero stays so
    return c.to(torch.uint8).view(-1), scale


def _plain_adamw(s):
    case, st = s["case"], s["moments"]
    dev = st["m"].device
    st["step"][:1] += 1
    t = st["step"][0].double()
    b1, b2 = _BETAS
    alpha = (_LR / (1 - b1 ** t)).float()
    root = (1 / torch.sqrt(1 - b2 ** t)).float()
    at = 0
    for p, grad in zip(s["params"], s["grads"]):
        n = p.numel()
        end = at + _room(n)
        g = grad.float().view(-1)
        if s["coef"] is not None:
            g = g * s["coef"]
        g = F.pad(g, (0, end - at - n))
        if case["bits"] == 8:
            blocks = slice(at // 256, end // 256)
            m = _first_values(st["m"][at:end], st["m_scale"][blocks])
            r = _root_values(st["v"][at:end], st["v_scale"][blocks])
            v = r * r
        else:
            m, v = st["m"][at:end], st["v"][at:end]
        m = m * b1 + g * (1 - b1)
        v = v * b2 + g * g * (1 - b2)
        r = torch.sqrt(v)
        whole = st["master"] is not None and p.dtype == torch.bfloat16
        old = st["master"][at:at + n] if whole else p.float().view(-1)
        new = old * (1 - _LR * _DECAY) - alpha * (m / (r * root + _EPS))[:n]
        word = _random(at // 256, end - at, st["step"][0].to(torch.int64), dev) if case["bits"] == 8 or p.dtype == torch.bfloat16 else None
        if whole:
            st["master"][at:at + n] = new
            p.copy_(new.to(p.dtype).view(p.shape))
        elif p.dtype == torch.bfloat16:
            chance = (((word * 0x3C6EF373) & 0xFFFFFFFF) >> 16)[:n]
            bits = (new.view(torch.int32).to(torch.int64) + chance) & ~0xFFFF
            p.copy_(bits.to(torch.int32).view(torch.float32).to(p.dtype).view(p.shape))
        else:
            p.copy_(new.view(p.shape))
        if case["bits"] == 8:
            st["m"][at:end], st["m_scale"][blocks] = _first_codes(m, word & 0xFFFF)
            st["v"][at:end], st["v_scale"][blocks] = _root_codes(r, word >> 16)
        else:
            st["m"][at:end], st["v"][at:end] = m, v
        at = end
    if case["bits"] == 32:
        return [*s["params"], st["m"], st["v"]]
    r = _root_values(st["v"], st["v_scale"])
    return [*s["params"], _first_values(st["m"], st["m_scale"]).bfloat16(), (r * r).bfloat16()]


# ---- 4-bit numbers -----------------------------------------------------------------------------------------------------------

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _blocks(x):
    """(blocks of 32 columns, their scales' bytes): the least power of two that brings a block's largest element to 7 or less."""
    m, k = x.shape
    b = F.pad(x.float(), (0, -k % 32)).view(m, -1, 32)
    bits = b.abs().amax(2).view(torch.int32).to(torch.int64)
    return b, (((bits + 0x1FFFFF) >> 23) - 2).clamp(0, 254)


def _levels(b, byte):
    """Codes 0..15 (sign in bit 3), nearest with ties to the even code."""
    y = b.double() * torch.exp2(127.0 - byte.double())[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=b.device, dtype=torch.float64)
    a = y.abs()
    up, down = torch.bucketize(a, edges, right=True), torch.bucketize(a, edges)
    code = torch.where(up % 2 == 0, up, down)
    return code + 8 * (y < 0)


def _values(code, byte):
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], device=code.device, dtype=torch.float64)
    return (table[code] * torch.exp2(byte.double() - 127.0)[..., None]).flatten(1)


def _pack(code, k):
    """Codes of whole blocks as rows of bytes whose pitch is a multiple of 16; the columns of k."""
    c = code.flatten(1).to(torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4))[:, :(k + 1) // 2]


def _tiles(byte):
    """Scales (rows, blocks) as tiles of 128 rows x 4 blocks: (row tiles, block tiles, 512), zero past the matrix."""
    m, n = byte.shape
    t = F.pad(byte, (0, -n % 4, 0, -m % 128)).to(torch.uint8)
    t = t.view(t.shape[0] // 128, 4, 32, t.shape[1] // 4, 4)
    return t.permute(0, 3, 2, 1, 4).contiguous().flatten(2)


def _unpacked(q, tiles):
    """The f32 values of a packed matrix, whole blocks."""
    code = torch.stack((q & 15, q >> 4), 2).flatten(1).to(torch.int64)
    code = F.pad(code, (0, -code.shape[1] % 32))
    rt, kt = tiles.shape[:2]
    byte = tiles.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)
    byte = byte[:code.shape[0], :code.shape[1] // 32].to(torch.int64)
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], device=q.device)
    return (table[code].view(code.shape[0], -1, 32) * torch.exp2(byte.double() - 127.0).float()[..., None]).flatten(1)


def _packed_normal(rows, k, spread, g):
    """A packed matrix of normal values whose rows differ in size, in a buffer of whole 16-byte rows."""
    v = torch.empty((rows, k), device="cuda").normal_(0, 1, generator=g)
    v *= torch.empty((rows, 1), device="cuda").uniform_(0.5 * spread, 2 * spread, generator=g)
    step = max(1, (1 << 24) // k)
    q = torch.zeros((rows, ((k + 1) // 2 + 15) // 16 * 16), device="cuda", dtype=torch.uint8)
    bytes_ = []
    for at in range(0, rows, step):
        b, byte = _blocks(v[at:at + step])
        q[at:at + step, :(k + 1) // 2] = _pack(_levels(b, byte), k)
        bytes_.append(byte)
    return q[:, :(k + 1) // 2], _tiles(torch.cat(bytes_))


def _plain_linear(s):
    y = _unpacked(s["x_q"], s["x_scale"]) @ _unpacked(s["w_q"], s["w_scale"]).T
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["act"] == "relu":
        y = torch.clamp(y, min=0.0)
    elif s["act"] == "sigmoid":
        y = 1.0 / (1.0 + torch.exp(-y))
    return y.to(s["kind"])


# ---- the cases ---------------------------------------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dev = case["op"], "cuda"
    s = dict(case=case, op=op)
    if op == "adamw":
        shapes = _shapes(case)
        s["params"], s["grads"], ms, rs = [], [], [], []
        for shape in shapes:
            kind = _dtype(case, shape)
            fan = shape[-1] if len(shape) == 2 else 1000
            size = torch.empty((), device=dev).uniform_(1e-4, 1e-2, generator=g)
            # a table's rows that the batch names, and those that earlier ones named
            now, ever = ((torch.rand((shape[0], 1), device=dev, generator=g) < q for q in (0.03, 0.3)) if case["kind"] == "tables"
                         else (torch.ones((), device=dev, dtype=torch.bool),) * 2)
            s["params"].append(torch.empty(shape, device=dev).normal_(0, fan ** -0.5, generator=g).to(kind))
            s["grads"].append((torch.empty(shape, device=dev).normal_(0, 1, generator=g) * size * now).to(kind))
            m = torch.empty(shape, device=dev).normal_(0, 0.3, generator=g) * size * ever
            r = torch.empty(shape, device=dev).normal_(0, 0.5, generator=g).exp_() * size * ever
            pad = (0, _room(m.numel()) - m.numel())
            ms.append(F.pad(m.view(-1), pad))
            rs.append(F.pad(r.view(-1), pad))
        m, r = torch.cat(ms), torch.cat(rs)
        st = dict(m=m, v=r * r, m_scale=None, v_scale=None, master=None)
        if case["bits"] == 8:
            st["m"], st["m_scale"] = _first_codes(m)
            st["v"], st["v_scale"] = _root_codes(r)
        if case["master"]:
            st["master"] = torch.cat([F.pad(p.float().view(-1), (0, _room(p.numel()) - p.numel())) for p in s["params"]])
        # the count of steps; the second word is the step's own
        st["step"] = torch.tensor([_STEPS, 0], device=dev, dtype=torch.int32)
        s["moments"] = st
        s["coef"] = torch.empty(1, device=dev).uniform_(0.3, 0.9, generator=g) if case["clip"] else None
        return s
    kind = s["kind"] = _TYPES[case["type"]]
    if op == "quantize":
        # activations of rows of different size
        x = torch.empty((case["rows"], case["dim"]), device=dev).normal_(0, 1, generator=g)
        s["x"] = (x * torch.empty((case["rows"], 1), device=dev).uniform_(0.1, 8, generator=g)).to(kind)
        return s
    s["x_q"], s["x_scale"] = _packed_normal(case["rows"], case["inner"], 1.0, g)
    s["w_q"], s["w_scale"] = _packed_normal(case["cols"], case["inner"], case["inner"] ** -0.5, g)
    s["bias"] = torch.empty(case["cols"], device=dev).normal_(0, 0.5, generator=g) if case["bias"] else None
    s["act"] = case["act"]
    return s


def run(state):
    s = state
    if s["op"] == "adamw":
        if not own:
            return _plain_adamw(s)
        from dlrm_embedding_bag_b200 import optim
        st = optim.AdamWState(**s["moments"])
        optim.adamw_step(s["params"], s["grads"], st, lr=_LR, betas=_BETAS, eps=_EPS, weight_decay=_DECAY, grad_scale=s["coef"], seed=_SEED)
        if s["case"]["bits"] == 32:
            return [*s["params"], st.m, st.v]
        # the moments as the values that they stand for
        return [*s["params"], *optim.adamw_moments(st, dtype=torch.bfloat16)]
    if s["op"] == "quantize":
        if not own:
            b, byte = _blocks(s["x"])
            return _values(_levels(b, byte), byte)[:, :s["case"]["dim"]].bfloat16()
        from dlrm_embedding_bag_b200 import fp4
        q, scale = fp4.quantize_rows(s["x"])
        # the 4-bit numbers as the values that they stand for
        return fp4.dequantize_rows(q, scale, s["case"]["dim"], dtype=torch.bfloat16)
    if not own:
        return _plain_linear(s)
    from dlrm_embedding_bag_b200 import fp4
    return fp4.linear_fp4(s["x_q"], s["x_scale"], s["w_q"], s["w_scale"], s["bias"], s["act"], out_dtype=s["kind"])


def work(case):
    if case["op"] == "adamw":
        total = flops = 0
        for shape in _shapes(case):
            n, size = math.prod(shape), 4 if _dtype(case, shape) == torch.float32 else 2
            # weight in and out, gradient in, moments in and out
            each = 3 * size + (4 if case["bits"] == 8 else 16)
            if case["bits"] == 8:
                each += 2 + 4  # the moments written out as values
            if case["master"] and size == 2:
                each += 8 - size  # the master in and out; the weight is written only
            total, flops = total + n * each, flops + 14 * n
        return dict(bytes=total, flops=flops)
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "quantize":
        m, k = case["rows"], case["dim"]
        packed = m * ((k + 1) // 2 + (k + 31) // 32)
        return dict(bytes=m * k * (size + 2) + 2 * packed, flops=4 * m * k)
    m, k, n = case["rows"], case["inner"], case["cols"]
    return dict(bytes=(m + n) * ((k + 1) // 2 + (k + 31) // 32) + size * m * n + (4 * n if case["bias"] else 0), flops=2 * m * k * n)


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------------------


def _exact_8bit(x, frac, least, top, chance):
    """Blocks of 256 values >= 0 scaled to `top` and brought down to a grid of `frac` mantissa bits, one step up by chance of the part that
    is left over; the scaled-back values."""
    peak = x.amax(1, keepdim=True)
    unit = torch.where(peak > 0, peak / top, torch.ones_like(peak))
    y = x / unit
    step = torch.exp2((torch.frexp(y.clamp(min=2.0 ** least))[1] - 1 - frac).double())
    low = torch.floor(y / step)
    up = (y / step - low) + chance / 65536.0 >= 1.0
    return ((low + up) * step).clamp(max=top), unit, step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        outs = []
        at = max(1, (1 << 23) // case["dim"])
        grid = torch.tensor([-6, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float64)
        # whether a level's code is even: 6, 4, 3, 2, 1.5, 1, 0.5, 0 have codes 7 .. 0
        even = torch.tensor([0, 1, 0, 1, 0, 1, 0, 1, 0, 1, 0, 1, 0, 1, 0], device="cuda", dtype=torch.bool)
        for r in range(0, case["rows"], at):
            x = s["x"][r:r + at].double()
            wide = torch.zeros((x.shape[0], -(-case["dim"] // 32) * 32), device="cuda", dtype=torch.float64)
            wide[:, :case["dim"]] = x
            wide = wide.reshape(x.shape[0], -1, 32)
            peak = torch.linalg.vector_norm(wide, math.inf, dim=2, keepdim=True)
            part, power = torch.frexp(peak)
            unit = torch.exp2((power - 3 + (part > 0.875)).double())
            y = wide / unit
            above = torch.searchsorted(grid, y.reshape(-1)).clamp(1, 14)
            lo, hi = grid[above - 1], grid[above]
            y1 = y.reshape(-1)
            near_hi = (hi - y1 < y1 - lo) | ((hi - y1 == y1 - lo) & even[above])
            v = torch.where(near_hi, hi, lo).reshape(y.shape) * unit
            outs.append(v.reshape(x.shape[0], -1)[:, :case["dim"]])
        return torch.cat(outs)
    if op == "linear":
        def values(q, tiles):
            rows, size = q.shape
            rank = torch.arange(size * 2, device="cuda")
            nibble = (q.long()[:, rank // 2] >> (4 * (rank % 2))) & 15
            e, f = (nibble >> 1) & 3, nibble & 1
            v = torch.where(e > 0, (1.0 + 0.5 * f.double()) * torch.exp2((e - 1).double()), 0.5 * f.double())
            v = torch.where(nibble >= 8, -v, v)
            row = torch.arange(rows, device="cuda")[:, None]
            block = (rank // 32)[None]
            byte = tiles[row // 128, block // 4, row % 32 * 16 + row % 128 // 32 * 4 + block % 4]
            return v * torch.exp2(byte.double() - 127.0)
        y = torch.einsum("mk,nk->mn", values(s["x_q"], s["x_scale"]), values(s["w_q"], s["w_scale"]))
        if s["bias"] is not None:
            y += s["bias"].double()
        if s["act"] == "relu":
            y = torch.maximum(y, torch.zeros_like(y))
        elif s["act"] == "sigmoid":
            y = torch.reciprocal(torch.exp(-y) + 1.0)
        return y
    st = s["moments"]
    b1, b2 = _BETAS
    t = _STEPS + 1
    coef = float(s["coef"]) if s["coef"] is not None else 1.0
    params, ms, vs, at = [], [], [], 0
    for p, grad in zip(s["params"], s["grads"]):
        n = p.numel()
        end = at + _room(n)
        g = torch.zeros(end - at, device="cuda", dtype=torch.float64)
        g[:n] = grad.reshape(-1).double() * coef
        if case["bits"] == 8:
            by = slice(at // 256, end // 256)
            m = st["m"][at:end].double().reshape(-1, 256).mul(st["m_scale"][by, None].double()).reshape(-1)
            c = st["v"][at:end].long()
            r = torch.where(c < 16, c.double() / 16, (1 + (c % 16).double() / 16) * torch.exp2((c // 16 - 1).double())) * 2.0 ** -14
            v = r.reshape(-1, 256).mul(st["v_scale"][by, None].double()).reshape(-1).square()
        else:
            m, v = st["m"][at:end].double(), st["v"][at:end].double()
        m = torch.lerp(g, m, b1)
        v = torch.lerp(g.square(), v, b2)
        new = p.reshape(-1).double() * (1 - _LR * _DECAY) - _LR * ((m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + _EPS))[:n]
        if p.dtype == torch.bfloat16 and st["master"] is None:
            # between two bf16 numbers, up by chance
            chance = ((_random(at // 256, end - at, torch.tensor(t, device="cuda"), "cuda")[:n] * 0x3C6EF373) % (1 << 32)) // 65536
            step = torch.exp2((torch.frexp(new)[1] - 8).double())
            low = torch.floor(new.abs() / step)
            new = torch.sign(new) * (low + (new.abs() / step - low + chance.double() / 65536.0 >= 1.0)) * step
        params.append(new.reshape(p.shape))
        if case["bits"] == 8:
            word = _random(at // 256, end - at, torch.tensor(t, device="cuda"), "cuda").reshape(-1, 256)
            y, unit, _ = _exact_8bit(m.abs().reshape(-1, 256), 3, -6, 448.0, (word % 65536).double())
            m = (torch.sign(m).reshape(-1, 256) * y * unit).reshape(-1)
            r = torch.sqrt(v).reshape(-1, 256)
            y, unit, step = _exact_8bit(r, 4, -14, 1.9375, (word // 65536).double())
            v = (torch.where((r > 0) & (y == 0), step, y) * unit).square().reshape(-1)
        ms.append(m)
        vs.append(v)
        at = end
    return [*params, torch.cat(ms), torch.cat(vs)]
