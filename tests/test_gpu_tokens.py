"""The embedding lookup and the table's gradient on the GPU, against 64 bits.

Lookups are one rounded product, so their bits are compared. A gradient is a
sum of n terms in f32, in an order of the kernel's own: its error is at most
n * 2^-24 times the sum of the terms' magnitudes (n - 1 additions, the scale),
plus half a step of the output's type, eps / 2.
"""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
IDS = dict(f32=F32, bf16=BF16)


@pytest.fixture(scope="module")
def tokens():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from dlrm_embedding_bag_b200 import tokens as _tokens

    return _tokens


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _matrix(g, rows, cols, dtype, pitch=None, offset=0):
    """(rows, cols) normals inside a buffer of NaNs with the given pitch and start."""
    pitch = cols if pitch is None else pitch
    buf = torch.full((rows * pitch + offset + 16,), float("nan"), device=DEV, dtype=dtype)
    m = buf[offset:offset + rows * pitch].view(rows, pitch)[:, :cols] if rows else \
        torch.empty((0, cols), device=DEV, dtype=dtype)
    m.copy_(torch.empty((rows, cols), device=DEV).normal_(0, 1, generator=g))
    return m, buf


def _ids(seed, T, rows, kind):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        v = rng.integers(0, rows, T)
    elif kind == "one":  # every token the same row
        v = np.full(T, rows // 2)
    elif kind == "skew":  # a power law over scattered rows
        p = np.arange(1, rows + 1) ** -1.2
        v = rng.permutation(rows)[rng.choice(rows, T, p=p / p.sum())]
    elif kind == "ends":  # the first and the last row
        v = np.where(rng.random(T) < 0.5, 0, rows - 1)
    return v.astype(np.int32)


def _same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


LOOKUPS = [  # T, rows, D
    (1, 1, 1), (1, 10, 4), (3, 7, 8), (5, 100, 16), (64, 1000, 16), (33, 50, 24), (1000, 300, 64),
    (257, 90, 100), (129, 33, 129), (77, 40, 1000), (4099, 999, 128), (20, 10, 4100),
    (70000, 50, 12), (500, 90, 18), (500, 90, 34), (500, 90, 130), (300, 90, 515), (301, 90, 2),
]


@pytest.mark.parametrize("T,rows,D", LOOKUPS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
def test_lookup(tokens, T, rows, D, dt, odt):
    g = _gen(T + rows + D)
    table, _ = _matrix(g, rows, D, IDS[dt])
    ids = torch.from_numpy(_ids(T, T, rows, "uniform")).to(DEV)
    pad = int(ids[T // 2])
    out = tokens.embedding_lookup(table, ids, scale=D ** 0.5, padding_idx=pad,
                                  out_dtype=IDS[odt])
    scale = torch.tensor(D ** 0.5, device=DEV)
    ref = table.float()[ids.long()] * scale
    ref[ids == pad] = 0.0
    assert out.dtype == IDS[odt]
    assert _same_bits(out, ref.to(IDS[odt]))


@pytest.mark.parametrize("pitch,offset", [(128, 0), (104, 0), (103, 0), (104, 4), (100, 1),
                                          (102, 0), (102, 2), (102, 1)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_lookup_strides_and_what_is_left_alone(tokens, pitch, offset, dt):
    g = _gen(pitch + offset)
    table, _ = _matrix(g, 60, 100, IDS[dt], pitch, offset)
    ids = torch.from_numpy(_ids(5, 211, 60, "skew")).to(DEV)
    out, buf = _matrix(g, 211, 100, IDS[dt], pitch, offset)
    before = buf.clone()
    got = tokens.embedding_lookup(table, ids, out=out)
    assert got is out
    assert _same_bits(out, table[ids.long()])
    kept = torch.ones_like(buf, dtype=torch.bool)
    kept[offset:offset + 211 * pitch].view(211, pitch)[:, :100] = False
    assert torch.isnan(buf[kept]).all() and torch.isnan(before[kept]).all()


def test_lookup_shapes_of_ids_and_empty_lists(tokens):
    table = torch.arange(24, device=DEV, dtype=F32).view(6, 4)
    ids = torch.tensor([[0, 5, 2], [1, 1, 3]], dtype=torch.int32, device=DEV)
    out = tokens.embedding_lookup(table, ids)
    assert out.shape == (2, 3, 4) and torch.equal(out, table[ids.long()])
    mine = torch.empty((2, 3, 4), device=DEV)
    assert tokens.embedding_lookup(table, ids, out=mine, scale=2.0) is mine
    assert torch.equal(mine, table[ids.long()] * 2)
    none = tokens.embedding_lookup(table, ids[:, :0])
    assert none.shape == (2, 0, 4)


def test_lookup_bad_ids_read_nothing(tokens):
    """Ids outside the table give zero rows and the flag, with or without a status word."""
    table = torch.ones((8, 20), device=DEV)
    ids = torch.tensor([0, 8, -1, 2 ** 31 - 1, -2 ** 31, 7], dtype=torch.int32, device=DEV)
    status = torch.full((1,), 77, dtype=torch.int32, device=DEV)
    out = tokens.embedding_lookup(table, ids, status=status)
    assert out.sum(1).tolist() == [20.0, 0.0, 0.0, 0.0, 0.0, 20.0]
    assert int(status) == 1
    assert torch.equal(tokens.embedding_lookup(table, ids), out)
    tokens.embedding_lookup(table, ids[:1], status=status)
    assert int(status) == 0


def test_lookup_rows_past_32_bit_offsets(tokens):
    """A table of more than 2^31 elements: its last rows are found."""
    rows, D = 70_000, 32768 // 1
    table = torch.empty((rows, D), dtype=BF16, device=DEV)  # 2.3e9 elements
    marks = torch.tensor([0, 65535, 65536, rows - 1], device=DEV)
    table[marks] = torch.arange(1, 5, device=DEV, dtype=BF16)[:, None]
    out = tokens.embedding_lookup(table, marks.to(torch.int32))
    assert (out == torch.arange(1, 5, device=DEV, dtype=BF16)[:, None]).all()


# ---------------------------------------------------------------------- gradient


def _reference(grad, ids, rows, L, scale, pad):
    """(sums, counts, sums of magnitudes) in 64 bits."""
    g = grad.double() * float(np.float32(scale))
    flat = ids.reshape(-1).long()
    live = (flat >= 0) & (flat < rows) & (flat != (-1 if pad is None else pad))
    t = torch.nonzero(live)[:, 0]
    terms, at = g[t // L], flat[t]
    out = torch.zeros((rows, g.shape[1]), dtype=torch.float64, device=DEV)
    mag, cnt = torch.zeros_like(out), torch.zeros(rows, dtype=torch.float64, device=DEV)
    out.index_add_(0, at, terms)
    mag.index_add_(0, at, terms.abs())
    cnt.index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    return out, cnt, mag


def _check_grad(out, grad, ids, rows, L=1, scale=1.0, pad=None, base=None):
    ref, cnt, mag = _reference(grad, ids, rows, L, scale, pad)
    unnamed = cnt == 0
    if base is not None:
        ref, mag, cnt = ref + base.double(), mag + base.double().abs(), cnt + 1
    half = torch.finfo(out.dtype).eps / 2
    tol = (cnt[:, None] + 1) * 2.0 ** -24 * mag * (1 + half) + half * ref.abs()
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), float((err - tol).max())
    if base is None:
        assert (out[unnamed] == 0).all()


GRADS = [  # T, rows, D
    (1, 1, 1), (1, 10, 4), (2, 2, 8), (31, 7, 8), (64, 1000, 16), (100, 3, 20), (1000, 300, 64),
    (1023, 255, 24), (1024, 256, 32), (1025, 257, 12), (4096, 65535, 16), (4097, 65536, 128),
    (777, 40, 1000), (5000, 100000, 36), (333, 50, 129), (150, 20, 4100), (30000, 17, 64),
    (150001, 70001, 4), (170001, 3000, 128), (400007, 900, 100), (31000, 70, 4100),
    (900, 200, 18), (900, 200, 33), (2000, 300, 130), (2000, 300, 131), (300, 90, 515),
    (40000, 300, 258), (511, 64, 64), (512, 40000, 100), (512, 2000000, 4), (513, 64, 64), (300, 9000, 1000),
    (700001, 900000, 4), (1000003, 70, 4), (1600001, 20000, 4),
    (337, 286356, 9), (64, 100000, 18), (20, 1192, 54),
    (8192, 300, 8), (8193, 70000, 8), (20000, 5, 16), (65536, 3000, 8), (65537, 3000, 8),
]


@pytest.mark.parametrize("T,rows,D", GRADS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["uniform", "skew", "one", "ends"])
def test_grad(tokens, T, rows, D, dt, kind):
    g = _gen(T + rows + D)
    grad, _ = _matrix(g, T, D, IDS[dt])
    ids = torch.from_numpy(_ids(T, T, rows, kind)).to(DEV)
    out = tokens.embedding_grad(grad, ids, rows, scale=0.3)
    assert out.dtype == IDS[dt]
    _check_grad(out, grad, ids, rows, scale=0.3)
    assert _same_bits(out, tokens.embedding_grad(grad, ids, rows, scale=0.3))


@pytest.mark.parametrize("T,rows,D", [(400, 30, 64), (513, 40, 16), (8193, 300, 40), (30000, 17, 64),
                                      (65536, 3000, 12), (65537, 64, 130), (150001, 70001, 4),
                                      (170001, 3000, 128), (400007, 900, 100), (31000, 70, 4100),
                                      (40000, 300, 258), (50001, 40, 33), (1000003, 70, 4),
                                      (1310720, 100000, 16), (1600001, 20000, 4)])
@pytest.mark.parametrize("dt,odt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("kind", ["uniform", "skew", "one", "ends"])
def test_grad_of_whole_numbers_is_exact(tokens, T, rows, D, dt, odt, kind):
    """Whole numbers of at most 8: every partial sum is below 2^24 and exact in any order, so
    no part of a long run can be lost, doubled or misplaced unseen. Each token's row is
    another one, and one column counts the tokens."""
    assert 8 * T < 2 ** 24
    g = _gen(T + rows)
    grad = torch.randint(-8, 9, (T, D), device=DEV, generator=g).to(IDS[dt])
    grad[:, D // 2] = 1.0
    ids = torch.from_numpy(_ids(T + 1, T, rows, kind)).to(DEV)
    want = torch.zeros((rows, D), device=DEV, dtype=torch.float64)
    want.index_add_(0, ids.long(), grad.double())
    out = tokens.embedding_grad(grad, ids, rows, dtype=IDS[odt])
    assert torch.equal(out, want.to(IDS[odt]))  # rounded once
    # added to a table of whole numbers, with padding: one step of the sparse update
    pad = int(torch.mode(ids).values) if kind != "one" else None
    table = torch.randint(-100, 101, (rows, D), device=DEV, generator=g).float()
    sums = want.clone()
    if pad is not None:
        sums[pad] = 0.0
    after = (table.double() - 2.0 * sums).float()
    assert 2 * 8 * T + 100 < 2 ** 25  # a sum's double and the table's value: even or small
    small = (2.0 * sums).abs().amax(1) + 100 < 2 ** 24
    tokens.embedding_grad(grad, ids, rows, scale=-2.0, padding_idx=pad, out=table, accumulate=True)
    assert torch.equal(table[small], after[small])


@pytest.mark.parametrize("T", [0, 5, 4000, 70000])
@pytest.mark.parametrize("D,pitch,offset", [(64, 128, 0), (64, 65, 0), (64, 66, 1), (3, 4, 0),
                                            (1, 2, 0), (200, 208, 8), (1000, 1004, 4), (6, 10, 2)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_grad_into_rows_that_lie_apart(tokens, T, D, pitch, offset, dt):
    """Columns of a wider buffer: every row is zeroed or written, every gap is left."""
    g = _gen(T + D)
    rows = 120000 if D * T < 10 ** 6 else 9000
    grad = torch.randint(-8, 9, (T, D), device=DEV, generator=g).to(IDS[dt])
    ids = torch.from_numpy(_ids(T, T, rows, "skew")).to(DEV)
    buf = torch.full((rows * pitch + offset + 16,), 77.0, device=DEV, dtype=IDS[dt])
    out = buf[offset:offset + rows * pitch].view(rows, pitch)[:, :D]
    tokens.embedding_grad(grad, ids, rows, out=out)
    want = torch.zeros((rows, D), device=DEV, dtype=torch.float64)
    want.index_add_(0, ids.long(), grad.double())
    assert torch.equal(out, want.to(IDS[dt]))
    out.fill_(77.0)
    assert (buf == 77.0).all()


@pytest.mark.parametrize("T", [300, 3000, 70000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_past_32_bit_offsets(tokens, T, accumulate):
    """A gradient of more than 2^31 elements (and, of many tokens, from as many): its last
    rows are written, and all that no token names."""
    rows, D = 70_000, 32768  # 2.3e9 elements
    out = torch.empty((rows, D), dtype=BF16, device=DEV)
    out.fill_(3.0 if accumulate else float("nan"))
    grad = torch.ones((T, D), dtype=BF16, device=DEV)
    ids = torch.arange(T, device=DEV, dtype=torch.int32) * 7 % 1000
    ids[-5:] = torch.tensor([65535, 65536, rows - 2, rows - 1, rows - 1], device=DEV)
    grad[-1] = 2.0
    tokens.embedding_grad(grad, ids, rows, out=out, accumulate=accumulate)
    base = 3.0 if accumulate else 0.0
    want = torch.zeros(rows, device=DEV)
    want.index_add_(0, ids.long(), grad[:, 0].float())
    want = (want + base).to(BF16)
    assert float(want[rows - 1]) == base + 3.0
    for c in (0, 1, 4097, D - 1):
        assert torch.equal(out[:, c], want)
    # every element, in slices that leave room
    for r in range(0, rows, 10_000):
        assert bool((out[r:r + 10_000] == want[r:r + 10_000, None]).all())


@pytest.mark.parametrize("dt,odt", [("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,D", [(900, 64), (9000, 60), (500, 7)])
def test_grad_types_and_padding(tokens, T, D, dt, odt):
    g = _gen(T + D)
    grad, _ = _matrix(g, T, D, IDS[dt])
    ids = torch.from_numpy(_ids(T, T, 500, "skew")).to(DEV)
    pad = int(torch.mode(ids).values)
    out = tokens.embedding_grad(grad, ids, 500, padding_idx=pad, dtype=IDS[odt])
    assert out.dtype == IDS[odt]
    _check_grad(out, grad, ids, 500, pad=pad)
    assert (out[pad] == 0).all()


@pytest.mark.parametrize("T,pad_all", [(50, True), (5000, True), (50, False), (5000, False)])
def test_grad_nothing_but_padding_or_bad_ids(tokens, T, pad_all):
    grad = torch.full((T, 16), float("nan"), device=DEV)
    ids = torch.full((T,), 3, dtype=torch.int32, device=DEV)
    if not pad_all:
        ids[::2] = -5
        ids[1::2] = 2 ** 31 - 1
    status = torch.full((1,), 9, dtype=torch.int32, device=DEV)
    out = tokens.embedding_grad(grad, ids, 40, padding_idx=3, status=status)
    assert (out == 0).all()
    assert int(status) == (0 if pad_all else 1)


@pytest.mark.parametrize("T", [60, 6000])
def test_grad_bad_ids_among_good_ones(tokens, T):
    g = _gen(T)
    grad, _ = _matrix(g, T, 32, F32)
    ids = torch.from_numpy(_ids(T, T, 45, "uniform") - 3).to(DEV)  # -3 .. 41
    ids[5] = 2 ** 31 - 1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = tokens.embedding_grad(grad, ids, 40, status=status)
    _check_grad(out, grad, ids, 40)
    assert int(status) == 1


@pytest.mark.parametrize("T", [0, 1, 60, 6000])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
def test_grad_accumulates_into_the_rows_that_tokens_name(tokens, T, odt):
    g = _gen(T + 1)
    grad, _ = _matrix(g, T, 48, F32)
    ids = torch.from_numpy(_ids(T, T, 2000, "skew")).to(DEV)
    table, _ = _matrix(g, 2000, 48, IDS[odt])
    base = table.clone()
    got = tokens.embedding_grad(grad, ids, 2000, scale=-0.1, out=table, accumulate=True)
    assert got is table
    _check_grad(table, grad, ids, 2000, scale=-0.1, base=base)
    named = torch.zeros(2000, dtype=torch.bool, device=DEV)
    named[ids.long()] = True
    assert _same_bits(table[~named], base[~named])


@pytest.mark.parametrize("T", [40, 4400])
@pytest.mark.parametrize("pitch,offset,dt", [(64, 0, "f32"), (41, 0, "f32"), (40, 1, "f32"),
                                             (64, 0, "bf16"), (44, 0, "bf16"), (40, 3, "bf16"),
                                             (42, 0, "f32"), (42, 2, "bf16"), (42, 1, "bf16")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_strides_and_what_is_left_alone(tokens, T, pitch, offset, dt, accumulate):
    g = _gen(pitch)
    grad, _ = _matrix(g, T, 40, IDS[dt], pitch, offset)
    out, buf = _matrix(g, 333, 40, IDS[dt], pitch, offset)
    base = out.clone() if accumulate else None
    ids = torch.from_numpy(_ids(5, T, 333, "skew")).to(DEV)
    tokens.embedding_grad(grad, ids, 333, out=out, accumulate=accumulate)
    _check_grad(out, grad, ids, 333, base=base)
    kept = torch.ones_like(buf, dtype=torch.bool)
    kept[offset:offset + 333 * pitch].view(333, pitch)[:, :40] = False
    assert torch.isnan(buf[kept]).all()


@pytest.mark.parametrize("B,L,N,D,F", [(16, 4, 1000, 16, 2), (300, 32, 5000, 64, 3),
                                       (50, 7, 90, 10, 2)])
def test_grad_of_sum_pooled_bags(tokens, B, L, N, D, F):
    """The gradient of embbag_sum_multi with respect to every table, from the
    pooled gradient as it lies, against the formula and against differences of
    the pooled sums themselves."""
    from dlrm_embedding_bag_b200 import ops

    g = _gen(B)
    idx = torch.from_numpy(np.stack([_ids(k, B * L, N, "skew") for k in range(F)])).to(DEV)
    off = (torch.arange(B, device=DEV, dtype=torch.int32) * L).repeat(F, 1).contiguous()
    dpooled = torch.empty((B, F, D), device=DEV).normal_(0, 1, generator=g)
    # whole-numbered tables: pooled sums and their differences are exact
    tables = [torch.randint(-8, 9, (N, D), device=DEV, generator=g).float() for _ in range(F)]
    step = [torch.randint(-4, 5, (N, D), device=DEV, generator=g).float() for _ in range(F)]
    before = ops.embbag_sum_multi(tables, idx, off, L)
    after = ops.embbag_sum_multi([t + s for t, s in zip(tables, step)], idx, off, L)
    total = 0.0
    for k in range(F):
        out = tokens.embedding_grad(dpooled[:, k], idx[k], N, L=L)
        _check_grad(out, dpooled[:, k].contiguous(), idx[k], N, L=L)
        total += float((out.double() * step[k].double()).sum())
    change = ((after - before).double() * dpooled.double())
    # the pooled sums are linear in the tables; the gradient's own error is
    # n 2^-24 of what it sums, n at most B * L
    tol = (B * L + 1) * 2.0 ** -24 * float(
        sum((dpooled[:, k].double().abs().repeat_interleave(L, 0)
             * step[k].double().abs()[idx[k].long()]).sum() for k in range(F)))
    assert abs(total - float(change.sum())) <= tol


@pytest.mark.parametrize("T", [50, 5000, 70000])
def test_grad_streams_scratch_and_graphs(tokens, T):
    """On a stream of its own, with the caller's scratch, captured and replayed
    with new inputs, next to another captured call with its own scratch."""
    g = _gen(3)
    D, N = 64, 700
    need = tokens.embedding_grad_scratch_bytes(T, N, D)
    calls = []
    side = torch.cuda.Stream()
    for k in range(2):
        grad, _ = _matrix(g, T, D, F32)
        ids = torch.from_numpy(_ids(k, T, N, "skew")).to(DEV)
        calls.append((grad, ids, torch.empty((N, D), device=DEV),
                      torch.full((need,), 255, dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for grad, ids, out, scratch in calls:
            tokens.embedding_grad(grad, ids, N, out=out, scratch=scratch)
    side.synchronize()
    for grad, ids, out, _ in calls:
        _check_grad(out, grad, ids, N)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for grad, ids, out, scratch in calls:
            tokens.embedding_grad(grad, ids, N, out=out, scratch=scratch)
            tokens.embedding_lookup(out, ids)
    for k, (grad, ids, out, scratch) in enumerate(calls):
        grad.mul_(-2.0)
        ids.copy_(torch.from_numpy(_ids(k + 9, T, N, "ends")))
        scratch.fill_(7)
        out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for grad, ids, out, _ in calls:
        _check_grad(out, grad, ids, N)


@pytest.mark.parametrize("T", [0, 40, 3000, 100000])
def test_grad_waits_for_what_writes_its_output(tokens, T):
    """A bf16 layer lets the kernel behind it start before it ends: a gradient into
    the layer's own output still comes after it, and a layer on the gradient after that."""
    from dlrm_embedding_bag_b200 import mlp

    g = _gen(T + 7)
    rows, D = 60000, 64
    a, _ = _matrix(g, rows, 512, BF16)
    w, _ = _matrix(g, D, 512, BF16)
    grad, _ = _matrix(g, T, D, F32)
    ids = torch.from_numpy(_ids(T, T, rows, "skew")).to(DEV)
    out = torch.empty((rows, D), device=DEV)
    for _ in range(3):
        mlp.linear_bf16(a, w, None, "none", out_f32=out)
        tokens.embedding_grad(grad, ids, rows, out=out)
        seen = mlp.to_bf16(out)
        torch.cuda.synchronize()
        _check_grad(out, grad, ids, rows)
        assert _same_bits(seen, out.to(BF16))


@pytest.mark.parametrize("T", [0, 5, 600, 70000])
def test_a_layer_waits_for_a_gradient_that_is_its_bias(tokens, T):
    """A bf16 layer reads its bias before it waits for the kernel in front, which so must
    not let it start early: the bias here is the last row of a gradient."""
    from dlrm_embedding_bag_b200 import mlp

    g = _gen(T + 11)
    rows, D = 300000, 128
    a, _ = _matrix(g, 256, 64, BF16)
    w, _ = _matrix(g, D, 64, BF16)
    grad, _ = _matrix(g, T, D, F32)
    ids = torch.full((T,), rows - 1, dtype=torch.int32, device=DEV)
    ids[: T // 2] = 3
    out = torch.empty((rows, D), device=DEV)
    for k in range(3):
        out.fill_(float(k + 5))
        tokens.embedding_grad(grad, ids, rows, out=out)
        seen, _ = mlp.linear_bf16(a, w, out[rows - 1])
        torch.cuda.synchronize()
        _check_grad(out, grad, ids, rows)
        again, _ = mlp.linear_bf16(a, w, out[rows - 1].clone())
        assert _same_bits(seen, again)


@pytest.mark.parametrize("T", [300, 6000, 90000])
def test_grads_at_the_same_time(tokens, T):
    """Calls that overlap on four streams, each with the scratch that torch gives it."""
    g = _gen(T)
    N, D = 5000, 40
    calls = []
    for k in range(4):
        grad, _ = _matrix(g, T, D, F32)
        calls.append((grad, torch.from_numpy(_ids(k, T, N, "skew")).to(DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        for grad, ids, stream in calls:
            with torch.cuda.stream(stream):
                outs.append(tokens.embedding_grad(grad, ids, N))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        grad, ids, _ = calls[i % 4]
        _check_grad(out, grad, ids, N)
        assert _same_bits(out, outs[i % 4])


def test_first_calls_under_capture():
    """In a new process every operator's first call may be a captured one: their
    set-up makes no call that a capture forbids."""
    code = """
import torch
from dlrm_embedding_bag_b200 import int8, tokens
dev = "cuda"
x = torch.randn(70000, 32, device=dev); ids = torch.randint(0, 900, (70000,), device=dev).int()
w = torch.zeros(4096, 512, dtype=torch.int8, device=dev); ws = torch.ones(4096, device=dev)
torch.cuda.synchronize()
outs = []
side = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=side):
    for T in (100, 3000, 12000, 20000, 40000, 66000):
        outs.append(tokens.embedding_grad(x[:T], ids[:T], 900))
        outs.append(tokens.embedding_lookup(x, ids[:T]))
    for M in (1, 2, 4, 16, 64, 128, 600, 3000):
        q, s, _ = int8.rms_norm_int8(x[:16 * M].view(M, 512))
        outs.append(int8.linear_int8(q, s, w, ws, out_dtype=torch.bfloat16))
w.copy_(torch.randint(-9, 9, w.shape, device=dev).to(torch.int8))
graph.replay()
torch.cuda.synchronize()
i = 0
for T in (100, 3000, 12000, 20000, 40000, 66000):
    assert torch.equal(outs[i], tokens.embedding_grad(x[:T], ids[:T], 900)), T
    assert torch.equal(outs[i + 1], x[ids[:T].long()]), T
    i += 2
for M in (1, 2, 4, 16, 64, 128, 600, 3000):
    q, s, _ = int8.rms_norm_int8(x[:16 * M].view(M, 512))
    assert torch.equal(outs[i], int8.linear_int8(q, s, w, ws, out_dtype=torch.bfloat16)), M
    i += 1
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]


def test_grad_refusals(tokens):
    grad = torch.zeros((6, 8), device=DEV)
    ids = torch.zeros(6, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="rows"):
        tokens.embedding_grad(grad, ids, 4, L=2)
    with pytest.raises(ValueError, match="accumulate needs out"):
        tokens.embedding_grad(grad, ids, 4, accumulate=True)
    with pytest.raises(ValueError, match="padding_idx"):
        tokens.embedding_grad(grad, ids, 4, padding_idx=4)
    with pytest.raises(ValueError, match="overlap"):
        tokens.embedding_grad(grad[:1].expand(6, 8), ids, 4)
    with pytest.raises(TypeError, match="int32"):
        tokens.embedding_grad(grad, ids.long(), 4)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        tokens.embedding_grad(grad.half(), ids, 4)
    with pytest.raises(tokens.TokensError, match="DLRM_ERR_SCRATCH"):
        tokens.embedding_grad(grad.repeat(200, 1), ids.repeat(200), 4,
                              scratch=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(tokens.TokensError, match="DLRM_ERR_SHAPE"):
        tokens.embedding_grad(grad, ids, 2 ** 31, out=None, accumulate=False)
    with pytest.raises(ValueError, match="out must be"):
        tokens.embedding_grad(grad, ids, 4, out=torch.zeros((5, 8), device=DEV))
    with pytest.raises(ValueError, match="unit column stride"):
        tokens.embedding_lookup(torch.zeros((8, 6), device=DEV).t(), ids)
    with pytest.raises(ValueError, match="must be on"):
        tokens.embedding_lookup(grad, ids.cpu())
