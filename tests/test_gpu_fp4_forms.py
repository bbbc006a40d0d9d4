"""The 4-bit layer in every form of its kernels, against its definition in 64 bits (tolerances: the
header of test_gpu_fp4.py) and on whole numbers exactly. test_fp4_forms.py holds the shapes to the
forms that they stand for."""
from __future__ import annotations

import pytest
import torch

from test_gpu_fp4 import BF16, DEV, F32, _check_layer, _gen, _layer, fp4  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

# (tokens, columns, channels) by what they take: a tile's tokens and the CTAs of a cluster that share
# it, or of one token the blocks that a lane has in flight and the channels of a warp
FORMS = {
    (64, 1): [(70, 500, 301)],
    (64, 2): [(7, 3052, 430), (122, 3041, 27), (356, 4333, 851)],
    (64, 4): [(5, 4097, 515), (61, 3901, 130)],
    (128, 1): [(1500, 701, 1303)],
    (128, 2): [(282, 8147, 2510), (449, 5287, 1071), (80, 6635, 7594)],
    (128, 4): [(198, 4684, 1033), (2131, 4661, 1), (125, 6161, 2967)],
    (256, 1): [(4003, 1301, 2999)],
}
ONES = {
    (1, 1): [(1, 1000, 301)],
    (1, 4): [(1, 1000, 3001), (1, 33, 2503), (1, 1024, 2368)],
    (2, 1): [(1, 1999, 700)],
    (2, 4): [(1, 2048, 2401), (1, 4096, 4096), (1, 4097, 5003), (1, 6401, 4062)],
    (4, 1): [(1, 4096, 333), (1, 4099, 2367)],
}
ALL = [(f, s) for t in (FORMS, ONES) for f, shapes in t.items() for s in shapes]


@pytest.mark.parametrize("form,shape", ALL, ids=lambda v: "x".join(map(str, v)))
def test_every_form(fp4, form, shape):  # noqa: F811
    g = _gen(41)
    m, k, n = shape
    for act, out, bias in (("none", F32, False), ("relu", BF16, True), ("sigmoid", F32, True),
                           ("none", BF16, True)):
        ops = _layer(fp4, g, m, k, n, bias, wide=0.5)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        buf = torch.full((m + 1, n + 7), 9.0, device=DEV, dtype=out)
        y = fp4.linear_fp4(*ops, act, out=buf[:m, 3:3 + n], status=status)
        assert status.item() == 0
        _check_layer(fp4, y, *ops, act)
        assert (buf[:, :3] == 9).all() and (buf[:, 3 + n:] == 9).all() and (buf[m:] == 9).all()
        assert torch.equal(y, fp4.linear_fp4(*ops, act, out=torch.empty_like(buf)[:m, 3:3 + n]))


@pytest.mark.parametrize("form,shape", ALL, ids=lambda v: "x".join(map(str, v)))
def test_every_form_on_whole_numbers(fp4, form, shape):  # noqa: F811
    """Sums below 2^24 that f32 holds exactly in any order: no part of a joined sum may be lost."""
    g = _gen(42)
    m, k, n = shape
    x, w = (torch.randint(-2, 3, (r, k), device=DEV, generator=g).float() for r in (m, n))
    (xq, xs), (wq, ws) = fp4.quantize_rows(x), fp4.quantize_rows(w)
    b = torch.randint(-99, 100, (n,), device=DEV, generator=g).float()
    y = fp4.linear_fp4(xq, xs, wq, ws, b, out=torch.empty((m, n + 3), device=DEV)[:, :n])
    assert torch.equal(y.double(), x.double() @ w.double().T + b.double())


# (tokens, columns, channels) whose outputs, pitched, leave as whole lines through the copy engine
LINES = [(4099, 1300, 4072), (5003, 1301, 3000), (4100, 1500, 4008), (4225, 1111, 3976)]


@pytest.mark.parametrize("start", [16, 48])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", LINES, ids=lambda s: "x".join(map(str, s)))
def test_whole_lines_with_a_pitch(fp4, shape, dtype, start):  # noqa: F811
    """What lies before, between, beside and behind the output's rows stays as it was. (Rows are
    whole 16 bytes, that start on 16 but not on 128, and their last line is not full.)"""
    g = _gen(43)
    m, k, n = shape
    ops = _layer(fp4, g, m, k, n, True)
    size = 4 if dtype == F32 else 2
    pitch, first = n + 2 * 16 // size + 48 // size, start // size
    assert n * size % 16 == 0 and n * size % 128 != 0 and pitch * size % 16 == 0
    flat = torch.full((first + m * pitch + 64,), 9.0, device=DEV, dtype=dtype)
    rows = flat[first:first + m * pitch].view(m, pitch)
    y = fp4.linear_fp4(*ops, "relu", out=rows[:, :n])
    _check_layer(fp4, y, *ops, "relu")
    assert (rows[:, n:] == 9).all() and (flat[:first] == 9).all() and (flat[first + m * pitch:] == 9).all()
    assert torch.equal(y, fp4.linear_fp4(*ops, "relu", out_dtype=dtype))
