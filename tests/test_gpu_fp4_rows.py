"""4-bit rows: largest elements of a block, long rows that start anywhere, and what lies between
rows of codes. Codes and scales have no tolerance (header of test_gpu_fp4.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_gpu_fp4 import BF16, DEV, F32, LEVELS, _check_rows, _expect, _gen, _normal, _scales, fp4  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_of_a_block_by_halves(fp4, dtype, sign):  # noqa: F811
    """3.5 is 7 times 2^-1: its scale is 2^-1 and its level 6, so it becomes 3. The same at every
    power of two, and the next number above is 4 times the next scale."""
    for e in range(-124, 124, 7):
        for v, level, up in ((3.5, 6.0, -1), (7.0, 6.0, 0), (6.0, 6.0, 0), (4.0, 4.0, 0), (3.75, 4.0, 0),
                             (7.0625, 4.0, 1), (14.0, 6.0, 1)):
            x = torch.zeros((1, 32), device=DEV, dtype=dtype)
            x[0, 5] = sign * v * 2.0 ** e
            q, s = fp4.quantize_rows(x)
            assert _scales(fp4, s, 1, 32)[0].item() == 127 + e + up, (v, e)
            assert fp4.dequantize_rows(q, s)[0, 5].item() == sign * level * 2.0 ** (e + up), (v, e)
            _check_rows(fp4, x, q, s, (v, e))
    x = torch.zeros((1, 32), device=DEV)
    x[0, 31] = float(np.nextafter(np.float32(3.5), np.float32(4)))
    q, s = fp4.quantize_rows(x)
    assert _scales(fp4, s, 1, 32)[0].item() == 127 and fp4.dequantize_rows(q, s)[0, 31].item() == 4.0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("k", [257, 490, 999, 1000, 1001, 1024, 1535, 4097])
def test_long_rows_that_start_anywhere(fp4, dtype, k):  # noqa: F811
    """Pieces of 8, 16 and 32 lanes, some of them past a row's end, rows of values at every offset and
    pitch; codes with bytes of others in front of, between and behind their rows."""
    g = _gen(51)
    m, width = 11, (k + 1) // 2
    for start in range(0, 9):
        x = _normal(g, m, k, dtype, k + start % 4, start)
        code, byte = _expect(x)
        gap = start % 4
        qbuf = torch.full((start + m * (width + gap) + 8,), 77, device=DEV, dtype=torch.uint8)
        rows = qbuf[start:start + m * (width + gap)].view(m, width + gap)
        q = rows[:, :width]
        _, s = fp4.quantize_rows(x, out=q)
        _check_rows(fp4, x, q, s, start)
        assert (rows[:, width:] == 77).all() and (qbuf[:start] == 77).all()
        assert (qbuf[start + m * (width + gap):] == 77).all()
        sign = 1 - 2 * (code >= 8).double()
        want = sign * LEVELS.to(DEV)[code % 8] * torch.exp2(byte.double() - 127).repeat_interleave(32, 1)[:, :k]
        for out_dtype in (F32, BF16):
            for pitch in (k, k + 1, k + 3, (k + 7) // 8 * 8):
                ybuf = torch.full((start + m * pitch + 16,), 5.0, device=DEV, dtype=out_dtype)
                y = ybuf[start:start + m * pitch].view(m, pitch)
                fp4.dequantize_rows(q, s, k, out=y[:, :k])
                assert torch.equal(y[:, :k].double(), want), (start, pitch)
                assert (y[:, k:] == 5).all() and (ybuf[:start] == 5).all()
                assert (ybuf[start + m * pitch:] == 5).all()
