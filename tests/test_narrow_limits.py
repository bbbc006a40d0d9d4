"""Sizes that the 4-bit layer cannot take are refused as sizes, before any CUDA call."""
import pytest

A, W, Y, S = 0x10000, 0x20000, 0x30000, 0x40000  # aligned, never dereferenced
SHAPE = -2


@pytest.fixture(scope="module")
def optim():
    from dlrm_embedding_bag_b200 import build

    build.build()
    from dlrm_embedding_bag_b200 import optim as _optim

    return _optim


@pytest.mark.parametrize("m,n", [(1 << 30, 1 << 30), (1 << 22, 1 << 22), ((1 << 31) - 1025, 128 * 64 + 1),
                                 (64 * 128 + 1, (1 << 31) - 1025)])
def test_more_tiles_than_are_counted(optim, m, n):
    assert -(-m // 64) * -(-n // 128) > (1 << 31) - 1
    assert optim._lib.dlrm_linear_fp4(A, 32, S, W, 32, S, None, m, n, 64, 0, Y, 0, n, None, None) == SHAPE


@pytest.mark.parametrize("kw", [dict(ldx=1 << 40), dict(ldw=1 << 40), dict(ldx=1 << 62, ldw=1 << 62)])
def test_pitches_that_no_map_takes(optim, kw):
    kw = dict(dict(ldx=32, ldw=32), **kw)
    assert optim._lib.dlrm_linear_fp4(A, kw["ldx"], S, W, kw["ldw"], S, None, 4, 8, 64, 0, Y, 0, 8, None,
                                      None) == SHAPE
