"""The root that becomes a code, against the square root that CUDA offers (correctly rounded in f32),
over every exponent and many significands.

Blocks with one element that is not zero: the block's scale is then that element's root times
1 / 1.9375 rounded, which shows it. The root is r + (x - r^2) y / 2 from r = x y, and y = 1 / sqrt(x)
within 2^-22: r is within 2^-21.7 of the root, what is left after the step is its square's half and
the rounding of y / 2 and of the residual, below 2^-43 of the root, and the last rounding. So it is
within one last place everywhere, and another number than the nearest only where the root is
within 2^-43 of the middle of two: 2^-43 / 2^-25 of them, 2^-18, where roots spread evenly.

That is so from x = 2^-100 on. Below, the residual x - r^2 (2^-21.7 x at most) is a number of f32 that
ends at 2^-149: it is off by up to 2^-150, which is 2^-151 / x of the root. At x = 2^-126 that
is 2^-25, a quarter to a half of a last place (2^-23 to 2^-24), so that many roots come out as the
neighbour, but none farther: the last rounding adds half a place to a half at most. At 2^-100 it
is 2^-51, which the 2^-43 above cover.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
C = torch.tensor(1 / 1.9375, dtype=torch.float32).item()


@pytest.fixture(scope="module")
def optim():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from dlrm_embedding_bag_b200 import optim as _optim

    return _optim


def _roots(optim, values, b2):
    """(second moments of the gradients `values`, the scales that a step from nothing stores)."""
    n = values.numel()
    grad = torch.zeros((n, 256), device=DEV)
    grad[torch.arange(n, device=DEV), torch.arange(n, device=DEV) * 37 % 256] = values
    p = torch.zeros_like(grad)
    st = optim.adamw_state([p], bits=8)
    optim.adamw_step([p], [grad], st, lr=0.0, betas=(0.5, b2))
    # every product rounds by itself, as these do
    return values * values * torch.tensor(1.0 - b2, device=DEV), st.v_scale


def _check(v, scale):
    """Scales within a last place's, and how many of the roots of moments from 2^-100 on are another
    number than the nearest."""
    want = v.sqrt()
    c = torch.tensor(C, device=DEV)
    near = scale == want * c
    up = torch.nextafter(want, torch.full_like(want, float("inf"))) * c
    down = torch.nextafter(want, torch.zeros_like(want)) * c
    live = v >= 2.0 ** -126
    assert (near | (scale == up) | (scale == down))[live].all()
    assert (scale[~live] == 0).all()
    return (~near & (v >= 2.0 ** -100)).sum().item()


@pytest.mark.parametrize("b2", [0.3, 0.999])
def test_many_significands(optim, b2):
    """2^18 of them in each of two neighbouring binades of the moment. 1 in 2^18 at most is expected
    to be off: 12 of 2^19 would be ten more."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    off = 0
    for e in (0, 1):
        x = torch.empty(1 << 18, device=DEV).uniform_(1, 2, generator=g) * 2.0 ** (e / 2)
        off += _check(*_roots(optim, x, b2))
    assert off <= 12


def test_every_exponent(optim):
    """Gradients of every binade whose square is a number of f32, on both sides of the least normal
    one, and past the largest."""
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    e = torch.arange(-76, 64, device=DEV).repeat_interleave(1024)
    x = torch.empty(e.numel(), device=DEV).uniform_(1, 2, generator=g) * torch.exp2(e.float())
    v, scale = _roots(optim, x, 0.25)
    gone = v > torch.finfo(torch.float32).max
    assert torch.equal(scale.isnan(), gone | (x * x).isinf())
    ok = ~scale.isnan()
    # 2^17 roots at most: half of one is expected
    assert _check(v[ok], scale[ok]) <= 6
