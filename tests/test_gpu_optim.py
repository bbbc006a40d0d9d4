"""The AdamW step over many tensors on the GPU, against its formula in 64 bits.

Bounds, with u = 2^-24 (half a step of f32). First moment: beta1 and 1 - beta1 are
rounded once each, as are the scaled gradient and its product; the rest is one fused
rounding: 5 u of |b1 m| + |b1c g|. Second: the squares' factors round once each, the
gradient twice as it enters twice: 7 u of a sum of positive terms. The weight: sqrt and
quotient are within 2 u each (a last place), root, alpha, the product with eps round
once each, and v's error enters by half: the step alpha M / (sqrt(v) root + eps) is
within 20 u of what it is for M = |b1 m| + |b1c g|; p itself rounds three times (the
decay's factor, its product, the sum): 4 u. A result in bf16 from a master is 2^-8 of
it; at random, it is one of the two neighbours: less than 2^-7. 8-bit moments are one of
the two neighbours on their grid: within a step of the exact ones, 2^-3 (first) or 2^-4
(root) relative, plus what f32 adds (16 u of the block's largest).

Products and sums that round each by itself are within the same bounds: of the first moment b1 m
rounds as a factor, a product and a sum (3 u), the gradient once as it is scaled besides (4 u); of the
second b2 v 3 u, the square 2 u by its gradient, and by itself, its factor, product and sum 4 u.
"""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


@pytest.fixture(scope="module")
def optim():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from dlrm_embedding_bag_b200 import optim as _optim

    return _optim


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype=F32, std=1.0):
    return torch.empty(shape, device=DEV).normal_(0, std, generator=g).to(dtype)


def _pieces(optim, params, flat):
    """The arena's part of each parameter, in its shape."""
    at, total = optim.arena_offsets(params)
    assert flat.numel() == total
    return [flat[o:o + p.numel()].view(p.shape) for o, p in zip(at, params)]


def _padding(optim, params, flat):
    at, total = optim.arena_offsets(params)
    used = torch.zeros(total, dtype=torch.bool, device=DEV)
    for o, p in zip(at, params):
        used[o:o + p.numel()] = True
    return flat[~used]


def _exact(p, m, v, g, t, lr, b1, b2, eps, wd, coef=1.0):
    """(p, m, v) after the step and the size of the step's numerator's terms, in 64 bits."""
    p, m, v, g = p.double(), m.double(), v.double(), g.double() * coef
    terms = (b1 * m).abs() + ((1 - b1) * g).abs()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    den = v.div(1 - b2 ** t).sqrt() + eps
    alpha = lr / (1 - b1 ** t)
    return p * (1 - lr * wd) - alpha * m / den, m, v, terms, alpha * terms / den


SIZES = [(1,), (3, 5), (255,), (256,), (257,), (0,), (2047,), (2048,), (2049,), (64, 1000), (5, 7, 11)]


@pytest.mark.parametrize("gtype", [F32, BF16], ids=["g32", "g16"])
@pytest.mark.parametrize("ptype", [F32, BF16], ids=["p32", "p16"])
def test_three_steps_in_32_bits(optim, ptype, gtype):
    g = _gen(1)
    lr, betas, eps, coef = 3e-2, (0.8, 0.95), 1e-6, 0.37
    wds = [0.1 * (i % 3) for i in range(len(SIZES))]
    params = [_normal(g, s, ptype) for s in SIZES]
    state = optim.adamw_state(params, master=ptype == BF16)
    c = torch.tensor([coef], device=DEV)
    coef = c.double().item()
    for t in range(1, 4):
        grads = [_normal(g, s, gtype, 10.0 ** (i - 5)) for i, s in enumerate(SIZES)]
        old = [x.clone() for x in _pieces(optim, params, state.master)] if ptype == BF16 else \
            [p.clone() for p in params]
        m0, v0 = state.m.clone(), state.v.clone()
        optim.adamw_step(params, grads, state, lr=lr, betas=betas, eps=eps, weight_decay=wds,
                         grad_scale=c)
        assert state.step.tolist() == [t, 0]
        new = _pieces(optim, params, state.master) if ptype == BF16 else params
        for i, (p, q, gr, m, v, ma, va, wd) in enumerate(zip(
                old, new, grads, _pieces(optim, params, m0), _pieces(optim, params, v0),
                _pieces(optim, params, state.m), _pieces(optim, params, state.v), wds)):
            pe, me, ve, terms, step = _exact(p, m, v, gr, t, lr, *betas, eps, wd, coef)
            assert ((ma.double() - me).abs() <= 5 * U * terms + 2.0 ** -149).all(), i
            assert ((va.double() - ve).abs() <= 7 * U * ve + 2.0 ** -149).all(), i
            assert ((q.double() - pe).abs() <= 4 * U * p.double().abs() + 20 * U * step
                    + U * step).all(), i
        if ptype == BF16:
            for p, w in zip(params, new):
                assert torch.equal(p, w.to(BF16))
        for flat in (state.m, state.v):
            assert (_padding(optim, params, flat) == 0).all()


# ---- moments in 8 bits ------------------------------------------------------------------


def _root_grid(code):
    """Values of the roots' codes, by the format's words."""
    c = code.long()
    e, f = c // 16, (c % 16).double()
    return torch.where(e > 0, (16 + f) * 2.0 ** (e - 19).double(), f * 2.0 ** -18)


def _read(state):
    """8-bit moments in 64 bits: m, and the root of v."""
    m = state.m.to(F32).double().view(-1, 256) * state.m_scale.double()[:, None]
    r = _root_grid(state.v).view(-1, 256) * state.v_scale.double()[:, None]
    return m.view(-1), r.view(-1)


def _check_8bit(state, m, v, gmax=0.0):
    """The stored moments against the exact arena m, v: scales, and a step of the grid."""
    u = 16 * U
    top = m.view(-1, 256).abs().amax(1)
    live = top / 448 >= 2.0 ** -126 * (1 + u)
    assert ((state.m_scale.double() - top / 448).abs() <= u * (top + gmax) / 448)[live].all()
    r = v.sqrt()
    rtop = r.view(-1, 256).amax(1)
    assert ((state.v_scale.double() - rtop / 1.9375).abs() <= u * rtop / 1.9375).all()
    ms, rs = _read(state)
    unit = (top / 448)[:, None].expand(-1, 256).reshape(-1)
    step = torch.maximum(m.abs(), unit * 2.0 ** -6) * 2.0 ** -3
    dead = ~live[:, None].expand(-1, 256).reshape(-1)
    slack = u * (top + gmax)[:, None].expand(-1, 256).reshape(-1)
    assert (((ms - m).abs() <= step + slack) | dead).all()
    runit = (rtop / 1.9375)[:, None].expand(-1, 256).reshape(-1)
    rstep = torch.maximum(r, runit * 2.0 ** -14) * 2.0 ** -4
    assert ((rs - r).abs() <= rstep * (1 + u) + u * r).all()
    assert ((rs > 0) == (r > 0)).all(), "a root that is not zero stays so"


@pytest.mark.parametrize("ptype", [F32, BF16], ids=["p32", "p16"])
@pytest.mark.parametrize("master", [False, True])
def test_steps_in_8_bits(optim, ptype, master):
    g = _gen(2)
    lr, betas, eps, wd = 1e-2, (0.9, 0.99), 1e-8, 0.05
    shapes = [s for s in SIZES if s != (0,)] + [(0,), (3000,)]
    params = [_normal(g, s, ptype) for s in shapes]
    state = optim.adamw_state(params, bits=8, master=master)
    whole = master and ptype == BF16
    for t in range(1, 5):
        # elements of very different size, some without any gradient
        grads = [(_normal(g, s) * torch.exp(3 * _normal(g, s)) * (_normal(g, s) > -1)) for s in shapes]
        if t == 3:
            grads = [x.to(BF16) for x in grads]
        m0, r0 = _read(state)
        old = [x.clone() for x in (_pieces(optim, params, state.master) if whole else params)]
        optim.adamw_step(params, grads, state, lr=lr, betas=betas, eps=eps, weight_decay=wd,
                         seed=9)
        me, ve = torch.zeros_like(m0), torch.zeros_like(m0)
        rows = zip(params, old, grads, _pieces(optim, params, m0), _pieces(optim, params, r0 * r0),
                   _pieces(optim, params, me), _pieces(optim, params, ve),
                   _pieces(optim, params, state.master) if whole else params)
        for p, q, gr, m, v, mo, vo, w in rows:
            pe, mx, vx, terms, step = _exact(q, m, v, gr, t, lr, *betas, eps, wd)
            mo.copy_(mx)
            vo.copy_(vx)
            # the moments that were read are products of a code and a scale: two more roundings
            # of the first, four of the second
            bound = 4 * U * q.double().abs() + 26 * U * step
            if whole:
                assert torch.equal(p, w.to(BF16))
            elif ptype == BF16:
                bound = bound + 2.0 ** -7 * (pe.abs() + bound)
            assert ((w.double() - pe).abs() <= bound).all()
        # what cancels in a block's largest moment is as large as the terms
        _check_8bit(state, me, ve, gmax=2 * me.view(-1, 256).abs().amax(1))
        for flat in (state.m.view(torch.uint8), state.v):
            assert (_padding(optim, params, flat) == 0).all()


def test_random_rounding_has_the_right_mean(optim):
    """Many steps from one state by many seeds: moments and bf16 weights are right on average.
    A code is off by less than a step and by none on average: the mean of N is within 6 of its
    standard deviations (at most step / 2 / sqrt(N)) of the exact value, plus the 2^-16 of
    a step by which 16 random bits are coarse."""
    g = _gen(3)
    n, N = 2048, 400
    p0 = _normal(g, (n,), BF16)
    grad = _normal(g, (n,)) * torch.exp(_normal(g, (n,)))
    first = optim.adamw_state([p0], bits=8)
    optim.adamw_step([p0.clone()], [grad], first, lr=0.0)
    lr, betas, eps = 1e-3, (0.9, 0.999), 1e-8
    total = [torch.zeros(n, device=DEV, dtype=torch.float64) for _ in range(3)]
    m0, r0 = _read(first)
    grad2 = _normal(g, (n,)) * 0.1
    for seed in range(N):
        st = optim.AdamWState(*[None if x is None else x.clone() for x in first])
        p = p0.clone()
        optim.adamw_step([p], [grad2], st, lr=lr, betas=betas, eps=eps, seed=seed * 7919)
        m, r = _read(st)
        for s, x in zip(total, (m, r, p.double())):
            s += x / N
    pe, me, ve, _, _ = _exact(p0, m0, r0 * r0, grad2, 2, lr, *betas, eps, 0.0)
    re = ve.sqrt()
    top = me.view(-1, 256).abs().amax(1, keepdim=True).expand(-1, 256).reshape(-1)
    rtop = re.view(-1, 256).amax(1, keepdim=True).expand(-1, 256).reshape(-1)
    steps = (torch.maximum(me.abs(), top / 448 * 2.0 ** -6) * 2.0 ** -3,
             torch.maximum(re, rtop / 1.9375 * 2.0 ** -14) * 2.0 ** -4, pe.abs() * 2.0 ** -7)
    for name, mean, exact, step in zip("mrp", total, (me, re, pe), steps):
        far = (mean - exact).abs() / step
        assert (far <= 6 * 0.5 / math.sqrt(N) + 2.0 ** -16 + 1e-4).all(), (name, far.max())
        # and over all elements together: 2048 N draws
        bias = ((mean - exact) / step).mean().abs().item()
        assert bias <= 6 * 0.5 / math.sqrt(N * n) + 2.0 ** -16 + 1e-4, (name, bias)


def test_equal_calls_give_equal_bits_and_seeds_differ(optim):
    g = _gen(4)
    p0, grad = _normal(g, (5000,), BF16), _normal(g, (5000,))

    def run(seed):
        p = p0.clone()
        st = optim.adamw_state([p], bits=8)
        for _ in range(3):
            optim.adamw_step([p], [grad], st, lr=1e-3, seed=seed)
        return p, st.m.view(torch.uint8), st.v, st.m_scale, st.v_scale

    a, b, c = run(5), run(5), run(6)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert not torch.equal(a[1], c[1]) and not torch.equal(a[2], c[2])


def test_moments_are_read(optim):
    g = _gen(5)
    params = [_normal(g, (700,)), _normal(g, (3, 300))]
    st = optim.adamw_state(params, bits=8)
    optim.adamw_step(params, [_normal(g, p.shape) for p in params], st, lr=1e-3)
    m, r = _read(st)
    for dtype, eps in ((F32, U), (BF16, 2.0 ** -8)):
        mv, vv = optim.adamw_moments(st, dtype=dtype)
        assert mv.dtype == dtype and mv.shape == st.m.shape
        assert ((mv.double() - m).abs() <= (eps + 2 * U) * m.abs()).all()
        assert ((vv.double() - r * r).abs() <= (eps + 4 * U) * r * r).all()
    with pytest.raises(ValueError, match="32 bits"):
        optim.adamw_moments(optim.adamw_state(params))


# ---- values at the ends ---------------------------------------------------------------------


@pytest.mark.parametrize("bits", [8, 32])
def test_no_gradient_at_all(optim, bits):
    """Zeros in, zeros kept: only the decay moves a weight."""
    p = _normal(_gen(6), (1000,))
    q = p.clone()
    st = optim.adamw_state([p], bits=bits)
    optim.adamw_step([p], [torch.zeros_like(p)], st, lr=0.5, weight_decay=0.25)
    assert torch.equal(p, q * 0.875)
    assert (st.m.view(torch.uint8) == 0).all() and (st.v.view(torch.uint8) == 0).all()
    if bits == 8:
        assert (st.m_scale == 0).all() and (st.v_scale == 0).all()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite_gradients(optim, bits, bad):
    """They reach their own element at once; in 8 bits their block's others from the next step."""
    g = _gen(7)
    p, grad = _normal(g, (1024,)), _normal(g, (1024,))
    grad[300] = bad
    st = optim.adamw_state([p], bits=bits)
    optim.adamw_step([p], [grad], st, lr=1e-3)
    # inf / inf
    assert p[300].isnan() and p.isnan().sum() == 1
    optim.adamw_step([p], [torch.zeros_like(grad)], st, lr=1e-3)
    hurt = torch.zeros(1024, dtype=torch.bool, device=DEV)
    hurt[256:512] = True
    assert torch.equal(p.isnan(), hurt) if bits == 8 else p.isnan().sum() == 1


def test_moments_round_as_elementary_operations_do(optim):
    """What becomes codes is the formula's f32 value, every product, sum and root rounded once: the
    scales bit for bit. (Nothing is fused and the root is the nearest, but for a few of 2^20.)"""
    g = _gen(31)
    n = 256 * 4000
    p, grad = torch.zeros(n, device=DEV), _normal(g, (n,))
    st = optim.adamw_state([p], bits=8)
    m = v = torch.zeros(n, device=DEV)
    one = torch.ones((), device=DEV)
    for step in range(2):
        grad = _normal(g, (n,))
        m0, v0 = (t.view(-1, 256) for t in (st.m.float(), torch.zeros(n, device=DEV)))
        if step:
            c = st.v.int().view(-1, 256)
            v0 = torch.where(c < 16, (c % 16) * 2.0 ** -18, (1 + (c % 16) / 16) * torch.exp2((c // 16 - 15).float()))
            v0 = (v0 * st.v_scale[:, None]) ** 2
        m0 = m0 * st.m_scale[:, None]
        x = grad.view(-1, 256)
        m = m0 * 0.9 + x * (1 - 0.9)
        v = v0 * 0.999 + x * x * (1 - 0.999)
        optim.adamw_step([p], [grad], st, lr=1e-3)
        assert torch.equal(st.m_scale, m.abs().amax(1) * (one / 448))
        far = st.v_scale != v.sqrt().amax(1) * (one / 1.9375)
        assert far.sum() <= 4


def test_squares_that_leave_f32(optim):
    """A finite gradient whose square is infinite: no step of its element, its block's moments NaN."""
    p, grad = torch.ones(512, device=DEV), torch.ones(512, device=DEV)
    grad[3] = 1e25
    st = optim.adamw_state([p], bits=8)
    optim.adamw_step([p], [grad], st, lr=1e-3)
    assert p[3] == 1 and p.isfinite().all() and (p[4:] < 1).all()
    assert st.v_scale[0].isnan() and st.v_scale[1].isfinite()


def test_first_moments_too_small_for_a_scale_are_dropped(optim):
    p = torch.zeros(256, device=DEV)
    st = optim.adamw_state([p], bits=8)
    optim.adamw_step([p], [torch.full_like(p, 1e-36)], st, lr=1e-3, betas=(0.0, 0.0), eps=1e-30)
    assert (st.m_scale == 0).all() and (st.m.view(torch.uint8) == 0).all()
    # squares of such gradients vanish in f32, here as in 32 bits
    assert (st.v == 0).all() and p.isfinite().all()


def test_bf16_weights_at_the_ends(optim):
    p = torch.tensor([float("inf"), -float("inf"), float("nan"), 3.3e38, 0.0, -0.0], device=DEV).to(BF16)
    q = p.clone()
    st = optim.adamw_state([p])
    optim.adamw_step([p], [torch.zeros(6, device=DEV)], st, lr=1e-3)
    assert torch.equal(p.view(torch.int16)[[0, 1, 3, 4]], q.view(torch.int16)[[0, 1, 3, 4]])
    assert p[2].isnan() and p[5] == 0


@pytest.mark.parametrize("bits", [8, 32])
def test_what_lies_behind_a_tensor_stays_zero(optim, bits):
    """Also where the clipping coefficient is not a number."""
    params = [torch.ones(3, device=DEV), torch.ones(700, device=DEV, dtype=BF16)]
    st = optim.adamw_state(params, bits=bits, master=True)
    bad = torch.full((1,), float("nan"), device=DEV)
    optim.adamw_step(params, [torch.ones_like(p) for p in params], st, lr=1e-3, grad_scale=bad)
    assert all(p.isnan().all() for p in params)
    for flat in (st.m, st.v, st.master):
        if flat.dtype == torch.float8_e4m3fn:
            flat = flat.view(torch.uint8)
        assert (_padding(optim, params, flat) == 0).all()


def test_masters_of_f32_parameters_are_not_made(optim):
    assert optim.adamw_state([torch.zeros(3, device=DEV)], master=True).master is None


# ---- lists, layouts, streams, graphs ------------------------------------------------------


@pytest.mark.parametrize("bits", [8, 32])
def test_more_tensors_than_a_launch_takes(optim, bits):
    """250 tensors, some empty, in three launches: as one by one, and counted once."""
    g = _gen(8)
    sizes = [(37 * i) % 401 for i in range(250)]
    params = [_normal(g, (n,)) for n in sizes]
    grads = [_normal(g, (n,)) for n in sizes]
    alone = [p.clone() for p in params]
    st = optim.adamw_state(params, bits=bits)
    n0 = optim.launch_count()
    optim.adamw_step(params, grads, st, lr=1e-2)
    assert optim.launch_count() == n0 + 3 and st.step.tolist() == [1, 0]
    for p, q, gr in zip(params, alone, grads):
        optim.adamw_step([q], [gr], optim.adamw_state([q]), lr=1e-2)
        assert torch.equal(p, q)


def test_nothing_to_step(optim):
    p = torch.zeros(0, device=DEV)
    st = optim.adamw_state([p])
    optim.adamw_step([p], [p.clone()], st, lr=1e-2)
    optim.adamw_step([], [], st, lr=1e-2)
    assert st.step.tolist() == [2, 0]
    st8 = optim.adamw_state([p], bits=8)
    optim.adamw_step([p], [p.clone()], st8, lr=1e-2)
    assert st8.step.tolist() == [1, 0] and optim.adamw_moments(st8)[0].numel() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bits", [8, 32])
def test_starts_that_are_not_aligned(optim, dtype, bits):
    """Views at odd offsets give the bits of aligned ones, and nothing around them changes."""
    g = _gen(9)
    n = 3001
    p, grad = _normal(g, (n,), dtype), _normal(g, (n,), dtype)
    st, st1 = optim.adamw_state([p], bits=bits), optim.adamw_state([p], bits=bits)
    q = p.clone()
    optim.adamw_step([q], [grad], st, lr=1e-2)
    for at_p, at_g in ((1, 0), (0, 3), (5, 2)):
        bp = torch.full((n + 16,), 7.0, device=DEV, dtype=dtype)
        bg = torch.full((n + 16,), float("nan"), device=DEV, dtype=dtype)
        bp[at_p:at_p + n] = p
        bg[at_g:at_g + n] = grad
        for t in st1:
            if t is not None:
                t.view(torch.uint8).zero_() if t.dtype == torch.float8_e4m3fn else t.zero_()
        optim.adamw_step([bp[at_p:at_p + n]], [bg[at_g:at_g + n]], st1, lr=1e-2)
        assert torch.equal(bp[at_p:at_p + n], q)
        assert (bp[:at_p] == 7).all() and (bp[at_p + n:] == 7).all()
        for a, b in zip(st, st1):
            assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_refusals_on_the_device(optim):
    p = torch.zeros((4, 6), device=DEV)
    st = optim.adamw_state([p])
    with pytest.raises(ValueError, match="contiguous"):
        optim.adamw_step([p.T], [p.T], st, lr=1.0)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        optim.adamw_step([p], [p.half()], st, lr=1.0)
    with pytest.raises(ValueError, match="CUDA device"):
        optim.adamw_step([p], [p.cpu()], st, lr=1.0)
    st2 = optim.adamw_state([p, p])
    with pytest.raises(ValueError, match=r"params\[1\] is there twice"):
        optim.adamw_step([p, p], [p.clone(), p.clone()], st2, lr=1.0)
    with pytest.raises(TypeError, match=r"grads\[0\] must be a torch.Tensor"):
        optim.adamw_step([p], [None], st, lr=1.0)
    with pytest.raises(optim.NarrowError, match="DLRM_ERR_ARG"):
        optim.adamw_step([p], [p.clone()], st, lr=1.0, eps=0.0)
    with pytest.raises(optim.NarrowError, match="DLRM_ERR_ARG"):
        optim.adamw_step([p], [p.clone()], st, lr=1.0, betas=(0.9, 1.0))
    assert st.step.tolist() == [0, 0]


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_steps_count_and_follow_the_rate(optim, bits):
    """A captured step replayed three times is three steps, with the rate of its time."""
    g = _gen(10)
    p = _normal(g, (4000,), BF16)
    grad = _normal(g, (4000,))
    rates = [1e-2, 3e-3, 0.0]
    q, st = p.clone(), optim.adamw_state([p], bits=bits, master=True)
    for r in rates:
        optim.adamw_step([q], [grad], st, lr=torch.tensor([r], device=DEV), seed=3)
    st2 = optim.adamw_state([p], bits=bits, master=True)
    lr = torch.zeros(1, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        optim.adamw_step([p], [grad], st2, lr=lr, seed=3)
    assert st2.step.tolist() == [0, 0]
    for r in rates:
        lr.fill_(r)
        graph.replay()
    assert torch.equal(p, q) and st2.step.tolist() == [3, 0]
    for a, b in zip(st, st2):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # the number and the tensor give the same bits where f32 holds the rate
    a, b = q.clone(), q.clone()
    sa, sb = (optim.AdamWState(*[None if x is None else x.clone() for x in st]) for _ in range(2))
    optim.adamw_step([a], [grad], sa, lr=2.0 ** -7)
    optim.adamw_step([b], [grad], sb, lr=torch.full((1,), 2.0 ** -7, device=DEV))
    assert torch.equal(a, b)


def test_two_states_on_two_streams(optim):
    g = _gen(11)
    ps = [_normal(g, (200_000,)) for _ in range(2)]
    grads = [_normal(g, (200_000,)) for _ in range(2)]
    want = []
    for p, gr in zip(ps, grads):
        q = p.clone()
        st = optim.adamw_state([q], bits=8)
        for _ in range(5):
            optim.adamw_step([q], [gr], st, lr=1e-3)
        want.append(q)
    states = [optim.adamw_state([p], bits=8) for p in ps]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, gr, st, s in zip(ps, grads, states, streams):
            with torch.cuda.stream(s):
                optim.adamw_step([p], [gr], st, lr=1e-3)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ps, want))


def test_many_steps_taken_before(optim):
    """The count of a long run: corrections of 1, and of a t in between."""
    p0 = _normal(_gen(12), (300,))
    grad = _normal(_gen(13), (300,))
    for t0 in (0, 9, 1234, 2_000_000_000):
        p, st = p0.clone(), optim.adamw_state([p0])
        st.step[0] = t0
        optim.adamw_step([p], [grad], st, lr=1e-2, betas=(0.9, 0.999))
        z = torch.zeros_like(p0)
        pe, _, _, _, step = _exact(p0, z, z, grad, t0 + 1, 1e-2, 0.9, 0.999, 1e-8, 0.0)
        assert ((p.double() - pe).abs() <= 4 * U * p0.double().abs() + 21 * U * step).all(), t0
        assert st.step[0].item() == t0 + 1


def test_more_elements_than_32_bits_count(optim):
    """A tensor of 2^31 + 999 elements: its end is stepped as it is alone (without random
    rounding, whose bits are the place's)."""
    n = (1 << 31) + 999
    tail = 5000
    p = torch.zeros(n, device=DEV, dtype=BF16)
    grad = torch.zeros(n, device=DEV, dtype=BF16)
    g = _gen(14)
    p[-tail:] = _normal(g, (tail,), BF16)
    grad[-tail:] = _normal(g, (tail,), BF16)
    at = (n - tail) // 256 * 256
    q, gq = p[at:].clone(), grad[at:].clone()
    st = optim.adamw_state([p], bits=8, master=False)
    optim.adamw_step([p], [grad], st, lr=1e-2)
    s1 = optim.adamw_state([q], bits=8)
    optim.adamw_step([q], [gq], s1, lr=1e-2)
    assert torch.equal(st.m_scale[at // 256:], s1.m_scale)
    assert torch.equal(st.v_scale[at // 256:], s1.v_scale)
    assert ((p[at:].float() - q.float()).abs() <= 2.0 ** -7 * q.float().abs()).all()
    assert (p[:at] == 0).all() and (p[at:] != 0).sum() > tail - 100


def test_the_networks_layers_are_stepped_and_served(optim):
    """Steps on the layers that an MLP holds (bf16 weights, f32 biases), by gradients of the
    network; then the same layers in 4 bits."""
    from dlrm_embedding_bag_b200 import fp4, mlp

    g = _gen(15)
    dims = [13, 64, 96, 1]
    layers = []
    for k, n in zip(dims, dims[1:]):
        w = mlp.bf16_empty(n, k)
        w.copy_(_normal(g, (n, k), BF16, k ** -0.5))
        layers.append((w, torch.zeros(n, device=DEV), "relu" if n > 1 else "none"))
    # weights with a pitch are stepped as contiguous copies
    params = [t for w, b, _ in layers for t in (w.contiguous(), b)]
    state = optim.adamw_state(params, bits=8, master=True)
    x, y = _normal(g, (512, 13)), _normal(g, (512, 1))
    for _ in range(3):
        leaves = [p.detach().float().requires_grad_() for p in params]
        h = x
        for i in range(len(dims) - 1):
            h = h @ leaves[2 * i].T + leaves[2 * i + 1]
            if i < len(dims) - 2:
                h = h.relu()
        ((h - y) ** 2).mean().backward()
        before = [p.clone() for p in params]
        optim.adamw_step(params, [l.grad for l in leaves], state, lr=1e-2)
        assert all(not torch.equal(a, b) for a, b in zip(before, params))
    net = mlp.MLP(mlp.fp4_layers([(params[2 * i], params[2 * i + 1], a)
                                  for i, (_, _, a) in enumerate(layers)]), mode="fp4")
    (out, _), inputs = net.forward(x, keep=True)
    assert out.shape == (512, 1) and out.isfinite().all()
    for i, (q, s) in enumerate(inputs):
        assert q.shape == (512, (dims[i] + 1) // 2)
    assert fp4.dequantize_rows(*inputs[0], 13).shape == (512, 13)
