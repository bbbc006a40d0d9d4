"""Steps that go on from a state whose step count the user has set, against the same steps from
one whose second word is zero: equal bits."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def optim():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from dlrm_embedding_bag_b200 import optim as _optim

    return _optim


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype=F32):
    return torch.empty(shape, device=DEV).normal_(0, 1, generator=g).to(dtype)


def _bits(state):
    return [t.view(torch.uint8) if t.element_size() == 1 else t for t in state if t is not None]


# one chunk; a few; fewer chunks than CTAs fit; many more; more tensors than a launch takes
LISTS = [[(5,)], [(3000,), (0,), (1025, 3)], [(300, 1000)], [(4000, 1000), (17,)], [(50 + i,) for i in range(200)]]


@pytest.mark.parametrize("sizes", LISTS, ids=["one", "few", "wave", "many", "launches"])
@pytest.mark.parametrize("bits", [8, 32])
def test_a_count_that_is_set(optim, bits, sizes):
    """Both numbers filled with the count, or counted up or down, or the word left at anything above
    -2^30: every element is stepped once, and the word is zero again."""
    g = _gen(1)
    params = [_normal(g, s, BF16 if i % 2 else F32) for i, s in enumerate(sizes)]
    grads = [_normal(g, s) for s in sizes]

    def run(step):
        ps = [p.clone() for p in params]
        st = optim.adamw_state(ps, bits=bits)
        for i in range(3):
            step(st.step, i)
            optim.adamw_step(ps, grads, st, lr=1e-2)
        return ps, st

    def same(first, second):
        want_p, want = run(first)
        got_p, got = run(second)
        assert all(torch.equal(a, b) for a, b in zip(want_p, got_p))
        assert all(torch.equal(a, b) for a, b in zip(_bits(want), _bits(got)))
        assert got.step[1].item() == 0
        return got.step[0].item()

    for t in (1, 7, 1000, 3907, 2_000_000_000):
        def clean(step, i, t=t):
            if i == 1:
                step.copy_(torch.tensor([t, 0], dtype=torch.int32))

        def filled(step, i, t=t):
            if i == 1:
                step.fill_(t)

        assert same(clean, filled) == t + 2
    # a step that is left out of the count's steps, by a sum over both numbers
    assert same(lambda step, i: step[0].add_(1), lambda step, i: step.add_(1)) == 6
    # a step taken back
    assert same(lambda step, i: step[0].sub_(int(i > 0)), lambda step, i: step.sub_(int(i > 0))) == 1
    for word in (1, 2, 3906, (1 << 31) - 1, -1, -2, -3907, 1 - (1 << 30)):
        assert same(lambda step, i: None, lambda step, i, w=word: step[1].fill_(w)) == 3


def test_a_captured_step_goes_on_from_a_count(optim):
    g = _gen(2)
    p, grad = _normal(g, (200_000,)), _normal(g, (200_000,))
    q = p.clone()
    st, want = optim.adamw_state([p], bits=8), optim.adamw_state([q], bits=8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        optim.adamw_step([p], [grad], st, lr=1e-3)
    st.step.fill_(40)
    want.step[0] = 40
    for _ in range(3):
        graph.replay()
        optim.adamw_step([q], [grad], want, lr=1e-3)
        assert torch.equal(p, q) and st.step.tolist() == want.step.tolist()
    assert st.step.tolist() == [43, 0]


def test_elements_past_the_32_bit_count(optim):
    """A tensor of 2^32 + 777 elements and one behind it in the arena: the first one's end has the scales
    that it has alone, the other (f32, without random rounding) the weights."""
    n, tail = (1 << 32) + 777, 3000
    p, grad = (torch.zeros(n, device=DEV, dtype=BF16) for _ in range(2))
    g = _gen(3)
    p[-tail:], grad[-tail:] = _normal(g, (tail,), BF16), _normal(g, (tail,), BF16)
    w, gw = _normal(g, (700,)), _normal(g, (700,))
    at = (n - tail) // 256 * 256
    q, gq, u = p[at:].clone(), grad[at:].clone(), w.clone()
    st = optim.adamw_state([p, w], bits=8)
    optim.adamw_step([p, w], [grad, gw], st, lr=1e-2)
    alone = optim.adamw_state([q, u], bits=8)
    optim.adamw_step([q, u], [gq, gw], alone, lr=1e-2)
    assert torch.equal(w, u)
    assert torch.equal(st.m_scale[at // 256:], alone.m_scale)
    assert torch.equal(st.v_scale[at // 256:], alone.v_scale)
    # each is one of the two neighbours
    assert ((p[at:].float() - q.float()).abs() <= 2.0 ** -7 * q.float().abs()).all()
    # a zero stays: its block has no moments. (Counted in parts.)
    assert all((part == 0).all() for part in p[:at].split(1 << 30))
    m, _ = optim.adamw_moments(st, dtype=BF16)
    assert all((part == 0).all() for part in m[:at].split(1 << 30))
    one, _ = optim.adamw_moments(alone, dtype=F32)
    # Chance may take the other neighbour: a step, 2^-3 of the larger one (below the least normal code
    # 2^-9 of the scale); and bf16 rounds by 2^-8.
    size = one.abs().view(-1, 256).amax(1, keepdim=True).expand(-1, 256).reshape(-1)
    far, last = (m[at:].float() - one).abs(), m[at:].float().abs()
    assert (far <= (2.0 ** -3 + 2.0 ** -7) * torch.maximum(last, one.abs()) + 2.0 ** -9 * size / 448).all()
