"""The 8-bit rows, the norm in front of them and the 8-bit layer on the GPU, against 64 bits.

Bounds, with u = 2^-24 (half a step of f32). Of a level v = y / s: h = x + r,
t = h w, 127 / A, the lift and two products round once each, and A carries the
same two roundings as t: at most 8 u relative, |v| <= 127, so a rounded level
lies within 1/2 + 127 * 8 u of the exact one. Of a scale: the squares' sum of K
terms is within (K + 3) u (all terms positive), its root within half of that;
the mean, eps, the root, A, the product and the division round once each: at
most ((K + 3) / 2 + 8) u. Of a layer: the sum is exact, its conversion, two
products and the addition round once each; a rounding to bf16 is 2^-8.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
DT = dict(f32=F32, bf16=BF16)
U = 2.0 ** -24


@pytest.fixture(scope="module")
def int8():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from dlrm_embedding_bag_b200 import int8 as _int8

    return _int8


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, rows, cols, dtype=F32, pitch=None, std=1.0):
    pitch = cols if pitch is None else pitch
    buf = torch.full((rows, pitch), float("nan"), device=DEV, dtype=dtype)
    buf[:, :cols] = torch.empty((rows, cols), device=DEV).normal_(0, std, generator=g).to(dtype)
    return buf[:, :cols]


def _check_rows(q, scale, y, K, what=""):
    """(q, scale) against the exact rows y (64 bits)."""
    s = y.abs().amax(1) / 127.0
    assert ((scale.double() - s).abs() <= ((K + 3) / 2 + 8) * U * s).all(), what
    live = s > 0
    v = y[live] / s[live][:, None]
    assert ((q[live].double() - v).abs() <= 0.5 + 127 * 8 * U).all(), what
    assert (q[~live] == 0).all() and (q.to(torch.int16).abs() <= 127).all(), what


SHAPES = [(1, 1), (1, 8), (3, 7), (2, 16), (5, 100), (33, 128), (17, 250), (8, 512), (4, 1000),
          (3, 1024), (2, 2048), (7, 4096), (2, 4104), (2, 5000), (1, 8192), (2, 16384),
          (1, 40000), (1, 131072), (3000, 24), (700, 130), (9, 2), (6, 129), (5, 255), (4, 1026),
          (3, 2046), (3, 2049), (2, 4097), (2, 8193), (2, 8194), (1, 16386), (1, 20001)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quantize_rows(int8, M, K, dt):
    g = _gen(M + K)
    x = _normal(g, M, K, DT[dt], std=3.0)
    q, s = int8.quantize_rows(x)
    assert q.dtype == torch.int8 and q.shape == (M, K) and s.shape == (M,)
    _check_rows(q, s, x.double(), K)


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("residual,weight", [(True, True), (False, True), (True, False)])
def test_rms_norm(int8, M, K, dt, residual, weight):
    g = _gen(M + K)
    x = _normal(g, M, K, DT[dt])
    r = _normal(g, M, K, DT[dt], std=2.0) if residual else None
    w = torch.empty(K, device=DEV).normal_(1, 0.3, generator=g) if weight else None
    q, s, h = int8.rms_norm_int8(x, w, residual=r, eps=1e-5)
    hd = x.double() + (r.double() if residual else 0.0)
    y = hd / torch.sqrt(hd.square().mean(1, keepdim=True) + np.float64(np.float32(1e-5)))
    _check_rows(q, s, y * (w.double() if weight else 1.0), K)
    if residual:
        assert torch.equal(h, (x.float() + r.float()).to(DT[dt]))
    else:
        assert h is None


@pytest.mark.parametrize("pitch", [104, 112, 101, 100, 102])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K", [100, 96, 97])
def test_norm_strides_in_place_and_what_is_left_alone(int8, pitch, dt, K):
    g = _gen(pitch + K)
    M = 19
    x = _normal(g, M, K, DT[dt], pitch)
    r = _normal(g, M, K, DT[dt], pitch)
    w = torch.empty(K, device=DEV).normal_(1, 0.3, generator=g)
    want = (x.float() + r.float()).to(DT[dt])
    hd = x.double() + r.double()
    buf = torch.full((M + 1, 128), 99, device=DEV, dtype=torch.int8)
    scales = torch.full((M + 1,), -1.0, device=DEV)
    q, s, h = int8.rms_norm_int8(x, w, residual=r, out=buf[:M, :K], scale_out=scales[:M],
                                 residual_out=r)
    assert h is r and torch.equal(r, want)
    y = hd / torch.sqrt(hd.square().mean(1, keepdim=True) + 1e-6) * w.double()
    _check_rows(q, s, y, K)
    assert (buf[:, K:] == 99).all() and (buf[M] == 99).all() and float(scales[M]) == -1.0
    base = torch.as_strided(r, (M, pitch), (pitch, 1))
    assert torch.isnan(base[:, K:].float()).all()


@pytest.mark.parametrize("K", [64, 4096, 20000, 66, 1001, 20001])
def test_rows_of_zeros_tiny_huge_and_not_finite(int8, K):
    g = _gen(K)
    x = _normal(g, 9, K)
    x[0] = 0.0
    x[1] *= 1e-30            # squares vanish
    x[2] *= 1e25             # squares leave f32
    x[3, K // 2] = float("inf")
    x[4, K - 1] = float("nan")
    x[5, 0] = -float("inf")
    x[6] = 0.0
    x[6, K - 1] = 1e-44      # a subnormal alone
    x[7] = torch.finfo(F32).max
    for eps in (0.0, 1e-6):
        q, s, _ = int8.rms_norm_int8(x, eps=eps)
        bad = torch.tensor([3, 4, 5], device=DEV)
        assert torch.isnan(s[bad]).all() and (q[bad] == 0).all()
        assert torch.isnan(int8.dequantize_rows(q, s)[bad]).all()
        good = torch.tensor([0, 1, 2, 7, 8], device=DEV)
        y = x[good].double()
        y = y / torch.sqrt(y.square().mean(1, keepdim=True) + np.float64(np.float32(eps))
                           + (y == 0).all(1, keepdim=True))
        _check_rows(q[good], s[good], y, K, f"eps={eps}")
        assert int(q[6, K - 1]) == 127 and (q[6, :K - 1] == 0).all()
        if eps == 0.0:  # a row with one value: its norm is sqrt(K)
            assert abs(float(s[6]) * 127 - K ** 0.5) <= K ** 0.5 * 64 * U
    q, s = int8.quantize_rows(x)
    good = torch.tensor([0, 1, 2, 7, 8], device=DEV)
    _check_rows(q[good], s[good], x[good].double(), K)
    assert torch.isnan(s[3:6]).all() and int(q[6, K - 1]) == 127


@pytest.mark.parametrize("K", [5, 64, 1000, 6924, 20001])
def test_eps_that_leaves_f32_with_the_squares(int8, K):
    # the mean of the squares and eps are finite, their sum is not
    x = _normal(_gen(K), 6, K).clamp(-8, 8) * 1e19 / 8
    x[1] = 1.5e19
    x[2] *= 1e-19
    for eps in (3e38, 1e-29, 1e-31):
        q, s, _ = int8.rms_norm_int8(x, eps=eps)
        y = x.double()
        y = y / torch.sqrt(y.square().mean(1, keepdim=True) + np.float64(np.float32(eps)))
        _check_rows(q, s, y, K, f"eps={eps}")


@pytest.mark.parametrize("K", [5, 64, 1000, 1001, 4096, 6924, 20000, 20001])
@pytest.mark.parametrize("M", [9, 700])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1.0, 1e20, 1e-20, 1e-35])
@pytest.mark.parametrize("residual", [False, True])
def test_products_with_the_weight_that_leave_f32(int8, K, M, dt, size, residual):
    """Finite rows, weights and normed rows, with h * weight above f32's largest value
    or among its subnormals and zeros: q and scale hold y all the same. (x and residual
    do not overlap, so h is exact. A scale among f32's subnormals is off by half of
    their step, 2^-150, besides.)"""
    g = _gen(K + M)
    w = torch.empty(K, device=DEV).normal_(1, 0.3, generator=g) * size
    w[K // 2] = 0.0
    x = _normal(g, M, K).clamp(-4, 4)
    for i, f in enumerate((8e37, 1e30, 1e-10, 1e-25, 1e-30, 1e-38)):
        x[i] *= f
    x[6] = 0.0
    x[7] = 0.0
    x[7, 1] = 3e5        # one value, at a weight
    x[8] = 0.0
    x[8, K // 2] = 2.0   # ... and where the weight is zero
    x = x.to(DT[dt])
    r = None
    if residual:
        odd = torch.arange(K, device=DEV) % 2 == 1
        r = torch.where(odd, x, torch.zeros_like(x))
        x = torch.where(odd, torch.zeros_like(x), x)
    h = x.double() + (r.double() if residual else 0.0)
    for eps in (0.0, 1e-6):
        q, s, total = int8.rms_norm_int8(x, w, residual=r, eps=eps)
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + np.float64(np.float32(eps))
                           + (h == 0).all(1, keepdim=True))
        y = y * w.double()
        exact = y.abs().amax(1) / 127.0
        assert ((s.double() - exact).abs() <= ((K + 3) / 2 + 8) * U * exact + 2.0 ** -149).all()
        live = exact > 0
        v = y[live] / exact[live][:, None]
        assert ((q[live].double() - v).abs() <= 0.5 + 127 * 8 * U).all()
        assert (q[~live] == 0).all() and (s[~live] == 0).all()
        if residual:
            assert torch.equal(total.double(), h)
    if residual:  # the sum over its own residual: a row is read before it is written
        q2, s2, h2 = int8.rms_norm_int8(x, w, residual=r, residual_out=r, eps=1e-6)
        assert h2 is r and torch.equal(r.double(), h)
        assert torch.equal(q2, q) and torch.equal(s2, s)
    x[0, K - 1] = float("inf")
    x[1, 0] = float("nan")
    x[2, K // 2] = -float("inf")
    q, s, _ = int8.rms_norm_int8(x, w)
    assert torch.isnan(s[:3]).all() and (q[:3] == 0).all() and not torch.isnan(s[3:]).any()


def test_values_of_rows(int8):
    g = _gen(4)
    for M, K in ((1, 1), (5, 16), (40, 100), (3, 4099), (7, 1026), (2, 2), (300, 33)):
        q, s = int8.quantize_rows(_normal(g, M, K))
        exact = q.double() * s.double()[:, None]
        for dt in (F32, BF16):
            v = int8.dequantize_rows(q, s, dtype=dt)
            half = torch.finfo(dt).eps / 2
            assert ((v.double() - exact).abs() <= (half + U) * exact.abs()).all()


def test_empty_batches(int8):
    x = torch.empty((0, 32), device=DEV)
    q, s = int8.quantize_rows(x)
    assert q.shape == (0, 32) and s.shape == (0,)
    w, ws = int8.quantize_rows(torch.ones((5, 32), device=DEV))
    assert int8.linear_int8(q, s, w, ws).shape == (0, 5)
    assert int8.dequantize_rows(q, s).shape == (0, 32)


@pytest.mark.parametrize("K", [1, 32, 33, 592, 1001])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_empty_batches_of_any_width(int8, K, dt):
    """Through the norm, the layer and a network: no rows in, no rows out."""
    from dlrm_embedding_bag_b200 import mlp

    x = torch.empty((0, K), device=DEV, dtype=DT[dt])
    w, ws = int8.quantize_rows(torch.ones((5, K), device=DEV))
    for q, s, h in ((*int8.quantize_rows(x), None),
                    int8.rms_norm_int8(x, torch.ones(K, device=DEV), residual=x)):
        assert q.shape == (0, K) and s.shape == (0,)
        assert h is None or (h.shape == (0, K) and h.dtype == x.dtype)
        assert int8.linear_int8(q, s, w, ws, ws, "relu", out_dtype=x.dtype).shape == (0, 5)
        # a buffer of the binding's own making, as a caller keeps it between batches
        assert int8.linear_int8(int8.int8_empty(0, K), s, w, ws).shape == (0, 5)
    net = mlp.MLP(mlp.int8_layers(_weights(_gen(1), [K, 37, 3])), mode="int8")
    y32, y16 = net.forward(x, last_bf16=True)
    assert y32.shape == (0, 3) and y16.shape == (0, 3)


# ------------------------------------------------------------------------- layer


def _ints(g, rows, cols, lo=-127, hi=127, extra=0):
    pitch = (cols + 15) // 16 * 16 + extra
    buf = torch.full((rows, pitch), 77, device=DEV, dtype=torch.int8)
    buf[:, :cols] = torch.randint(lo, hi + 1, (rows, cols), device=DEV, generator=g).to(torch.int8)
    return buf[:, :cols]


def _check_layer(y, xq, xs, wq, ws, bias, act, rows=None):
    if rows is not None:
        y, xq, xs = y[rows], xq[rows], xs[rows]
    acc = xq.double() @ wq.double().T  # exact: below 2^53
    z = acc * xs.double()[:, None] * ws.double()
    mag = z.abs()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    tol = 5 * U * mag
    if act == "relu":
        z = z.clamp(min=0)
    elif act == "sigmoid":
        z = 1 / (1 + torch.exp(-z))
        # slope at most 1/4; the exponential, the sum and the quotient: a few steps more
        tol = tol / 4 + 8 * U * z
    half = torch.finfo(y.dtype).eps / 2 if y.dtype != F32 else 0.0
    tol = tol * (1 + half) + half * z.abs()
    err = (y.double() - z).abs()
    assert (err <= tol).all(), float((err - tol).max())


def _layer(int8, M, N, K, act="none", bias=True, dt=F32, seed=0, extra=0, rows=None, out=None):
    g = _gen(M * 7 + N * 3 + K + seed)
    xq, wq = _ints(g, M, K, extra=extra), _ints(g, N, K, lo=-128, extra=extra)
    xs = torch.empty(M, device=DEV).uniform_(0.001, 0.1, generator=g)
    ws = torch.empty(N, device=DEV).uniform_(0.001, 0.1, generator=g) / K ** 0.5
    b = torch.empty(N, device=DEV).normal_(0, 0.5, generator=g) if bias else None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = int8.linear_int8(xq, xs, wq, ws, b, act, out_dtype=dt, out=out, status=status)
    assert int(status) == 0
    _check_layer(y, xq, xs, wq, ws, b, act, rows)
    return y


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 33, 64, 65, 100, 129, 257])
@pytest.mark.parametrize("N,K", [(1, 1), (7, 16), (64, 64), (130, 100), (33, 129), (300, 592),
                                 (128, 1000)])
def test_linear_shapes(int8, M, N, K):
    _layer(int8, M, N, K, dt=F32 if (M + N) % 2 else BF16)


@pytest.mark.parametrize("act", ["none", "relu", "sigmoid"])
@pytest.mark.parametrize("M", [1, 6, 200])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_linear_activations_and_types(int8, act, M, bias, dt):
    _layer(int8, M, 150, 200, act=act, bias=bias, dt=DT[dt])


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (4, 5000, 2100), (20, 2048, 8192),
                                   (2048, 592, 512), (1000, 1000, 1000), (5000, 512, 592),
                                   (300, 9000, 272), (4096, 4096, 256), (3001, 2999, 1037)])
def test_linear_larger(int8, M, N, K):
    rows = torch.from_numpy(np.random.default_rng(M).choice(M, min(M, 200), replace=False)).to(DEV)
    _layer(int8, M, N, K, act="relu", rows=rows, dt=BF16)
    _layer(int8, M, N, K, rows=rows)


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("K", [131071, 60000])
def test_linear_longest_sums_are_exact(int8, M, K):
    """All products 2^14: the largest sum that int32 has to hold."""
    xq = int8.int8_empty(M, K)
    wq = int8.int8_empty(3, K)
    xq.fill_(-128)
    wq.fill_(-128)
    wq[1].fill_(127)
    ones = torch.ones(M, device=DEV)
    y = int8.linear_int8(xq, ones, wq, torch.ones(3, device=DEV))
    want = torch.tensor([K * 16384, -K * 16256, K * 16384], dtype=torch.float64)
    assert torch.equal(y.cpu(), want.float().expand(M, 3))


@pytest.mark.parametrize("M", [1, 5, 90, 400])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_linear_pitches_and_what_is_left_alone(int8, M, dt):
    for N, pitch, offset in ((100, 100, 0), (100, 112, 0), (100, 111, 0), (99, 128, 3),
                             (260, 264, 1)):
        buf = torch.full(((M + 1) * pitch + offset,), float("nan"), device=DEV, dtype=DT[dt])
        rows = buf[offset:].view(M + 1, pitch)
        _layer(int8, M, N, 200, act="relu", dt=DT[dt], extra=32, out=rows[:M, :N])
        rows[:M, :N] = float("nan")
        assert torch.isnan(buf.float()).all()


def test_linear_one_row_of_any_pitch(int8):
    """The pitch of a single row (of x, or of w) is never used to find another."""
    g = _gen(8)
    xq = torch.randint(-127, 128, (1, 37), device=DEV, generator=g).to(torch.int8)
    wq = torch.randint(-127, 128, (1, 37), device=DEV, generator=g).to(torch.int8)
    y = int8.linear_int8(xq, torch.ones(1, device=DEV), wq, torch.ones(1, device=DEV))
    assert float(y) == float(xq.double() @ wq.double().T)


def test_linear_scales_that_are_not_finite(int8):
    """A row that could not be rounded (scale NaN, levels 0) stays NaN, through ReLU too."""
    xq = torch.zeros((3, 16), dtype=torch.int8, device=DEV)
    xs = torch.tensor([1.0, float("nan"), 0.0], device=DEV)
    wq = torch.ones((20, 16), dtype=torch.int8, device=DEV)
    for act in ("none", "relu", "sigmoid"):
        y = int8.linear_int8(xq, xs, wq, torch.ones(20, device=DEV), None, act)
        assert torch.isnan(y[1]).all() and not torch.isnan(y[[0, 2]]).any()


def test_streams_and_graphs(int8):
    """The norm and the layer captured together and replayed with new inputs."""
    g = _gen(12)
    for M in (1, 50, 300):
        x = _normal(g, M, 512, BF16)
        r = _normal(g, M, 512, BF16)
        w = torch.ones(512, device=DEV)
        wq, ws = int8.quantize_rows(_normal(g, 256, 512))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q, s, _ = int8.rms_norm_int8(x, w, residual=r)
            y = int8.linear_int8(q, s, wq, ws)
        side.synchronize()
        _check_layer(y, q, s, wq, ws, None, "none")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q, s, _ = int8.rms_norm_int8(x, w, residual=r)
            y = int8.linear_int8(q, s, wq, ws)
        x.mul_(-3.0)
        graph.replay()
        torch.cuda.synchronize()
        hd = x.double() + r.double()
        _check_rows(q, s, hd / torch.sqrt(hd.square().mean(1, keepdim=True) + 1e-6), 512)
        _check_layer(y, q, s, wq, ws, None, "none")


@pytest.mark.parametrize("M", [1, 2, 4, 20, 300, 2000])
@pytest.mark.parametrize("N,K", [(256, 512), (700, 4096)])
def test_layer_waits_for_what_the_kernel_before_it_writes(int8, M, N, K):
    """A bf16 layer lets the kernel behind it start before it ends: an 8-bit layer whose
    scales and bias are the last rows of its output gets them all the same, and so for
    weights and rows that a rounding has just written."""
    from dlrm_embedding_bag_b200 import mlp

    g = _gen(M + N + K)
    rows, width = 60000, max(M, N)
    a, b = _normal(g, rows, 64, BF16), _normal(g, width, 64, BF16)
    y = torch.empty((rows, width), device=DEV)
    w, x = _normal(g, N, K), _normal(g, M, K)
    wq, xq = int8.int8_empty(N, K), int8.int8_empty(M, K)
    scale = torch.empty(max(M, N), device=DEV)
    for k in range(3):
        y.fill_(float("nan"))
        wq.fill_(99)
        xq.fill_(77)
        a.mul_(-0.5)
        w.mul_(-0.5)
        int8.quantize_rows(x, out=xq, scale_out=scale[:M])
        int8.quantize_rows(w, out=wq, scale_out=scale[:N])
        mlp.linear_bf16(a, b, out_f32=y)
        got = int8.linear_int8(xq, y[-1, :M], wq, y[-2, :N], y[-3, :N])
        int8.quantize_rows(w, out=wq, scale_out=scale[:N])
        again = int8.linear_int8(xq, y[-1, :M], wq, y[-2, :N], y[-3, :N])
        torch.cuda.synchronize()
        _check_layer(got, xq, y[-1, :M].clone(), wq, y[-2, :N].clone(), y[-3, :N].clone(), "none")
        assert torch.equal(got, again)


# ------------------------------------------------------------------ whole networks


def _weights(g, widths):
    out = []
    for k, n in zip(widths, widths[1:]):
        w = torch.empty((n, k), device=DEV).normal_(0, k ** -0.5, generator=g)
        out.append((w, torch.empty(n, device=DEV).normal_(0, 0.1, generator=g), "relu"))
    return out


@pytest.mark.parametrize("M", [1, 3, 70, 500])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_mlp_of_int8_layers(int8, M, dt):
    """Every layer of a network against 64 bits on the inputs that the kernels gave it:
    plain rounding, a norm, and a residual stack of three normed layers."""
    from dlrm_embedding_bag_b200 import mlp

    g = _gen(M)
    widths = [200, 96, 96, 96, 96, 33]
    layers = mlp.int8_layers(_weights(g, widths))
    norms = [None] + [torch.empty(96, device=DEV).normal_(1, 0.2, generator=g) for _ in range(4)]
    net = mlp.MLP(layers, mode="int8", norms=norms, eps=1e-5)
    assert net.out_features == 33
    x = _normal(g, M, 200, DT[dt])
    (y32, y16), inputs = net.forward(x, last_bf16=True, keep=True)
    h, total = x, None
    for i, (((wq, ws), b, act), (q, s)) in enumerate(zip(layers, inputs)):
        rows = h.double()
        if norms[i] is not None:
            if total is not None:
                rows = rows + total.double()
                total = rows.float().to(BF16)  # the running sum, rounded once
            else:
                total = h
            rows = rows / torch.sqrt(rows.square().mean(1, keepdim=True)
                                     + np.float64(np.float32(1e-5))) * norms[i].double()
        _check_rows(q, s, rows, rows.shape[1], f"layer {i}")
        last = i == len(layers) - 1
        h = y32 if last else int8.linear_int8(q, s, wq, ws, b, act, out_dtype=BF16)
        _check_layer(h, q, s, wq, ws, b, act)
    assert y32.shape == (M, 33) and torch.equal(y16.float(), y32.to(BF16).float())
    y, none = net.forward(x)
    assert none is None and torch.equal(y, y32)
    none, yb = net.forward(x, last_f32=False, last_bf16=True)
    assert none is None and yb.dtype == BF16 and torch.equal(yb.float(), y32.to(BF16).float())


@pytest.mark.parametrize("M", [0, 1, 70])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("widths", [[96] * 5, [40, 40, 40, 33, 33, 33]])
def test_residual_stack_that_begins_with_the_input(int8, M, dt, widths):
    """Norms on every layer: the stack starts at the input, whatever the input's type.
    Where widths change it starts again."""
    from dlrm_embedding_bag_b200 import mlp

    g = _gen(M + len(widths))
    layers = mlp.int8_layers(_weights(g, widths))
    norms = [torch.empty(k, device=DEV).normal_(1, 0.2, generator=g) for k in widths[:-1]]
    net = mlp.MLP(layers, mode="int8", norms=norms)
    x = _normal(g, M, widths[0], DT[dt])
    (y, _), inputs = net.forward(x, keep=True)
    assert y.shape == (M, widths[-1])
    h, total = x, None
    for i, (((wq, ws), b, act), (q, s)) in enumerate(zip(layers, inputs)):
        rows = h.double()
        if total is not None and total.shape == h.shape:
            rows = rows + total.double()
        total = rows.float().to(BF16)  # the running sum, rounded once
        rows = rows / torch.sqrt(rows.square().mean(1, keepdim=True)
                                 + np.float64(np.float32(1e-6))) * norms[i].double()
        if M:
            _check_rows(q, s, rows, rows.shape[1], f"layer {i}")
        h = int8.linear_int8(q, s, wq, ws, b, act, out_dtype=BF16)


def test_dlrm_forward_in_int8(int8):
    """The whole forward on 8-bit layers: each stage against 64 bits on its own
    inputs, and the captured graph against the eager call."""
    from dlrm_embedding_bag_b200 import mlp, ops

    g = _gen(77)
    B, F, N, D, L = 300, 5, 400, 32, 4
    P = (F + 1) * F // 2
    bottom = mlp.MLP(mlp.int8_layers(_weights(g, [13, 64, D])), mode="int8")
    tops = _weights(g, [D + P, 48, 1])
    tops[-1] = (*tops[-1][:2], "sigmoid")
    top = mlp.MLP(mlp.int8_layers(tops), mode="int8")
    tables = [torch.empty((N, D), device=DEV).normal_(0, 0.3, generator=g) for _ in range(F)]
    idx = torch.randint(0, N, (F, B * L), device=DEV, generator=g).to(torch.int32)
    off = (torch.arange(B, device=DEV, dtype=torch.int32) * L).repeat(F, 1).contiguous()
    x = _normal(g, B, 13).abs()
    ctr, t = mlp.dlrm_forward(bottom, top, x, tables, idx, off, L, keep=True)
    assert ctr.shape == (B, 1) and ((ctr > 0) & (ctr < 1)).all()
    assert torch.equal(t["z"][:, :D], t["dense32"])
    dense, pooled = t["dense32"].double(), t["pooled"].double()
    v = torch.cat([dense[:, None], pooled], 1)
    i, j = torch.tril_indices(F + 1, F + 1, -1, device=DEV)
    dots = (v[:, i] * v[:, j]).sum(2)
    bound = (v[:, i] * v[:, j]).abs().sum(2)
    assert ((t["z"][:, D:].double() - dots).abs() <= 1e-5 * bound + 1e-30).all()
    q, s = t["top_inputs"][0]
    _check_rows(q, s, t["z"].double(), D + P)
    q, s = t["top_inputs"][1]
    (wq, ws), b, act = top.layers[1]
    _check_layer(ctr, q, s, wq, ws, b, act)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = mlp.dlrm_forward(bottom, top, x, tables, idx, off, L)
    x.mul_(0.5)
    idx.copy_((idx + 7) % N)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, mlp.dlrm_forward(bottom, top, x, tables, idx, off, L))
    assert not torch.equal(again, ctr)
    with pytest.raises(ValueError, match="same mode"):
        mlp.dlrm_forward(bottom, mlp.MLP([(tables[0].to(BF16), None, "none")], mode="bf16"), x,
                         tables, idx, off, L)
    assert ops.launch_count() > 0


def test_mlp_refusals(int8):
    from dlrm_embedding_bag_b200 import mlp

    w = torch.zeros((8, 16), device=DEV)
    layers = [(w, None, "none")]
    with pytest.raises(ValueError, match="w_q, w_scale"):
        mlp.MLP(layers, mode="int8")
    with pytest.raises(ValueError, match="mode must be"):
        mlp.MLP(layers, mode="int4")
    with pytest.raises(ValueError, match="norms need"):
        mlp.MLP(layers, norms=[None])
    with pytest.raises(ValueError, match="1 entries"):
        mlp.MLP(mlp.int8_layers(layers), mode="int8", norms=[None, None])
    net = mlp.MLP(mlp.int8_layers(layers), mode="int8")
    with pytest.raises(ValueError, match="one input"):
        net.forward(torch.zeros((4, 8), device=DEV), a_hi=torch.zeros((4, 8), device=DEV))


def test_lookup_norm_layer_and_gradient_together(int8):
    """A step over token histories: rows looked up with a scale, normed into 8
    bits, multiplied; and the table's gradient from the rows' own gradients, each
    against 64 bits on the inputs that it was given."""
    from dlrm_embedding_bag_b200 import tokens

    g = _gen(5)
    N, D, out = 500, 256, 64
    table = _normal(g, N, D, BF16, std=0.1)
    ids = torch.randint(0, N, (20, 30), device=DEV, generator=g).to(torch.int32)
    ids[:, 25:] = 0  # padding
    wq, ws = int8.quantize_rows(_normal(g, out, D, std=D ** -0.5))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rows = tokens.embedding_lookup(table, ids, scale=16.0, padding_idx=0).view(-1, D)
        q, s, h = int8.rms_norm_int8(rows, residual=rows)
        y = int8.linear_int8(q, s, wq, ws)
        grad = tokens.embedding_grad(rows, ids, N, scale=16.0, padding_idx=0)
    side.synchronize()
    want = table[ids.view(-1).long()].float() * 16.0
    want[ids.view(-1) == 0] = 0
    assert torch.equal(rows, want.to(BF16))
    hd = 2 * rows.double()
    _check_rows(q, s, hd / torch.sqrt(hd.square().mean(1, keepdim=True) + 1e-6), D)
    assert torch.equal(h, rows * 2) and (q[ids.view(-1) == 0] == 0).all()
    _check_layer(y, q, s, wq, ws, None, "none")
    ref = torch.zeros((N, D), dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref)
    ref.index_add_(0, ids.view(-1).long(), rows.double() * 16)
    mag.index_add_(0, ids.view(-1).long(), rows.double().abs() * 16)
    ref[0] = mag[0] = 0
    tol = 60 * U * mag + 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8)
    assert ((grad.double() - ref).abs() <= tol).all()


def test_refusals(int8):
    from dlrm_embedding_bag_b200.tokens import TokensError

    q = torch.zeros((4, 32), dtype=torch.int8, device=DEV)
    s = torch.ones(4, device=DEV)
    with pytest.raises(ValueError, match="w_q must be"):
        int8.linear_int8(q, s, q[:, :16], s)
    with pytest.raises(ValueError, match="x_scale"):
        int8.linear_int8(q, s[:3], q, s)
    with pytest.raises(TypeError, match="int8"):
        int8.linear_int8(q.to(torch.uint8), s, q, s)
    with pytest.raises(TokensError, match="DLRM_ERR_ALIGN"):
        int8.linear_int8(q[:, 1:17], s, q[:, :16], s)
    with pytest.raises(TokensError, match="DLRM_ERR_ALIGN"):
        odd = torch.zeros((4, 24), dtype=torch.int8, device=DEV)
        int8.linear_int8(odd, s, odd, s)
    with pytest.raises(TokensError, match="DLRM_ERR_SHAPE"):
        long = torch.zeros((1, 131072), dtype=torch.int8, device=DEV)
        int8.linear_int8(long, s[:1], long, s[:1])
    x = torch.zeros((4, 32), device=DEV)
    with pytest.raises(ValueError, match="residual must be"):
        int8.rms_norm_int8(x, residual=x.to(BF16))
    with pytest.raises(ValueError, match="weight"):
        int8.rms_norm_int8(x, s)
    with pytest.raises(ValueError, match="residual_out needs"):
        int8.rms_norm_int8(x, residual_out=x)
    with pytest.raises(TokensError, match="DLRM_ERR_ARG"):
        int8.rms_norm_int8(x, eps=-1.0)
    with pytest.raises(ValueError, match="overlap"):
        int8.quantize_rows(x[:1].expand(4, 32))
