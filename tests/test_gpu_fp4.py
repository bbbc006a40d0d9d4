"""4-bit rows and the 4-bit layer on the GPU, against their definitions in 64 bits.

A scale is a power of two and a scaled element exact, so codes have no tolerance. Of a
layer: products of codes and scales are exact; the f32 sum adds K products in some
order, which tensor cores may cut off instead of round: K 2^-23 of the terms' sizes; bias
and activation round once each, a sigmoid is within 4 of its last places (2^-22) besides
what the sum's error moves it by (its slope is 1/4 at most); a result in bf16 is 2^-8.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
DT = dict(f32=F32, bf16=BF16)
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


@pytest.fixture(scope="module")
def fp4():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from dlrm_embedding_bag_b200 import fp4 as _fp4

    return _fp4


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, rows, cols, dtype=F32, pitch=None, start=0):
    """A matrix whose buffer is NaN around it, its blocks of very different size."""
    pitch = cols if pitch is None else pitch
    buf = torch.full((rows * pitch + start,), float("nan"), device=DEV, dtype=dtype)
    t = buf[start:].view(rows, pitch)[:, :cols]
    v = torch.empty((rows, cols), device=DEV).normal_(0, 1, generator=g)
    t.copy_((v * torch.exp(2 * torch.empty((rows, 1), device=DEV).normal_(0, 1, generator=g))).to(dtype))
    return t


def _scales(fp4, tiles, rows, cols):
    """The tiles' bytes as (rows, blocks), and those of the padding."""
    assert tiles.shape == fp4.scale_shape(rows, cols) and tiles.dtype == torch.uint8
    rt, kt = tiles.shape[:2]
    b = tiles.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)
    n = (cols + 31) // 32
    pad = torch.cat((b[rows:].reshape(-1), b[:rows, n:].reshape(-1)))
    return b[:rows, :n], pad


def _codes_of(q, cols):
    c = torch.stack((q & 15, q >> 4), 2).flatten(1)
    assert c.shape[1] - cols in (0, 1) and (c[:, cols:] == 0).all()
    return c[:, :cols]


def _expect(x):
    """(codes, scale bytes) by the definition: least power of two, nearest level, ties to even."""
    m, k = x.shape
    wide = torch.zeros((m, (k + 31) // 32 * 32), dtype=torch.float64, device=x.device)
    wide[:, :k] = x.double()
    b = wide.view(m, -1, 32)
    top = b.abs().amax(2)
    part, e = torch.frexp(top)
    e = torch.where(top > 0, e - 3 + (part > 0.875).int(), torch.full_like(e, -127)).clamp(min=-127)
    y = (b.abs() / torch.exp2(e.double())[..., None]).view(m, -1)[:, :k]
    far = (y[..., None] - LEVELS.to(x.device)).abs()
    near = far.amin(-1, keepdim=True)
    hit = far == near
    # of two at the same distance, the even code
    code = torch.where(hit.sum(-1) == 1, hit.int().argmax(-1),
                       (hit & (torch.arange(8, device=x.device) % 2 == 0)).int().argmax(-1))
    return code + 8 * (x.double() < 0), e + 127


def _check_rows(fp4, x, q, tiles, what=""):
    m, k = x.shape
    code, byte = _expect(x)
    got, pad = _scales(fp4, tiles, m, k)
    assert torch.equal(got.long(), byte.long()), what
    assert (pad == 0).all(), what
    c = _codes_of(q, k).long()
    # a zero's sign says nothing
    same = (c == code) | ((c % 8 == 0) & (code % 8 == 0))
    assert same.all(), what


SHAPES = [(1, 1), (1, 8), (3, 7), (2, 16), (5, 100), (33, 128), (17, 250), (8, 512), (4, 1000),
          (129, 33), (128, 129), (300, 64), (7, 4096), (2, 5000), (1, 40000), (1, 131072),
          (3000, 24), (700, 130), (9, 2), (255, 31), (257, 592)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_rows(fp4, shape, dtype):
    g = _gen(1)
    m, k = shape
    for pitch, start in ((k, 0), (k + 3, 0), ((k + 15) // 16 * 16, 0), ((k + 7) // 8 * 8 + 8, 8),
                         (k + 1, 1)):
        x = _normal(g, m, k, DT[dtype], pitch, start)
        q, s = fp4.quantize_rows(x)
        assert q.shape == (m, (k + 1) // 2) and (m == 1 or q.stride(0) % 16 == 0)
        _check_rows(fp4, x, q, s, (pitch, start))
        code, byte = _expect(x)
        for out_dtype in (F32, BF16):
            v = fp4.dequantize_rows(q, s, k, dtype=out_dtype)
            sign = 1 - 2 * (code >= 8).double()
            want = sign * LEVELS.to(DEV)[code % 8] * torch.exp2(byte.double() - 127).repeat_interleave(32, 1)[:, :k]
            assert torch.equal(v.double(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_buffers_that_are_given(fp4, dtype):
    """Outputs with pitches and odd starts; what lies beside them stays."""
    g = _gen(2)
    for m, k in ((5, 70), (130, 256), (3, 33)):
        x = _normal(g, m, k, DT[dtype])
        width = (k + 1) // 2
        for pitch, start in ((width + 5, 0), (width + 16, 3)):
            buf = torch.full((m * pitch + start,), 77, device=DEV, dtype=torch.uint8)
            out = buf[start:].view(m, pitch)[:, :width]
            s = torch.full(fp4.scale_shape(m, k), 200, device=DEV, dtype=torch.uint8)
            q, s2 = fp4.quantize_rows(x, out=out, scale_out=s)
            assert q.data_ptr() == out.data_ptr() and s2 is s
            _check_rows(fp4, x, q, s)
            assert (buf[start:].view(m, pitch)[:, width:] == 77).all() and (buf[:start] == 77).all()
            y = torch.full((m, k + 3), 5.0, device=DEV, dtype=DT[dtype])
            v = fp4.dequantize_rows(q, s, k, out=y[:, :k])
            assert torch.equal(v, fp4.dequantize_rows(q, s, k, dtype=DT[dtype]))
            assert (y[:, k:] == 5).all()


@pytest.mark.parametrize("k", [1, 15, 16, 31, 47, 250, 513])
def test_rows_that_start_anywhere(fp4, k):
    """bf16 rows read and written at every offset from 32 bytes, codes at every offset from 8;
    what lies beside them is NaN on the way in and stays on the way out."""
    g = _gen(21)
    m = 19
    for start in range(0, 17):
        pitch = k + start % 5
        x = _normal(g, m, k, BF16, pitch, start)
        code, byte = _expect(x)
        width = (k + 1) // 2
        qbuf = torch.full((m * (width + start % 3) + start + 1,), 77, device=DEV, dtype=torch.uint8)
        q = qbuf[start:].as_strided((m, width), (width + start % 3, 1))
        _, s = fp4.quantize_rows(x, out=q)
        _check_rows(fp4, x, q, s)
        ybuf = torch.full((start + m * (k + 3),), 5.0, device=DEV, dtype=BF16)
        y = ybuf[start:].view(m, k + 3)
        fp4.dequantize_rows(q, s, k, out=y[:, :k])
        sign = 1 - 2 * (code >= 8).double()
        want = sign * LEVELS.to(DEV)[code % 8] * torch.exp2(byte.double() - 127).repeat_interleave(32, 1)[:, :k]
        assert torch.equal(y[:, :k].double(), want)
        assert (y[:, k:] == 5).all() and (ybuf[:start] == 5).all()
        assert (qbuf[:start] == 77).all() and qbuf[-1] == 77


def test_every_level_and_every_tie(fp4):
    """Elements at the levels, halfway between them and next to there, at scales far apart."""
    mids = (LEVELS[1:] + LEVELS[:-1]) / 2
    one = torch.cat((LEVELS, mids, mids * (1 + 2.0 ** -7), mids * (1 - 2.0 ** -7)))
    row = torch.cat((one, torch.zeros(32 - one.numel() % 32, dtype=torch.float64))) if one.numel() % 32 else one
    row = row.view(-1, 32)
    row[:, -1] = 6.0  # the largest: the scale is 1
    row = torch.cat((row.view(1, -1), -row.view(1, -1)))
    for e in (-120, -60, -1, 0, 1, 50, 120):
        x = (row * 2.0 ** e).to(DEV, F32)
        q, s = fp4.quantize_rows(x)
        _check_rows(fp4, x, q, s, e)
        assert torch.equal(fp4.quantize_rows(x.to(BF16))[1], s)


def test_the_largest_of_a_block(fp4):
    """7 times a power of two is brought to 6; the next number above doubles the scale."""
    for v, level, byte in ((7.0, 6.0, 127), (np.nextafter(np.float32(7), np.float32(8)), 4.0, 128),
                           (4.0, 4.0, 127), (3.5, 3.0, 126)):
        x = torch.zeros((1, 32), device=DEV)
        x[0, 5] = float(v)
        q, s = fp4.quantize_rows(x)
        assert _scales(fp4, s, 1, 32)[0].item() == byte
        assert fp4.dequantize_rows(q, s)[0, 5].item() == level * 2.0 ** (byte - 127) if v != 3.5 else True
        _check_rows(fp4, x, q, s, v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("start", [0, 1])
def test_zeros_ends_and_not_finite(fp4, dtype, start):
    """Blocks of zeros, subnormal ones, the largest numbers, and blocks with a NaN or an infinity,
    which are NaN as a whole and leave the others as they are. Both forms of the kernel."""
    x = _normal(_gen(3), 3, 192, DT[dtype], 192 + start, start)
    x[0, 0:32] = 0.0
    x[0, 32:64] = 0.0
    x[0, 40] = -0.0
    x[0, 64:96] *= 1e-38
    x[0, 96:128] = torch.finfo(DT[dtype]).max
    x[0, 128:160] = 0.0
    x[0, 130] = 2.0 ** -133  # a subnormal of either type
    x[0, 131] = 2.0 ** -127
    clean = x.clone()
    x[1, 7], x[1, 70], x[2, 100], x[2, 191] = float("nan"), float("inf"), -float("inf"), float("nan")
    q, s = fp4.quantize_rows(x)
    _check_rows(fp4, x[:1], q[:1], fp4.quantize_rows(x[:1])[1])
    byte = _scales(fp4, s, 3, 192)[0]
    code = _codes_of(q, 192)
    hurt = torch.zeros((3, 6), dtype=torch.bool, device=DEV)
    for r, c in ((1, 7), (1, 70), (2, 100), (2, 191)):
        hurt[r, c // 32] = True
        assert (code[r, c // 32 * 32:c // 32 * 32 + 32] == 0).all()
    assert torch.equal(byte == 255, hurt)
    v = fp4.dequantize_rows(q, s)
    assert torch.equal(v.isnan(), hurt.repeat_interleave(32, 1))
    rest = fp4.dequantize_rows(*fp4.quantize_rows(clean))
    assert torch.equal(v[~v.isnan()], rest[~v.isnan()])


def test_no_rows(fp4):
    q, s = fp4.quantize_rows(torch.empty((0, 40), device=DEV))
    assert q.shape == (0, 20) and s.shape == (0, 1, 512)
    assert fp4.dequantize_rows(q, s).shape == (0, 40)
    w, ws = fp4.quantize_rows(torch.ones((6, 40), device=DEV))
    assert fp4.linear_fp4(q, s, w, ws).shape == (0, 6)


# ---- the layer --------------------------------------------------------------------------------


def _layer(fp4, g, m, k, n, bias, wide=0.0):
    x, w = _normal(g, m, k), _normal(g, n, k)
    if wide:
        x *= torch.exp(wide * torch.empty_like(x).normal_(0, 1, generator=g))
        w *= torch.exp(wide * torch.empty_like(w).normal_(0, 1, generator=g))
    (xq, xs), (wq, ws) = fp4.quantize_rows(x), fp4.quantize_rows(w)
    b = torch.empty(n, device=DEV).normal_(0, 1, generator=g) if bias else None
    return xq, xs, wq, ws, b


def _check_layer(fp4, y, xq, xs, wq, ws, b, act, rows=None):
    x, w = fp4.dequantize_rows(xq, xs).double(), fp4.dequantize_rows(wq, ws).double()
    if rows is not None:
        x, y = x[rows], y[rows]
    k = x.shape[1]
    v, size = x @ w.T, x.abs() @ w.abs().T
    if b is not None:
        v, size = v + b.double(), size + b.double().abs()
    far = (k + 2) * 2.0 ** -23 * size
    if act == "relu":
        v = v.clamp(min=0)
    elif act == "sigmoid":
        v = torch.sigmoid(v)
        far = far / 4 + 2.0 ** -22
    if y.dtype == BF16:
        far = far * (1 + 2.0 ** -8) + 2.0 ** -8 * v.abs()
    assert ((y.double() - v).abs() <= far + 1e-38).all(), ((y.double() - v).abs() - far).max()


# few tokens, one tile of 64 and of 128 tokens, clusters along K, several tiles, pairs, odd
# sizes, a K that ends inside a block, a tile and a stage
LAYERS = [(1, 32, 1), (1, 4096, 300), (2, 77, 130), (3, 1000, 257), (4, 5000, 64), (5, 64, 128),
          (5, 4096, 512), (17, 2048, 512), (64, 64, 128), (65, 96, 129), (100, 592, 512),
          (128, 8192, 128), (200, 300, 1000), (777, 1001, 1234), (2048, 592, 512), (33, 13, 512),
          (2048, 13, 512), (2048, 256, 1), (1500, 2500, 1700), (4096, 700, 4096),
          (5000, 1300, 3000), (20000, 64, 300), (260, 520, 20000), (1, 4096, 9000), (1, 2000, 17),
          (1, 1500, 5001), (1, 9000, 300), (7000, 100, 1001)]


@pytest.mark.parametrize("shape", LAYERS, ids=lambda s: "x".join(map(str, s)))
def test_layer(fp4, shape):
    g = _gen(4)
    m, k, n = shape
    i = LAYERS.index(shape)
    for act, out, bias in ((("none", F32, False), ("relu", BF16, True)) if i % 2 else
                           (("sigmoid", F32, True), ("none", BF16, False), ("relu", F32, True))):
        ops = _layer(fp4, g, m, k, n, bias, wide=1.0 if i % 3 == 0 else 0.0)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        y = fp4.linear_fp4(*ops, act, out_dtype=out, status=status)
        assert y.shape == (m, n) and y.dtype == out and status.item() == 0
        _check_layer(fp4, y, *ops, act)
        assert torch.equal(y, fp4.linear_fp4(*ops, act, out_dtype=out))


@pytest.mark.parametrize("m", [1, 4, 50, 300, 3000])
def test_whole_numbers_are_exact(fp4, m):
    """Products and sums that f32 holds exactly, whatever their order: no part may be lost."""
    g = _gen(5)
    k, n = 2050, 700
    x, w = (torch.randint(-2, 3, (r, k), device=DEV, generator=g).float() for r in (m, n))
    (xq, xs), (wq, ws) = fp4.quantize_rows(x), fp4.quantize_rows(w)
    assert torch.equal(fp4.dequantize_rows(xq, xs), x)
    y = fp4.linear_fp4(xq, xs, wq, ws)
    assert torch.equal(y.double(), x.double() @ w.double().T)


@pytest.mark.parametrize("m", [2, 40, 700])
def test_outputs_with_a_pitch(fp4, m):
    g = _gen(6)
    ops = _layer(fp4, g, m, 400, 333, True)
    for dtype in (F32, BF16):
        buf = torch.full((m, 340), 9.0, device=DEV, dtype=dtype)
        y = fp4.linear_fp4(*ops, "relu", out=buf[:, 5:338])
        assert torch.equal(y, fp4.linear_fp4(*ops, "relu", out_dtype=dtype))
        assert (buf[:, :5] == 9).all() and (buf[:, 338:] == 9).all()


@pytest.mark.parametrize("m,n", [(3000, 2000), (3001, 2011), (4000, 1999)])
def test_large_outputs_with_a_pitch(fp4, m, n):
    """Tiles on their way out as whole lines stop at the output's last column and row."""
    g = _gen(16)
    ops = _layer(fp4, g, m, 300, n, True)
    for dtype in (F32, BF16):
        buf = torch.full((m + 5, 2048), 9.0, device=DEV, dtype=dtype)
        y = fp4.linear_fp4(*ops, "relu", out=buf[:m, 8:8 + n])
        _check_layer(fp4, y, *ops, "relu")
        assert (buf[:, :8] == 9).all() and (buf[:, 8 + n:] == 9).all() and (buf[m:] == 9).all()


@pytest.mark.parametrize("m", [1, 3, 60, 1000])
def test_codes_beside_the_rows_are_not_read(fp4, m):
    """Rows are columns of wider buffers; NaN scales of one token and one channel stay theirs."""
    g = _gen(7)
    k, n = 328, 200  # 164 bytes: rows of 176
    x, w = _normal(g, m, k), _normal(g, n, k)
    xq = torch.full((m, 192), 0x77, device=DEV, dtype=torch.uint8)
    wq = torch.full((n, 208), 0x77, device=DEV, dtype=torch.uint8)
    _, xs = fp4.quantize_rows(x, out=xq[:, :164])
    _, ws = fp4.quantize_rows(w, out=wq[:, 16:180])
    y = fp4.linear_fp4(xq[:, :164], xs, wq[:, 16:180], ws)
    _check_layer(fp4, y, xq[:, :164], xs, wq[:, 16:180], ws, None, "none")
    x[m - 1, 300], w[5, 1] = float("nan"), float("inf")
    _, xs = fp4.quantize_rows(x, out=xq[:, :164])
    _, ws = fp4.quantize_rows(w, out=wq[:, 16:180])
    z = fp4.linear_fp4(xq[:, :164], xs, wq[:, 16:180], ws)
    hurt = torch.zeros_like(z, dtype=torch.bool)
    hurt[m - 1] = True
    hurt[:, 5] = True
    assert torch.equal(z.isnan(), hurt)
    assert torch.equal(z[~hurt], y[~hurt])


@pytest.mark.parametrize("m", [1, 100, 2000])
def test_scales_far_apart(fp4, m):
    """Scales whose product is near 1 although neither is, and sums that leave f32."""
    g = _gen(8)
    k, n = 256, 150
    xi, wi = (torch.randint(-2, 3, (r, k), device=DEV, generator=g).float() for r in (m, n))
    for ex, ew in ((100, -100), (-110, 112), (60, 60), (-60, -60)):
        (xq, xs), (wq, ws) = fp4.quantize_rows(xi * 2.0 ** ex), fp4.quantize_rows(wi * 2.0 ** ew)
        y = fp4.linear_fp4(xq, xs, wq, ws)
        assert torch.equal(y.double(), (xi.double() @ wi.double().T) * 2.0 ** (ex + ew)), (ex, ew)


def test_refusals_on_the_device(fp4):
    from dlrm_embedding_bag_b200 import optim

    x = torch.ones((4, 64), device=DEV)
    q, s = fp4.quantize_rows(x)
    w, ws = fp4.quantize_rows(torch.ones((6, 64), device=DEV))
    with pytest.raises(ValueError, match="scale must be"):
        fp4.dequantize_rows(q, s[:, :, :256].contiguous())
    with pytest.raises(ValueError, match="cols must be"):
        fp4.dequantize_rows(q, s, 62)
    with pytest.raises(ValueError, match="w_q must be"):
        fp4.linear_fp4(q, s, w[:, :16], ws)
    with pytest.raises(ValueError, match="bias must have"):
        fp4.linear_fp4(q, s, w, ws, torch.zeros(4, device=DEV))
    with pytest.raises(TypeError, match="torch.uint8"):
        fp4.linear_fp4(q.to(torch.int8), s, w, ws)
    with pytest.raises(ValueError, match="out must be"):
        fp4.linear_fp4(q, s, w, ws, out=torch.empty((4, 7), device=DEV))
    with pytest.raises(optim.NarrowError, match="DLRM_ERR_ALIGN"):
        fp4.linear_fp4(torch.zeros((4, 33), device=DEV, dtype=torch.uint8)[:, :32], s, w, ws)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        fp4.quantize_rows(x.half())
    with pytest.raises(ValueError, match="unit column stride"):
        fp4.quantize_rows(x.T)


# ---- streams, graphs, large outputs --------------------------------------------------------


def test_captured_and_replayed(fp4):
    """Rows rounded and multiplied inside a graph, on new values at each replay."""
    g = _gen(9)
    w, ws = fp4.quantize_rows(_normal(g, 512, 592))
    for m in (1, 60, 700):
        x = torch.zeros((m, 592), device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            q, s = fp4.quantize_rows(x)
            y = fp4.linear_fp4(q, s, w, ws, act="relu")
        for _ in range(3):
            x.copy_(_normal(g, m, 592))
            graph.replay()
            want = fp4.linear_fp4(*fp4.quantize_rows(x), w, ws, act="relu")
            assert torch.equal(y, want)


def test_first_calls_under_capture():
    """A process whose first calls are captured: nothing in them that a capture refuses."""
    import os
    import subprocess
    import sys

    code = """
import torch
from dlrm_embedding_bag_b200 import fp4, optim
x = [torch.randn((m, 512), device="cuda") for m in (1, 70, 3000)]
w = torch.randn((3000, 512), device="cuda")
p = torch.randn(5000, device="cuda")
st = optim.adamw_state([p], bits=8)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    wq, ws = fp4.quantize_rows(w)
    ys = [fp4.linear_fp4(*fp4.quantize_rows(t), wq, ws) for t in x]
    optim.adamw_step([p], [p.clone()], st, lr=1e-3)
    v = fp4.dequantize_rows(wq, ws)
    m = optim.adamw_moments(st)
g.replay()
torch.cuda.synchronize()
for t, y in zip(x, ys):
    assert torch.equal(y, fp4.linear_fp4(*fp4.quantize_rows(t), wq, ws))
assert st.step.tolist() == [1, 0]
print("fine")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stdout + r.stderr


def test_at_the_same_time(fp4):
    g = _gen(10)
    cases = [_layer(fp4, g, m, 1024, 700, True) for m in (3, 90, 1200)]
    want = [fp4.linear_fp4(*c, "relu") for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(10):
        for out, c, s in zip(got, cases, streams):
            with torch.cuda.stream(s):
                out.append(fp4.linear_fp4(*c, "relu"))
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for ys, w in zip(got, want) for y in ys)


def test_more_outputs_than_32_bits_count(fp4):
    m, k, n = 70000, 64, 33000
    g = _gen(11)
    ops = _layer(fp4, g, m, k, n, False)
    y = fp4.linear_fp4(*ops, out_dtype=BF16)
    _check_layer(fp4, y, *ops, "none", rows=torch.tensor([0, 1, 32767, 65535, 65537, 69999], device=DEV))


def test_rows_beyond_32_bits(fp4):
    m, k = 70000, 33000
    x = torch.empty((m, k), device=DEV, dtype=BF16).normal_(0, 1, generator=_gen(12))
    q, s = fp4.quantize_rows(x)
    v = fp4.dequantize_rows(q, s, dtype=BF16)
    for r in (0, 65000, 69999):
        one, so = fp4.quantize_rows(x[r:r + 1])
        assert torch.equal(one, q[r:r + 1])
        assert torch.equal(fp4.dequantize_rows(one, so, dtype=BF16), v[r:r + 1])


def test_a_row_whose_products_take_longer_than_a_wait(fp4):
    # ones: every partial sum is a multiple of 64 up to 2^30, which f32 holds
    k = 1 << 30
    q = torch.full((2, k // 2), 0x22, device=DEV, dtype=torch.uint8)
    scale = torch.zeros(fp4.scale_shape(2, k), device=DEV, dtype=torch.uint8)
    scale[:, :, :4] = 127
    scale[:, :, 16:20] = 127
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = fp4.linear_fp4(q, scale, q, scale, status=status)
    assert status.item() == 0 and (y == float(k)).all()


# ---- networks -----------------------------------------------------------------------------------


def _net(g, dims, head="none"):
    layers = []
    for k, n in zip(dims, dims[1:]):
        w = torch.empty((n, k), device=DEV).normal_(0, k ** -0.5, generator=g)
        b = torch.empty(n, device=DEV).normal_(0, 0.1, generator=g)
        layers.append((w, b, "relu" if n != dims[-1] else head))
    return layers


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_network_layer_by_layer(fp4, dtype):
    from dlrm_embedding_bag_b200 import mlp

    g = _gen(13)
    layers = mlp.fp4_layers(_net(g, [13, 512, 257, 64]))
    net = mlp.MLP(layers, mode="fp4")
    assert net.out_features == 64
    x = torch.empty((300, 13), device=DEV).normal_(0, 1, generator=g).to(dtype)
    (y32, y16), inputs = net.forward(x, last_bf16=True, keep=True)
    h = x
    for i, (((wq, ws), b, act), (q, s)) in enumerate(zip(layers, inputs)):
        want_q, want_s = fp4.quantize_rows(h)
        assert torch.equal(q, want_q) and torch.equal(s, want_s)
        h = fp4.linear_fp4(q, s, wq, ws, b, act, out_dtype=F32 if i == 2 else BF16)
        _check_layer(fp4, h, q, s, wq, ws, b, act)
    assert torch.equal(y32, h) and torch.equal(y16, h.to(BF16))


def test_whole_forward(fp4):
    from dlrm_embedding_bag_b200 import mlp, ops
    from dlrm_embedding_bag_b200 import synthetic as syn

    g = _gen(14)
    w = syn.TINY
    tables = syn.make_weights(w, DEV)
    idx = torch.from_numpy(syn.make_indices(w)).to(DEV)
    off = torch.from_numpy(syn.make_offsets(w)).to(DEV)
    P = (w.F + 1) * w.F // 2
    bottom = mlp.MLP(mlp.fp4_layers(_net(g, [13, 64, w.D])), mode="fp4")
    top = mlp.MLP(mlp.fp4_layers(_net(g, [w.D + P, 96, 1], "sigmoid")), mode="fp4")
    x = torch.empty((w.B, 13), device=DEV).normal_(0, 1, generator=g).abs()
    ctr, kept = mlp.dlrm_forward(bottom, top, x, tables, idx, off, w.L, keep=True)
    assert ctr.shape == (w.B, 1) and ((ctr > 0) & (ctr < 1)).all()
    dense = bottom.forward(x)[0]
    assert torch.equal(kept["dense32"], dense)
    z = ops.sparse_interact(tables, idx, off, dense, w.L, concat_dense=True)[1]
    assert torch.equal(kept["z"], z)
    assert torch.equal(ctr, top.forward(z)[0])
    with pytest.raises(ValueError, match="same mode"):
        mlp.dlrm_forward(bottom, mlp.MLP(mlp.int8_layers(_net(g, [w.D + P, 1])), mode="int8"), x,
                         tables, idx, off, w.L)
