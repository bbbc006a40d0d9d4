"""The library of the optimiser step and the 4-bit layers on the CPU: it loads, exports
exactly what its headers declare, and refuses bad arguments before any CUDA call (no
call here reaches a kernel launch)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = [os.path.join(ROOT, "include", h) for h in ("dlrm_optim.h", "dlrm_fp4.h")]
OK, NULL, SHAPE, ALIGN, ARG = 0, -1, -2, -3, -9
A, W, Y, S = 0x10000, 0x20000, 0x30000, 0x40000  # aligned, never dereferenced
BIG = 1 << 31
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def optim():
    from dlrm_embedding_bag_b200 import build

    build.build()
    from dlrm_embedding_bag_b200 import optim as _optim

    return _optim


def _declarations():
    out = {}
    for h in HEADERS:
        src = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        for ret, name, params in re.findall(r"DLRM_API\s+([\w\s\*]+?)\b(\w+)\s*\(([^)]*)\)\s*;",
                                            src):
            plist = [] if params.strip() in ("", "void") else [p.strip() for p in params.split(",")]
            out[name] = (ret.strip(), [re.sub(r"\s*\b\w+$", "", p) for p in plist])
    return out


def test_exports_are_what_the_headers_declare(optim):
    out = subprocess.run(["nm", "-D", "--defined-only", optim.LIBRARY], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert exported == set(_declarations()) == set(optim.SIGNATURES)


def test_signatures_match_the_headers(optim):
    kinds = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "double": ctypes.c_double,
             "uint32_t": ctypes.c_uint32}
    for name, (ret, params) in _declarations().items():
        res, args = optim.SIGNATURES[name]
        want = [ctypes.c_void_p if "*" in p or p == "dlrm_stream_t" else kinds[p] for p in params]
        assert args == want, name
        assert res is kinds[ret], name


def test_headers_compile_as_c(tmp_path, optim):
    probe = tmp_path / "probe.c"
    probe.write_text('#include <stdio.h>\n#include "dlrm_optim.h"\n#include "dlrm_fp4.h"\n'
                     'int main(void) { printf("%d %d\\n", DLRM_ADAMW_BLOCK, DLRM_FP4_BLOCK); '
                     'return 0; }\n')
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(probe), "-o", str(exe)], check=True)
    from dlrm_embedding_bag_b200 import fp4

    said = subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()
    assert [int(v) for v in said] == [optim.BLOCK, fp4.BLOCK]


def test_missing_library_fails_loudly(optim, tmp_path):
    with pytest.raises(ImportError, match="no CPU fallback"):
        optim.load_library(str(tmp_path / "libdlrm_narrow.so"))


def _step(optim, n=2, params=(A, W), grads=(Y, S), counts=(300, 7), pd=(0, 1), gd=(0, 0),
          decays=None, bits=32, m=A, v=W, ms=None, vs=None, master=None, step=S, lr=1e-3, lr_dev=None,
          b1=0.9, b2=0.999, eps=1e-8, scale=None):
    def arr(kind, values):
        return None if values is None else (kind * len(values))(*values)

    return optim._lib.dlrm_adamw_step(
        n, arr(ctypes.c_void_p, params), arr(ctypes.c_void_p, grads),
        arr(ctypes.c_int64, counts), arr(ctypes.c_int32, pd), arr(ctypes.c_int32, gd),
        arr(ctypes.c_float, decays), bits, m, v, ms, vs, master, step, lr, lr_dev, b1, b2, eps,
        scale, 0, None)


def test_step_refusals(optim):
    for kw in (dict(params=None), dict(grads=None), dict(counts=None), dict(pd=None),
               dict(gd=None), dict(params=(A, None)), dict(grads=(None, S)), dict(m=None),
               dict(v=None), dict(step=None), dict(bits=8, ms=None, vs=S),
               dict(bits=8, ms=S, vs=None)):
        assert _step(optim, **kw) == NULL, kw
    for kw in (dict(n=-1), dict(n=BIG), dict(counts=(-1, 7)), dict(counts=(1 << 40, 7)),
               dict(counts=((1 << 40) - 1, 1)), dict(counts=(1 << 39, 1 << 39))):
        assert _step(optim, **kw) == SHAPE, kw
    for kw in (dict(pd=(2, 0)), dict(gd=(0, -1)), dict(bits=16), dict(bits=0), dict(lr=NAN),
               dict(lr=INF), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=NAN),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-60), dict(eps=INF), dict(eps=NAN),
               dict(decays=(0.0, NAN)), dict(decays=(INF, 0.0))):
        assert _step(optim, **kw) == ARG, kw
    for kw in (dict(params=(A + 2, W)), dict(params=(A, W + 1)), dict(grads=(Y, S + 2)),
               dict(m=A + 8), dict(v=W + 4), dict(master=A + 4), dict(step=S + 2),
               dict(lr_dev=S + 1), dict(scale=S + 2), dict(bits=8, ms=S + 4, vs=S),
               dict(bits=8, ms=S, vs=S + 8)):
        assert _step(optim, **kw) == ALIGN, kw
    assert optim.launch_count() == 0


def test_moments_refusals(optim):
    def call(n=512, m=A, v=W, ms=S, vs=S, mo=Y, vo=Y, dtype=0):
        return optim._lib.dlrm_adamw_moments(n, m, v, ms, vs, mo, vo, dtype, None)

    for name in ("m", "v", "ms", "vs", "mo", "vo"):
        assert call(**{name: None}) == NULL, name
    for kw in (dict(n=-256), dict(n=100), dict(n=1 << 40)):
        assert call(**kw) == SHAPE, kw
    assert call(dtype=2) == ARG
    for kw in (dict(m=A + 8), dict(v=A + 4), dict(ms=S + 2), dict(vs=S + 1), dict(mo=Y + 8),
               dict(vo=Y + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(n=0) == OK
    assert optim.launch_count() == 0


def test_scale_sizes(optim):
    size = optim._lib.dlrm_fp4_scale_bytes
    assert size(1, 1) == 512 and size(128, 128) == 512 and size(129, 129) == 4 * 512
    assert size(0, 5) == 0
    for bad in ((-1, 5), (5, 0), (BIG, 5), (5, BIG), (1 << 30, 1 << 30)):
        assert size(*bad) == SHAPE, bad


def test_quantize_refusals(optim):
    def q(x=A, ldx=64, dtype=0, M=3, K=64, q=W, ldq=32, scale=S):
        return optim._lib.dlrm_quantize_fp4(x, ldx, dtype, M, K, q, ldq, scale, None)

    def d(q=A, ldq=32, scale=S, M=3, K=64, y=Y, dtype=0, ldy=64):
        return optim._lib.dlrm_dequantize_fp4(q, ldq, scale, M, K, y, dtype, ldy, None)

    for call, pointers in ((q, ("x", "q", "scale")), (d, ("q", "scale", "y"))):
        for name in pointers:
            assert call(**{name: None}) == NULL, name
        for kw in (dict(M=-1), dict(M=BIG), dict(K=0), dict(K=BIG), dict(ldq=31)):
            assert call(**kw) == SHAPE, kw
        assert call(dtype=2) == ARG and call(scale=S + 2) == ALIGN
        assert call(M=0) == OK
    assert q(ldx=63) == SHAPE and d(ldy=63) == SHAPE
    assert q(M=1 << 30, K=1 << 30, ldx=1 << 30, ldq=1 << 29) == SHAPE
    assert q(x=A + 2) == ALIGN and d(y=Y + 2) == ALIGN and d(y=Y + 1, dtype=1) == ALIGN
    assert optim.launch_count() == 0


def test_linear_refusals(optim):
    def call(x=A, ldx=32, xs=S, w=W, ldw=32, ws=S, b=None, M=4, N=8, K=64, act=0, y=Y, yd=0,
             ldy=8, st=None):
        return optim._lib.dlrm_linear_fp4(x, ldx, xs, w, ldw, ws, b, M, N, K, act, y, yd, ldy, st,
                                          None)

    for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(M=-1), dict(M=BIG), dict(N=0), dict(N=BIG), dict(K=0), dict(K=BIG),
               dict(ldx=16), dict(ldw=16), dict(ldy=7)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(act=3), dict(act=-1), dict(yd=2)):
        assert call(**kw) == ARG, kw
    for kw in (dict(ldx=40), dict(ldw=40), dict(x=A + 8), dict(w=W + 8), dict(xs=S + 4),
               dict(ws=S + 8), dict(b=S + 2), dict(y=Y + 2), dict(y=Y + 1, yd=1),
               dict(st=S + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(M=0) == OK
    assert optim.launch_count() == 0


def test_python_checks(optim):
    """Wrong placements, types and networks are refused in the binding."""
    from dlrm_embedding_bag_b200 import fp4, mlp

    cpu, u8 = torch.zeros((4, 8)), torch.zeros((4, 8), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA device"):
        fp4.quantize_rows(cpu)
    with pytest.raises(ValueError, match="CUDA device"):
        fp4.dequantize_rows(u8, u8)
    with pytest.raises(ValueError, match="CUDA device"):
        fp4.linear_fp4(u8, u8, u8, u8)
    with pytest.raises(ValueError, match="act must be"):
        fp4.linear_fp4(u8, u8, u8, u8, act="gelu")
    with pytest.raises(ValueError, match="CUDA device"):
        optim.adamw_state([cpu])
    with pytest.raises(ValueError, match="at least one"):
        optim.adamw_state([])
    with pytest.raises(ValueError, match="bits must be"):
        optim.adamw_state([cpu], bits=4)
    with pytest.raises(TypeError, match="torch.Tensor"):
        optim.adamw_state([1.0])
    q = fp4.fp4_empty(3, 17, "cpu")
    assert q.shape == (3, 9) and q.stride() == (16, 1)
    assert fp4.fp4_empty(3, 64, "cpu").stride() == (32, 1)
    assert fp4.scale_shape(129, 5) == (2, 1, 512)
    assert optim.arena_offsets([torch.zeros(1), torch.zeros(256), torch.zeros(0), torch.zeros(3, 100)]) == \
        ((0, 256, 512, 512), 1024)
    with pytest.raises(ValueError, match="fp4_layers"):
        mlp.MLP([(cpu, None, "none")], mode="fp4")
    net = mlp.MLP([((u8, u8), None, "none")], mode="fp4")
    assert net.out_features == 4
    with pytest.raises(ValueError, match="one input"):
        net.forward(cpu, a_hi=cpu)
    with pytest.raises(ValueError, match="norms need"):
        mlp.MLP([((u8, u8), None, "none")], mode="fp4", norms=[cpu])


def _pretend(optim, monkeypatch):
    """CPU tensors stand in for the device's; what reaches the entry point is kept."""
    seen = []


    # a stub of a checked function sees CPU tensors as on device 0
    monkeypatch.setattr(optim, "_on", lambda t, name, index: None)
    monkeypatch.setattr(optim, "_flat", lambda t, name, dtype, index: (
        t.data_ptr() if t.dtype == dtype and t.is_contiguous()
        else (_ for _ in ()).throw(TypeError(f"{name} must be {dtype}"))))
    monkeypatch.setattr(optim, "_arena", lambda t, name, dtype, n, index: (
        optim._flat(t, name, dtype, index) if t is not None and t.numel() == n
        else (_ for _ in ()).throw(ValueError(f"{name} must have {n}"))))
    monkeypatch.setattr(optim, "_call", lambda fn, name, index, args: seen.append((name, args)))
    return seen


def test_step_lists_are_checked(optim, monkeypatch):
    """What the step's lists have to be, with CPU tensors in place of the device's."""
    seen = _pretend(optim, monkeypatch)
    params = [torch.zeros((3, 5)), torch.zeros(7, dtype=torch.bfloat16)]
    grads = [torch.zeros((3, 5)), torch.zeros(7)]
    zeros = lambda n: torch.zeros(n)  # noqa: E731
    st = optim.AdamWState(zeros(512), zeros(512), torch.zeros(2, dtype=torch.int32))
    optim.adamw_step(params, grads, st, lr=0.1, weight_decay=(0.5, 0.25))
    name, args = seen.pop()
    assert name == "dlrm_adamw_step" and args[0] == 2 and args[7] == 32
    for bad, match in (
            (dict(grads=grads[:1]), "grads must have 2"),
            (dict(grads=[grads[0], zeros(8)]), r"grads\[1\] must be \(7,\)"),
            (dict(grads=[torch.zeros((5, 3)), grads[1]]), r"grads\[0\] must be \(3, 5\)"),
            (dict(grads=[torch.zeros((5, 3)).T, grads[1]]), r"grads\[0\] must be contiguous"),
            (dict(params=[params[0], torch.zeros(7, dtype=torch.float16)]), r"params\[1\] must be float32"),
            (dict(st=st._replace(m=zeros(256))), "state.m must have 512"),
            (dict(st=st._replace(v=zeros(768))), "state.v must have 512"),
            (dict(st=st._replace(step=torch.zeros(1, dtype=torch.int32))), "state.step must have 2"),
            (dict(st=st._replace(master=zeros(22))), "state.master must have 512"),
            (dict(weight_decay=(0.1,)), "weight_decay must have 2"),
            (dict(lr=zeros(2)), "lr must have 1"),
            (dict(grad_scale=zeros(0)), "grad_scale must have 1"),
            (dict(st=st._replace(m=torch.zeros(512).to(torch.float8_e4m3fn))), "state.v must be"),
    ):
        kw = dict(params=params, grads=grads, st=st, lr=0.1)
        kw.update(bad)
        p, g, s = kw.pop("params"), kw.pop("grads"), kw.pop("st")
        with pytest.raises((ValueError, TypeError), match=match):
            optim.adamw_step(p, g, s, **kw)
        assert not seen
