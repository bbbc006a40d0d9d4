"""The token-level library on the CPU: it loads, exports exactly what its headers
declare, and refuses bad arguments before any CUDA call (no call here reaches
a kernel launch)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = [os.path.join(ROOT, "include", h) for h in ("dlrm_tokens.h", "dlrm_int8.h")]
OK, NULL, SHAPE, ALIGN, ARG, SCRATCH = 0, -1, -2, -3, -9, -10
A, W, Y, S = 0x10000, 0x20000, 0x30000, 0x40000  # aligned, never dereferenced
BIG = 1 << 31


@pytest.fixture(scope="module")
def tokens():
    from dlrm_embedding_bag_b200 import build

    build.build()
    from dlrm_embedding_bag_b200 import tokens as _tokens

    return _tokens


def _declarations():
    out = {}
    for h in HEADERS:
        src = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        for ret, name, params in re.findall(r"DLRM_API\s+([\w\s\*]+?)\b(\w+)\s*\(([^)]*)\)\s*;",
                                            src):
            plist = [] if params.strip() in ("", "void") else [p.strip() for p in params.split(",")]
            out[name] = (ret.strip(), [re.sub(r"\s*\b\w+$", "", p) for p in plist])
    return out


def test_exports_are_what_the_headers_declare(tokens):
    out = subprocess.run(["nm", "-D", "--defined-only", tokens.LIBRARY], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert exported == set(_declarations()) == set(tokens.SIGNATURES)


def test_signatures_match_the_headers(tokens):
    kinds = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "float": ctypes.c_float}
    for name, (ret, params) in _declarations().items():
        res, args = tokens.SIGNATURES[name]
        want = [ctypes.c_void_p if "*" in p or p == "dlrm_stream_t" else kinds[p] for p in params]
        assert args == want, name
        assert res is kinds[ret], name


def test_headers_compile_as_c(tmp_path):
    probe = tmp_path / "probe.c"
    probe.write_text('#include <stdio.h>\n#include "dlrm_tokens.h"\n#include "dlrm_int8.h"\n'
                     'int main(void) { printf("%d\\n", DLRM_INT8_MAX_K); return 0; }\n')
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(probe), "-o", str(exe)], check=True)
    from dlrm_embedding_bag_b200 import int8

    assert int(subprocess.run([str(exe)], capture_output=True, text=True).stdout) == int8.MAX_K


def test_missing_library_fails_loudly(tokens, tmp_path):
    with pytest.raises(ImportError, match="no CPU fallback"):
        tokens.load_library(str(tmp_path / "libdlrm_tokens.so"))


def test_lookup_refusals(tokens):
    def call(table=A, wd=0, ldw=8, rows=10, D=8, ids=W, T=4, pad=-1, out=Y, od=0, ldo=8, st=None):
        return tokens._lib.dlrm_embedding_lookup(table, wd, ldw, rows, D, ids, T, 1.0, pad, out,
                                                 od, ldo, st, None)

    for kw in (dict(table=None), dict(ids=None), dict(out=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(rows=0), dict(rows=BIG - 1), dict(D=0), dict(T=-1), dict(T=BIG), dict(ldw=7),
               dict(ldo=7)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(wd=2), dict(od=-1), dict(pad=-2), dict(pad=10)):
        assert call(**kw) == ARG, kw
    for kw in (dict(table=A + 2), dict(table=A + 1, wd=1), dict(out=Y + 2), dict(ids=W + 2),
               dict(st=S + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(T=0, ids=None, table=None, out=None) == OK  # nothing to do, nothing enqueued
    assert tokens.launch_count() == 0


def test_grad_refusals(tokens):
    def call(grad=A, gd=0, ldg=8, ids=W, T=602, L=1, rows=10, D=8, pad=-1, out=Y, od=0, ldo=8,
             scratch=S, room=1 << 30, st=None):
        return tokens._lib.dlrm_embedding_grad(grad, gd, ldg, ids, T, L, rows, D, 1.0, pad, out,
                                               od, ldo, 0, scratch, room, st, None)

    for kw in (dict(grad=None), dict(ids=None), dict(out=None), dict(scratch=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(rows=0), dict(rows=BIG - 1), dict(D=0), dict(T=-1), dict(T=BIG), dict(ldg=7),
               dict(ldo=7), dict(L=0), dict(L=3), dict(L=-1)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(gd=2), dict(od=-1), dict(pad=-2), dict(pad=10)):
        assert call(**kw) == ARG, kw
    for kw in (dict(grad=A + 2), dict(out=Y + 2), dict(ids=W + 2), dict(st=S + 2),
               dict(scratch=S + 8)):
        assert call(**kw) == ALIGN, kw
    need = tokens.embedding_grad_scratch_bytes(602, 10, 8)
    assert need > 0 and need % 16 == 0
    assert call(room=need - 1) == SCRATCH
    assert tokens.launch_count() == 0


def test_scratch_sizes(tokens):
    small = tokens.embedding_grad_scratch_bytes(1000, 5000, 64)
    assert small >= 1000 * 8
    assert tokens.embedding_grad_scratch_bytes(0, 1, 1) == 0
    assert tokens.embedding_grad_scratch_bytes(512, 1000, 64) == 0
    assert tokens.embedding_grad_scratch_bytes(512, 1 << 20, 64) > 512 * 8
    assert tokens.embedding_grad_scratch_bytes(513, 1000, 64) > 513 * 8
    # the largest token list: its size does not leave 64 bits
    assert tokens.embedding_grad_scratch_bytes(BIG - 1, BIG - 2, 4096) > (BIG - 1) * 8
    for bad in ((-1, 5, 5), (BIG, 5, 5), (5, 0, 5), (5, BIG - 1, 5), (5, 5, 0)):
        with pytest.raises(tokens.TokensError, match="DLRM_ERR_SHAPE"):
            tokens.embedding_grad_scratch_bytes(*bad)


def test_norm_refusals(tokens):
    def call(x=A, ldx=16, r=None, ldr=0, dt=0, w=None, M=3, K=16, eps=1e-6, h=None, ldh=0, q=Y,
             ldq=16, s=S):
        return tokens._lib.dlrm_rms_norm_int8(x, ldx, r, ldr, dt, w, M, K, eps, h, ldh, q, ldq, s,
                                              None)

    for kw in (dict(x=None), dict(q=None), dict(s=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(M=-1), dict(M=BIG), dict(K=0), dict(K=BIG), dict(ldx=15), dict(ldq=15),
               dict(r=W, ldr=15), dict(h=W, ldh=15)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(dt=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**kw) == ARG, kw
    for kw in (dict(x=A + 2), dict(r=W + 2, ldr=16), dict(h=W + 2, ldh=16), dict(w=W + 2),
               dict(s=S + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(M=0) == OK and call(M=0, x=None, q=None, s=None) == OK
    lib = tokens._lib
    assert lib.dlrm_quantize_int8(None, 16, 0, 3, 16, Y, 16, S, None) == NULL
    assert lib.dlrm_quantize_int8(A, 15, 0, 3, 16, Y, 16, S, None) == SHAPE
    assert lib.dlrm_quantize_int8(A, 16, 3, 3, 16, Y, 16, S, None) == ARG
    assert lib.dlrm_quantize_int8(A, 16, 0, 0, 16, Y, 16, S, None) == OK
    assert lib.dlrm_dequantize_int8(None, 16, S, 3, 16, Y, 0, 16, None) == NULL
    assert lib.dlrm_dequantize_int8(A, 16, S, 3, 16, Y, 0, 15, None) == SHAPE
    assert lib.dlrm_dequantize_int8(A, 16, S, 3, 16, Y + 1, 1, 16, None) == ALIGN
    assert lib.dlrm_dequantize_int8(A, 16, S, 0, 16, Y, 1, 16, None) == OK
    assert tokens.launch_count() == 0


def test_linear_refusals(tokens):
    def call(x=A, ldx=64, xs=S, w=W, ldw=64, ws=S, b=None, M=4, N=8, K=64, act=0, y=Y, yd=0,
             ldy=8, st=None):
        return tokens._lib.dlrm_linear_int8(x, ldx, xs, w, ldw, ws, b, M, N, K, act, y, yd, ldy,
                                            st, None)

    for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(M=-1), dict(M=BIG), dict(N=0), dict(N=BIG), dict(K=0), dict(ldx=48),
               dict(ldw=48), dict(ldy=7), dict(K=131072, ldx=131072, ldw=131072)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(act=3), dict(act=-1), dict(yd=2)):
        assert call(**kw) == ARG, kw
    for kw in (dict(ldx=72), dict(ldw=72), dict(x=A + 8), dict(w=W + 8), dict(xs=S + 2),
               dict(ws=S + 2), dict(b=S + 2), dict(y=Y + 2), dict(y=Y + 1, yd=1),
               dict(st=S + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(M=0) == OK
    assert tokens.launch_count() == 0


def test_python_checks(tokens):
    """Wrong placements and types are refused in the binding."""
    from dlrm_embedding_bag_b200 import int8

    cpu = torch.zeros((4, 8))
    ids = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        tokens.embedding_lookup(cpu, ids)
    with pytest.raises(TypeError, match="torch.Tensor"):
        tokens.embedding_lookup([1.0], ids)
    with pytest.raises(ValueError, match="CUDA device"):
        tokens.embedding_grad(cpu, ids, 4)
    with pytest.raises(ValueError, match="CUDA device"):
        int8.quantize_rows(cpu)
    with pytest.raises(ValueError, match="CUDA device"):
        int8.rms_norm_int8(cpu)
    with pytest.raises(ValueError, match="CUDA device"):
        int8.linear_int8(cpu.to(torch.int8), cpu[0], cpu.to(torch.int8), cpu[0])
    with pytest.raises(ValueError, match="act must be"):
        int8.linear_int8(cpu.to(torch.int8), cpu[0], cpu.to(torch.int8), cpu[0], act="gelu")
    q = int8.int8_empty(3, 17, "cpu")
    assert q.shape == (3, 17) and q.stride() == (32, 1)


def test_calls_run_on_their_tensors_device(tokens, monkeypatch):
    """A call on a device that is not current is made with that device current, on
    its stream; a failed one raises with the library's status."""
    seen, current = [], [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.old, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.old

    monkeypatch.setattr(tokens, "_get_device", lambda: current[0])
    monkeypatch.setattr(tokens, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(tokens.torch.cuda, "device", Device)

    def entry(a, stream):
        seen.append((a, stream, current[0]))
        return -2 if a == 7 else 0

    tokens._call(entry, "entry", 0, (5,))
    tokens._call(entry, "entry", 1, (6,))
    assert seen == [(5, 1000, 0), (6, 1001, 1)] and current == [0]
    with pytest.raises(tokens.TokensError, match="entry: DLRM_ERR_SHAPE") as e:
        tokens._call(entry, "entry", 1, (7,))
    assert e.value.status == -2 and current == [0]
    assert isinstance(e.value, tokens.ops.DlrmError)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("last_f32", [True, False])
def test_residual_stack_does_not_depend_on_the_inputs_type(tokens, monkeypatch, dtype, last_f32):
    """Which norms of an 8-bit network read a residual, and which: by widths alone."""
    from dlrm_embedding_bag_b200 import int8, mlp

    calls = []

    def norm(x, weight=None, *, residual=None, eps=1e-6):
        assert residual is None or residual.dtype == x.dtype
        calls.append(None if residual is None else residual.float().sum().item())
        total = None if residual is None else x + residual
        return x, torch.ones(x.shape[0]), total

    def linear(q, s, w_q, w_scale, bias, act, *, out_dtype):
        # every layer doubles its input's first columns
        return (2 * q.float()[:, :1]).expand(-1, w_q.shape[0]).to(out_dtype)

    monkeypatch.setattr(int8, "rms_norm_int8", norm)
    monkeypatch.setattr(int8, "linear_int8", linear)
    monkeypatch.setattr(mlp, "to_bf16", lambda t: t.to(torch.bfloat16))
    layers = [((torch.zeros((n, k), dtype=torch.int8), torch.ones(n)), None, "none")
              for k, n in ((8, 8), (8, 8), (8, 8), (8, 4), (4, 4), (4, 2))]
    net = mlp.MLP(layers, mode="int8", norms=[torch.ones(k) for k in (8, 8, 8, 8, 4, 4)])
    y32, y16 = net.forward(torch.ones((1, 8), dtype=dtype), last_f32=last_f32,
                           last_bf16=not last_f32)
    # sums before it: 1; 1 + 2; 3 + 4; then four columns wide, from 16 on
    assert calls == [None, 8 * 1.0, 8 * 3.0, 8 * 7.0, None, 4 * 16.0]
    y = y32 if last_f32 else y16
    assert y.dtype == (torch.float32 if last_f32 else torch.bfloat16) and (y == 64).all()


def test_a_networks_rounding_runs_where_its_layers_do(tokens, monkeypatch):
    """to_bf16 takes the current device's stream: MLP(mode="int8"), whose other calls run on
    their tensors' device, makes that one current around it."""
    from dlrm_embedding_bag_b200 import int8, mlp

    inside, seen = [], []

    class DeviceOf:
        def __init__(self, t):
            self.t = t

        def __enter__(self):
            inside.append(self.t)

        def __exit__(self, *exc):
            inside.pop()

    def to_bf16(t):
        seen.append(len(inside) == 1 and inside[0] is t)
        return t.to(torch.bfloat16)

    def norm(x, weight=None, *, residual=None, eps=1e-6):
        return x, torch.ones(x.shape[0]), residual

    monkeypatch.setattr(mlp.torch.cuda, "device_of", DeviceOf)
    monkeypatch.setattr(mlp, "to_bf16", to_bf16)
    monkeypatch.setattr(int8, "rms_norm_int8", norm)
    monkeypatch.setattr(int8, "linear_int8",
                        lambda q, s, w, ws, b, act, *, out_dtype: q.to(out_dtype))
    layers = [((torch.zeros((8, 8), dtype=torch.int8), torch.ones(8)), None, "none")] * 2
    net = mlp.MLP(layers, mode="int8", norms=[torch.ones(8)] * 2)
    _, y16 = net.forward(torch.ones((2, 8)), last_bf16=True)
    # the stack's first sum, and the last output's rounding
    assert y16.dtype == torch.bfloat16 and seen == [True, True]
