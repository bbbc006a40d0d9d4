"""Python binding of ``libdlrm_narrow.so``: the AdamW step over many tensors at once
(the C ABI in ``include/dlrm_optim.h``; the 4-bit layers of ``include/dlrm_fp4.h``
are bound in :mod:`.fp4`).

Argument marshalling only, as in :mod:`.tokens`: every function checks tensor
placement, dtype and shape, passes raw pointers and the stream to the C entry point,
and raises :class:`NarrowError` on a non-zero status. All tensors of a call are
on one device; the call runs there, on that device's current stream, whichever
device is current. If the library is missing, importing this module raises: there
is no fallback.

:func:`adamw_state` makes the buffers of a list of parameters, :func:`adamw_step`
takes one step in place, :func:`adamw_moments` reads 8-bit moments. The step stands
beside :func:`.tokens.embedding_grad` with ``accumulate`` (sparse SGD). It takes
contiguous tensors, bf16 and f32 in one list: a table, an :class:`.mlp.MLP`'s biases and those
of its weights whose columns are a multiple of 8. Weights of other widths have padded rows
(:func:`.mlp.bf16_empty`) and are refused: a contiguous copy is stepped and copied back.
"""
from __future__ import annotations

import ctypes
import os
from array import array
from operator import attrgetter
from typing import NamedTuple, Optional, Sequence, Tuple, Union

import torch

from . import ops
from .tokens import _empty_vector, _flat, _get_device, _on, _raw_stream

LIBRARY = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdlrm_narrow.so")
BLOCK = 256  # elements of the moments that share a scale; where tensors start

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_D = ctypes.c_double
# Every symbol that dlrm_optim.h and dlrm_fp4.h declare, with its ctypes signature.
SIGNATURES = {
    "dlrm_adamw_step": (_I, [_I64, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _D, _P, _D,
                             _D, _D, _P, ctypes.c_uint32, _P]),
    "dlrm_adamw_moments": (_I, [_I64, _P, _P, _P, _P, _P, _P, _I, _P]),
    "dlrm_narrow_last_cuda_error": (_I, []),
    "dlrm_narrow_launch_count": (_I64, []),
    # include/dlrm_fp4.h
    "dlrm_fp4_scale_bytes": (_I64, [_I64, _I64]),
    "dlrm_quantize_fp4": (_I, [_P, _I64, _I, _I64, _I64, _P, _I64, _P, _P]),
    "dlrm_dequantize_fp4": (_I, [_P, _I64, _P, _I64, _I64, _P, _I, _I64, _P]),
    "dlrm_linear_fp4": (_I, [_P, _I64, _P, _P, _I64, _P, _P, _I64, _I64, _I64, _I, _P, _I, _I64,
                             _P, _P]),
}


def load_library(path: str = LIBRARY) -> ctypes.CDLL:
    """Load the CUDA library and bind every declared symbol; raise if absent."""
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -m dlrm_embedding_bag_b200.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = load_library()
_step = _lib.dlrm_adamw_step
_moments = _lib.dlrm_adamw_moments


class NarrowError(ops.DlrmError):
    """A call into ``libdlrm_narrow.so`` returned a non-zero ``dlrm_status_t``."""

    def __init__(self, status: int, what: str):
        name = ops.STATUS.get(status, str(status))
        msg = f"{what}: {name} ({ops._lib.dlrm_status_string(status).decode()})"
        if status == -7:
            msg += f", cudaError {_lib.dlrm_narrow_last_cuda_error()}"
        RuntimeError.__init__(self, msg)
        self.status = status


def _call(fn, name: str, index: int, args: tuple) -> None:
    """Call the C entry point ``fn`` on device ``index`` and its current stream."""
    if index == _get_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != 0:
        raise NarrowError(rc, name)


class AdamWState(NamedTuple):
    """The buffers of an AdamW step; all of them are updated in place.

    ``m`` and ``v`` are flat: parameter i's elements start where those before it end,
    rounded up to a multiple of :data:`BLOCK`. In 32 bits they are f32; in 8 bits ``m`` is
    ``torch.float8_e4m3fn`` and ``v`` uint8 codes of the second moment's root (the
    format is in ``dlrm_optim.h``), with f32 ``m_scale`` and ``v_scale`` for each
    block. ``master`` (f32, flat, or None) holds the weights of bf16 parameters.
    ``step`` is int32 ``(2,)``: steps taken, and a word of the call's own, which a step leaves at
    zero and finds at any number above -2^30 (``state.step.fill_(t)`` goes on from step t, and
    ``state.step.sub_(1)`` from the one before).
    """

    m: torch.Tensor
    v: torch.Tensor
    step: torch.Tensor
    m_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None
    master: Optional[torch.Tensor] = None


def arena_offsets(params: Sequence[torch.Tensor]) -> Tuple[Tuple[int, ...], int]:
    """Where each parameter's elements start in the flat buffers, and the buffers' length."""
    at, total = [], 0
    for p in params:
        at.append(total)
        total += (p.numel() + BLOCK - 1) // BLOCK * BLOCK
    return tuple(at), total


def adamw_state(params: Sequence[torch.Tensor], *, bits: int = 32,
                master: bool = False) -> AdamWState:
    """The state of ``params`` before the first step: moments of zero in 32 or 8 bits, and with
    ``master`` f32 copies of the bf16 parameters (f32 ones need none)."""
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32 (got {bits})")
    params = list(params)
    if not params:
        raise ValueError("a state needs at least one parameter")
    index = None  # the first one's
    for i, p in enumerate(params):
        _on(p, f"params[{i}]", index)
        index = p.get_device()
        if p.dtype not in ops.TABLE_DTYPES:
            raise TypeError(f"params[{i}] must be float32 or bfloat16 (got {p.dtype})")
    dev = params[0].device
    at, total = arena_offsets(params)
    step = torch.zeros(2, dtype=torch.int32, device=dev)
    copies = None
    if master and any(p.dtype == torch.bfloat16 for p in params):
        copies = torch.zeros(total, dtype=torch.float32, device=dev)
        for o, p in zip(at, params):
            if p.dtype == torch.bfloat16:
                copies[o:o + p.numel()].view(p.shape).copy_(p.detach())
    kind = torch.float32  # whatever torch's default is
    if bits == 32:
        return AdamWState(torch.zeros(total, dtype=kind, device=dev),
                          torch.zeros(total, dtype=kind, device=dev), step, master=copies)
    return AdamWState(torch.zeros(total, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn),
                      torch.zeros(total, dtype=torch.uint8, device=dev), step,
                      torch.zeros(total // BLOCK, dtype=kind, device=dev),
                      torch.zeros(total // BLOCK, dtype=kind, device=dev), copies)


_CODES = ops.TABLE_DTYPES


_dtype_of, _shape_of = attrgetter("dtype"), attrgetter("shape")
# methods of the class, which map() calls without a lookup for each tensor
_device_of, _dense, _pointer, _length = (
    torch.Tensor.get_device, torch.Tensor.is_contiguous, torch.Tensor.data_ptr, torch.Tensor.numel)


def _refuse(tensors, name: str, index: int) -> None:
    """Raises for the first of ``tensors`` that is not a contiguous f32 or bf16 one there."""
    for i, t in enumerate(tensors):
        _on(t, f"{name}[{i}]", index)
        if t.dtype not in _CODES:
            raise TypeError(f"{name}[{i}] must be float32 or bfloat16 (got {t.dtype})")
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous")


def _list(tensors: Sequence[torch.Tensor], name: str, index: int):
    """(pointers, dtype codes) of contiguous f32 or bf16 tensors on device ``index``.

    Whole lists are asked at once, a third of the time of a loop over the tensors; which
    one is not right is looked for only then."""
    try:
        fine = all(map(_dense, tensors)) and set(map(_device_of, tensors)) <= {index}
        types = list(map(_dtype_of, tensors))
        codes = array("i", map(_CODES.__getitem__, types)) if len(set(types)) != 1 else \
            array("i", (_CODES[types[0]],)) * len(types)
    except (AttributeError, KeyError, TypeError):
        fine = False
    if not fine:
        _refuse(tensors, name, index)
        raise ValueError(f"{name} must be contiguous tensors on cuda:{index}")
    return array("q", map(_pointer, tensors)), codes


def _arena(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, n: int, index: int) -> int:
    """Pointer of a contiguous tensor of ``n`` elements of ``dtype`` on device ``index``."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == n \
            and t.get_device() == index and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if t is None:
        raise ValueError(f"{name} is missing")
    _flat(t, name, dtype, index)
    raise ValueError(f"{name} must have {n} elements (got {t.numel()})")


def _eight_bit(state: AdamWState) -> bool:
    if not isinstance(state.m, torch.Tensor):
        raise TypeError("state.m must be a torch.Tensor")
    return state.m.dtype == torch.float8_e4m3fn


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], state: AdamWState, *,
               lr: Union[float, torch.Tensor], betas: Tuple[float, float] = (0.9, 0.999),
               eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.0,
               grad_scale: Optional[torch.Tensor] = None, seed: int = 0) -> None:
    """One AdamW step on every parameter, in place: with ``g = grad_scale * grad`` and the
    step's number ``t`` (counted in ``state.step``, on the device)

    ``m = b1 m + (1 - b1) g``, ``v = b2 v + (1 - b2) g^2``,
    ``p = p (1 - lr weight_decay) - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps)``.

    ``params`` and ``grads`` are contiguous f32 or bf16 tensors in the order that the state
    was made for, each gradient of its parameter's shape and of either type. Up to 96 of
    them that are not empty are one launch. Arithmetic is f32. A bf16 parameter is
    rounded from its master, or without masters up or down at random (in proportion, so that
    steps below half a bf16 step are kept on average), as 8-bit moments are; the random bits are
    a function of ``seed``, the step and the element's place, so equal calls give equal bits.

    ``lr`` is a number or one f32 on the device (read when the step runs, so that a
    captured step follows a schedule), ``weight_decay`` a number or one for each
    parameter, ``grad_scale`` one f32 on the device (a clipping coefficient) or None.
    No parameter may overlap another, or a gradient.
    """
    index = state.step.get_device()
    n = len(params)
    if len(grads) != n:
        raise ValueError(f"grads must have {n} entries (got {len(grads)})")
    pp, pc = _list(params, "params", index)
    pg, gc = _list(grads, "grads", index)
    if len(set(pp)) != n:
        known = set()
        for i, p in enumerate(pp):
            if p in known:
                raise ValueError(f"params[{i}] is there twice")
            if p:  # (empty ones have no address)
                known.add(p)
    if list(map(_shape_of, params)) != list(map(_shape_of, grads)):
        i = next(i for i in range(n) if params[i].shape != grads[i].shape)
        raise ValueError(f"grads[{i}] must be {tuple(params[i].shape)} (got {tuple(grads[i].shape)})")
    counts = array("q", map(_length, params))
    total = sum([(c + BLOCK - 1) // BLOCK for c in counts]) * BLOCK
    ps = _arena(state.step, "state.step", torch.int32, 2, index)
    if _eight_bit(state):
        bits = 8
        pm = _arena(state.m, "state.m", torch.float8_e4m3fn, total, index)
        pv = _arena(state.v, "state.v", torch.uint8, total, index)
        pms = _arena(state.m_scale, "state.m_scale", torch.float32, total // BLOCK, index)
        pvs = _arena(state.v_scale, "state.v_scale", torch.float32, total // BLOCK, index)
    else:
        bits, pms, pvs = 32, None, None
        pm = _arena(state.m, "state.m", torch.float32, total, index)
        pv = _arena(state.v, "state.v", torch.float32, total, index)
    pw = _arena(state.master, "state.master", torch.float32, total, index) \
        if state.master is not None else None
    rate, pl = 0.0, None
    if isinstance(lr, torch.Tensor):
        pl = _arena(lr, "lr", torch.float32, 1, index)
    else:
        rate = lr
    pd, decays = None, None
    if not isinstance(weight_decay, (int, float)):
        decays = array("f", weight_decay)
        if len(decays) != n:
            raise ValueError(f"weight_decay must have {n} entries (got {len(decays)})")
    elif weight_decay != 0.0:
        decays = array("f", [weight_decay]) * n
    if decays is not None:
        pd = decays.buffer_info()[0]
    pgs = _arena(grad_scale, "grad_scale", torch.float32, 1, index) \
        if grad_scale is not None else None
    _call(_step, "dlrm_adamw_step", index,
          (n, pp.buffer_info()[0], pg.buffer_info()[0], counts.buffer_info()[0],
           pc.buffer_info()[0], gc.buffer_info()[0], pd, bits, pm, pv, pms, pvs, pw, ps, rate, pl,
           betas[0], betas[1], eps, pgs, seed & 0xffffffff))


def adamw_moments(state: AdamWState, *, dtype: torch.dtype = torch.float32):
    """``(m, v)`` of a state in 8 bits as flat f32 or bf16 values (those in 32 bits are
    ``state.m`` and ``state.v`` themselves)."""
    if not _eight_bit(state):
        raise ValueError("state holds moments in 32 bits: read state.m and state.v")
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be float32 or bfloat16 (got {dtype})")
    _on(state.m, "state.m", None)
    index, total = state.m.get_device(), state.m.numel()
    pm = _arena(state.m, "state.m", torch.float8_e4m3fn, total, index)
    pv = _arena(state.v, "state.v", torch.uint8, total, index)
    if total % BLOCK:
        raise ValueError(f"state.m must have a multiple of {BLOCK} elements (got {total})")
    pms = _arena(state.m_scale, "state.m_scale", torch.float32, total // BLOCK, index)
    pvs = _arena(state.v_scale, "state.v_scale", torch.float32, total // BLOCK, index)
    m, v = _empty_vector(total, dtype, index), _empty_vector(total, dtype, index)
    _call(_moments, "dlrm_adamw_moments", index,
          (total, pm, pv, pms, pvs, m.data_ptr(), v.data_ptr(), code))
    return m, v


def launch_count() -> int:
    """Kernels that ``libdlrm_narrow.so`` has launched in this process."""
    return int(_lib.dlrm_narrow_launch_count())
