"""Python binding of ``libdlrm_tokens.so``: embedding rows by token id, and the
table's gradient (the C ABI in ``include/dlrm_tokens.h``; the 8-bit layers of
``include/dlrm_int8.h`` are bound in :mod:`.int8`).

Argument marshalling only, as in :mod:`.ops`: every function checks tensor
placement, dtype and shape, passes raw pointers and the stream to the C entry
point, and raises :class:`~.ops.DlrmError` on a non-zero status. All tensors of
a call are on one device; the call runs there, on that device's current
stream, whichever device is current. If the library is missing, importing this
module raises: there is no fallback.

A table is a ``(rows, D)`` float32 or bfloat16 tensor with unit column stride;
its rows may be further apart (a column slice of a wider buffer).
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

from . import ops

LIBRARY = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdlrm_tokens.so")

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
# Every symbol that dlrm_tokens.h and dlrm_int8.h declare, with its ctypes signature.
SIGNATURES = {
    "dlrm_embedding_lookup": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _F, _I64, _P, _I, _I64, _P,
                                   _P]),
    "dlrm_embedding_grad_scratch_bytes": (_I64, [_I64, _I64, _I64]),
    "dlrm_embedding_grad": (_I, [_P, _I, _I64, _P, _I64, _I64, _I64, _I64, _F, _I64, _P, _I, _I64,
                                 _I, _P, _I64, _P, _P]),
    "dlrm_tokens_last_cuda_error": (_I, []),
    "dlrm_tokens_launch_count": (_I64, []),
    # include/dlrm_int8.h
    "dlrm_rms_norm_int8": (_I, [_P, _I64, _P, _I64, _I, _P, _I64, _I64, _F, _P, _I64, _P, _I64,
                                _P, _P]),
    "dlrm_quantize_int8": (_I, [_P, _I64, _I, _I64, _I64, _P, _I64, _P, _P]),
    "dlrm_dequantize_int8": (_I, [_P, _I64, _P, _I64, _I64, _P, _I, _I64, _P]),
    "dlrm_linear_int8": (_I, [_P, _I64, _P, _P, _I64, _P, _P, _I64, _I64, _I64, _I, _P, _I, _I64,
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
_lookup = _lib.dlrm_embedding_lookup
_grad = _lib.dlrm_embedding_grad
_scratch_bytes = _lib.dlrm_embedding_grad_scratch_bytes


class TokensError(ops.DlrmError):
    """A call into ``libdlrm_tokens.so`` returned a non-zero ``dlrm_status_t``."""

    def __init__(self, status: int, what: str):
        name = ops.STATUS.get(status, str(status))
        msg = f"{what}: {name} ({ops._lib.dlrm_status_string(status).decode()})"
        if status == -7:
            msg += f", cudaError {_lib.dlrm_tokens_last_cuda_error()}"
        RuntimeError.__init__(self, msg)
        self.status = status


# The raw handle of a device's current stream, without a Stream object around it
# (which alone costs 3 us a call).
_raw_stream = torch._C._cuda_getCurrentRawStream
_get_device = torch._C._cuda_getDevice
try:  # the allocator without an argument parser in front of it: 0.8 instead of 2.0 us
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    _empty_strided_cuda = None


def _empty(rows: int, cols: int, dtype: torch.dtype, index: int) -> torch.Tensor:
    """A new contiguous ``(rows, cols)`` tensor on device ``index``."""
    if _empty_strided_cuda is not None and index == _get_device():
        return _empty_strided_cuda((rows, cols), (cols, 1), dtype)
    return torch.empty((rows, cols), dtype=dtype, device=torch.device("cuda", index))


def _empty_vector(n: int, dtype: torch.dtype, index: int) -> torch.Tensor:
    """A new ``(n,)`` tensor on device ``index``."""
    if _empty_strided_cuda is not None and index == _get_device():
        return _empty_strided_cuda((n,), (1,), dtype)
    return torch.empty(n, dtype=dtype, device=torch.device("cuda", index))


def _call(fn, name: str, index: int, args: tuple) -> None:
    """Call the C entry point ``fn`` on device ``index`` and its current stream."""
    if index == _get_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != 0:
        raise TokensError(rc, name)


# The checks below run in front of every call: each first asks whether all is well
# and looks for what is not only then.

def _on(t: torch.Tensor, name: str, index: Optional[int]) -> None:
    """Raises unless ``t`` is a CUDA tensor (on device ``index`` if that is given)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (got {t.device})")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index} (got {t.device})")


def _pitch(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """(rows, columns, row pitch) of a 2-D tensor with unit column stride."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    rows, cols = shape
    if t.is_contiguous():
        return rows, cols, cols
    pitch, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    if rows <= 1:
        # the pitch of a single row says nothing (and may be smaller than the row)
        pitch = max(pitch, cols)
    elif pitch < cols:
        raise ValueError(f"{name}'s rows must not overlap")
    return rows, cols, pitch


def _matrix(t: torch.Tensor, name: str, index: Optional[int] = None):
    """(device index, dtype code, rows, columns, row pitch) of an f32 or bf16 matrix."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda) or \
            (index is not None and t.get_device() != index):
        _on(t, name, index)
    code = ops.TABLE_DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16 (got {t.dtype})")
    return (t.get_device(), code, *_pitch(t, name))


def _flat(t: torch.Tensor, name: str, dtype: torch.dtype, index: int) -> int:
    """Pointer of a contiguous tensor of ``dtype`` on device ``index``."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == index \
            and t.dtype is dtype and t.is_contiguous():
        return t.data_ptr()
    _on(t, name, index)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    raise ValueError(f"{name} must be contiguous")


def _status(status: Optional[torch.Tensor], index: int) -> Optional[int]:
    if status is None:
        return None
    if status.numel() != 1:
        raise ValueError("status must have one element")
    return _flat(status, "status", torch.int32, index)


def _padding(padding_idx: Optional[int], rows: int) -> int:
    if padding_idx is None:
        return -1
    if not 0 <= padding_idx < rows:
        raise ValueError(f"padding_idx must be in [0, {rows}) (got {padding_idx})")
    return padding_idx


def embedding_lookup(table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
                     padding_idx: Optional[int] = None, out_dtype: Optional[torch.dtype] = None,
                     out: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows of ``table`` by token id: ``scale * table[ids]``, ``(*ids.shape, D)``.

    ``table`` is ``(rows, D)``, ``ids`` int32 of any shape. The product is taken
    in f32 and rounded once to ``out_dtype`` (default: the table's). Rows of
    ``padding_idx`` are zero; an id outside ``[0, rows)`` reads nothing, its row
    is zero and ``FLAG_INDEX_OOB`` is set in ``status`` (one int32) if given.
    ``out`` may be given as ``(ids.numel(), D)`` rows with a pitch, or as a
    contiguous tensor of the result's shape.
    """
    index, wd, rows, D, ldw = _matrix(table, "table")
    pi = _flat(ids, "ids", torch.int32, index)
    T = ids.numel()
    if out is None:
        out_dtype = out_dtype or table.dtype
        od = ops.TABLE_DTYPES.get(out_dtype)
        if od is None:
            raise TypeError(f"out_dtype must be float32 or bfloat16 (got {out_dtype})")
        out = _empty(T, D, out_dtype, index)
        po, ldo = out.data_ptr(), D
        if ids.dim() != 1:
            out = out.view(*ids.shape, D)
    else:
        _on(out, "out", index)
        od = ops.TABLE_DTYPES.get(out.dtype)
        if od is None or (out_dtype is not None and out.dtype != out_dtype):
            raise TypeError(f"out must be {out_dtype or 'float32 or bfloat16'} (got {out.dtype})")
        if out.shape == (*ids.shape, D) and out.is_contiguous():
            ldo = D
        elif out.shape == (T, D):
            ldo = _pitch(out, "out")[2]
        else:
            raise ValueError(f"out must be {(*ids.shape, D)} (contiguous) or {(T, D)} "
                             f"(got {tuple(out.shape)})")
        po = out.data_ptr()
    _call(_lookup, "dlrm_embedding_lookup", index,
          (table.data_ptr(), wd, ldw, rows, D, pi, T, scale, _padding(padding_idx, rows), po, od,
           ldo, _status(status, index)))
    return out


@functools.lru_cache(maxsize=256)
def embedding_grad_scratch_bytes(T: int, rows: int, D: int) -> int:
    """Bytes of scratch that :func:`embedding_grad` needs for ``T`` ids (may be 0)."""
    n = _scratch_bytes(T, rows, D)
    if n < 0:
        raise TokensError(n, "dlrm_embedding_grad_scratch_bytes")
    return n


def embedding_grad(grad: torch.Tensor, ids: torch.Tensor, num_rows: int, *, L: int = 1,
                   scale: float = 1.0, padding_idx: Optional[int] = None,
                   dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                   accumulate: bool = False, scratch: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of a table from the gradients of its rows' uses:
    ``out[r] = scale * sum over t with ids[t] == r of grad[t // L]``.

    ``grad`` is ``(T // L, D)`` rows (any pitch) for ``T = ids.numel()`` int32
    ids. ``L = 1`` is the gradient of :func:`embedding_lookup`; with bags of
    ``L`` ids it is the gradient of :func:`.ops.embbag_sum_multi` with respect
    to table ``k``, from ``grad = dpooled[:, k]`` and ``ids = indices[k]``.

    The tokens are sorted by id and summed in f32 in a fixed order: equal
    inputs give equal bits. The result is a new ``(num_rows, D)`` tensor of
    ``dtype`` (default: grad's), or ``out``; rows that no token names are zero.
    With ``accumulate`` the sums are added to ``out`` instead and other rows
    are not touched, so ``out=table, scale=-lr`` is a sparse SGD step. Tokens of
    ``padding_idx`` and ids outside ``[0, num_rows)`` add nothing (the latter
    set ``FLAG_INDEX_OOB`` in ``status`` if given). ``scratch``: a uint8 tensor
    of at least :func:`embedding_grad_scratch_bytes` bytes; by default one is
    taken from torch's allocator for the call.
    """
    index, gd, n, D, ldg = _matrix(grad, "grad")
    pi = _flat(ids, "ids", torch.int32, index)
    T = ids.numel()
    if L < 1 or T % L != 0 or n != T // L:
        raise ValueError(f"grad must have ids.numel() / L = {T} / {L} rows (got {n})")
    room = embedding_grad_scratch_bytes(T, num_rows, D)  # refuses what the sizes rule out
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        dtype = dtype or grad.dtype
        od, ldo = ops.TABLE_DTYPES.get(dtype), D
        if od is None:
            raise TypeError(f"dtype must be float32 or bfloat16 (got {dtype})")
        out = _empty(num_rows, D, dtype, index)
    else:
        _, od, out_rows, out_cols, ldo = _matrix(out, "out", index)
        if dtype is not None and out.dtype != dtype:
            raise TypeError(f"out must be {dtype} (got {out.dtype})")
        if out_rows != num_rows or out_cols != D:
            raise ValueError(f"out must be ({num_rows}, {D}) (got {tuple(out.shape)})")
    ps = None
    if scratch is None:
        if room:
            scratch = _empty_vector(room, torch.uint8, index)
            ps = scratch.data_ptr()
    else:
        ps, room = _flat(scratch, "scratch", torch.uint8, index), scratch.numel()
    _call(_grad, "dlrm_embedding_grad", index,
          (grad.data_ptr(), gd, ldg, pi, T, L, num_rows, D, scale,
           _padding(padding_idx, num_rows), out.data_ptr(), od, ldo, 1 if accumulate else 0, ps,
           room, _status(status, index)))
    return out


def launch_count() -> int:
    """Kernels that ``libdlrm_tokens.so`` has launched in this process."""
    return int(_lib.dlrm_tokens_launch_count())
