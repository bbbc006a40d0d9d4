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


class TokensError(ops.DlrmError):
    """A call into ``libdlrm_tokens.so`` returned a non-zero ``dlrm_status_t``."""

    def __init__(self, status: int, what: str):
        name = ops.STATUS.get(status, str(status))
        msg = f"{what}: {name} ({ops._lib.dlrm_status_string(status).decode()})"
        if status == -7:
            msg += f", cudaError {_lib.dlrm_tokens_last_cuda_error()}"
        RuntimeError.__init__(self, msg)
        self.status = status


def _call(name: str, device: torch.device, *args) -> None:
    """Call the C entry point ``name`` on ``device`` and its current stream."""
    fn = getattr(_lib, name)
    index = device.index
    if index == torch.cuda.current_device():
        rc = fn(*args, torch.cuda.current_stream().cuda_stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, torch.cuda.current_stream().cuda_stream)
    if rc != 0:
        raise TokensError(rc, name)


def _tensor(t: torch.Tensor, name: str, device: Optional[torch.device]) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")


def _rows(t: torch.Tensor, name: str, device: Optional[torch.device] = None) -> Tuple[int, int, int]:
    """(pointer, dtype code, row pitch) of a 2-D f32 or bf16 tensor with unit column stride."""
    _tensor(t, name, device)
    code = ops.TABLE_DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16 (got {t.dtype})")
    return t.data_ptr(), code, _pitch(t, name)


def _pitch(t: torch.Tensor, name: str) -> int:
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    # the pitch of a single row says nothing (and may be smaller than the row)
    pitch = t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])
    if t.shape[0] > 1 and pitch < t.shape[1]:
        raise ValueError(f"{name}'s rows must not overlap")
    return pitch


def _flat(t: torch.Tensor, name: str, dtype: torch.dtype, device: torch.device) -> int:
    """Pointer of a contiguous tensor of ``dtype`` on ``device``."""
    _tensor(t, name, device)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _status(status: Optional[torch.Tensor], device: torch.device) -> Optional[int]:
    if status is None:
        return None
    if status.numel() != 1:
        raise ValueError("status must have one element")
    return _flat(status, "status", torch.int32, device)


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
    pw, wd, ldw = _rows(table, "table")
    rows, D = table.shape
    dev = table.device
    pi = _flat(ids, "ids", torch.int32, dev)
    T = ids.numel()
    if out is None:
        out = torch.empty((*ids.shape, D), dtype=out_dtype or table.dtype, device=dev)
        result = out
    else:
        result = out
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out must be {out_dtype} (got {out.dtype})")
    if out.shape == (*ids.shape, D) and out.is_contiguous():
        out = out.view(T, D) if T else out.reshape(0, D)
    if tuple(out.shape) != (T, D):
        raise ValueError(f"out must be {(*ids.shape, D)} or {(T, D)} (got {tuple(out.shape)})")
    po, od, ldo = _rows(out, "out", dev)
    _call("dlrm_embedding_lookup", dev, pw, wd, ldw, rows, D, pi, T, scale,
          _padding(padding_idx, rows), po, od, ldo, _status(status, dev))
    return result


def embedding_grad_scratch_bytes(T: int, rows: int, D: int) -> int:
    """Bytes of scratch that :func:`embedding_grad` needs for ``T`` ids."""
    n = _lib.dlrm_embedding_grad_scratch_bytes(T, rows, D)
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
    pg, gd, ldg = _rows(grad, "grad")
    dev = grad.device
    pi = _flat(ids, "ids", torch.int32, dev)
    T, D = ids.numel(), grad.shape[1]
    if L < 1 or T % L != 0 or grad.shape[0] != T // L:
        raise ValueError(f"grad must have ids.numel() / L = {T} / {L} rows (got {grad.shape[0]})")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((num_rows, D), dtype=dtype or grad.dtype, device=dev)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError(f"out must be {dtype} (got {out.dtype})")
    if tuple(out.shape) != (num_rows, D):
        raise ValueError(f"out must be ({num_rows}, {D}) (got {tuple(out.shape)})")
    po, od, ldo = _rows(out, "out", dev)
    need = embedding_grad_scratch_bytes(T, num_rows, D)
    if scratch is None:
        scratch = torch.empty(need, dtype=torch.uint8, device=dev)
    ps = _flat(scratch, "scratch", torch.uint8, dev)
    _call("dlrm_embedding_grad", dev, pg, gd, ldg, pi, T, L, num_rows, D, scale,
          _padding(padding_idx, num_rows), po, od, ldo, 1 if accumulate else 0, ps,
          scratch.numel(), _status(status, dev))
    return out


def launch_count() -> int:
    """Kernels that ``libdlrm_tokens.so`` has launched in this process."""
    return int(_lib.dlrm_tokens_launch_count())
