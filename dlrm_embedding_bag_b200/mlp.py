"""Python binding of the DLRMv1 MLP layers (the C ABI in ``include/dlrm_mlp.h``).

Argument marshalling only, as in :mod:`.ops`: pointers, row pitches and the
current stream go to ``dlrm_linear_f32a`` / ``dlrm_linear_bf16`` /
``dlrm_split_f32_bf16x3`` / ``dlrm_f32_to_bf16``; every layer runs in the
library's tcgen05 kernel. bf16 tensors are ``torch.bfloat16``
views whose row pitch is a multiple of 8 elements (16 bytes), as the layer's
TMA loads require; :func:`bf16_empty` makes such buffers.

Three arithmetics are offered (``mode``). ``"f32"`` (the default) is the pages' own: f32
activations times bf16 (or f32) weights with f32 results, through
``dlrm_linear_f32a``; each f32 activation travels between layers as three
bf16 planes that sum to it exactly (:func:`planes_empty`,
:func:`split_bf16x3`). ``"bf16"`` rounds activations to bf16 (one plane,
``dlrm_linear_bf16``), a third of the tensor work. ``"int8"`` rounds the rows of
activations to 8-bit integers in front of every layer, with one scale for each
row and for each output channel of the weights (:mod:`.int8`), half of the
bytes of ``"bf16"`` at twice its tensor rate.

A DLRMv1 forward (:func:`dlrm_forward`) is: bottom MLP on the dense features
-> ``dense`` (B, D); the sparse stage (pooled embeddings and the interaction
z, :func:`.ops.sparse_interact`); the top MLP whose first layer reads
``[dense | z]`` through the split-A form, ending in a sigmoid CTR head.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import torch

from . import ops

ACTS = {"none": 0, "relu": 1, "sigmoid": 2}


def _round8(n: int) -> int:
    return (n + 7) // 8 * 8


def bf16_empty(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """A ``(rows, cols)`` bf16 view whose row pitch is ``cols`` rounded up to 8."""
    return torch.empty((rows, _round8(cols)), dtype=torch.bfloat16, device=device)[:, :cols]


def _pitched(t: torch.Tensor, name: str, dtype: torch.dtype) -> Tuple[int, int]:
    """(pointer, row pitch in elements) of a 2-D CUDA tensor with unit column stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1]))


def _room(t: Optional[torch.Tensor], name: str, rows: int, cols: int) -> None:
    """Raises if an output's last two dimensions have no room for ``(rows, cols)``."""
    if t is not None and (t.dim() < 2 or t.shape[-2] < rows or t.shape[-1] < cols):
        raise ValueError(f"{name} must have room for ({rows}, {cols}) (got {tuple(t.shape)})")


def to_bf16(x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Round an f32 ``(rows, cols)`` tensor to bf16 (nearest even) into a pitched buffer."""
    px, ldx = _pitched(x, "x", torch.float32)
    rows, cols = x.shape
    if out is None:
        out = bf16_empty(rows, cols, x.device)
    py, ldy = _pitched(out, "out", torch.bfloat16)
    _room(out, "out", rows, cols)
    if rows == 0:  # nothing to round, and no pointers for the entry point
        return out
    ops._check(ops._lib.dlrm_f32_to_bf16(px, ldx, rows, cols, py, ldy, ops._stream()),
               "dlrm_f32_to_bf16")
    return out


def _to_bf16_there(x: torch.Tensor) -> torch.Tensor:
    """:func:`to_bf16` on x's device, where the 8-bit layers around it run, current or not."""
    with torch.cuda.device_of(x):
        return to_bf16(x)


def linear_bf16(a_lo: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                act: str = "none", *, a_hi: Optional[torch.Tensor] = None, f32: bool = True,
                bf16: bool = False, out_f32: Optional[torch.Tensor] = None,
                out_bf16: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None):
    """One layer ``act([a_lo | a_hi] w^T + bias)``; returns ``(y_f32, y_bf16)``.

    ``a_lo`` ``(M, K_lo)``, ``a_hi`` ``(M, K_hi)`` (optional) and ``w``
    ``(N, K_lo + K_hi)`` are bf16; ``bias`` is ``(N,)`` f32 or None. The f32
    and/or bf16 result is written to ``out_*`` or to new buffers (``f32`` /
    ``bf16`` select which are made); the one not requested is None.
    """
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    pa, lda = _pitched(a_lo, "a_lo", torch.bfloat16)
    M, k_lo = a_lo.shape
    if a_hi is not None:
        ph, ldh = _pitched(a_hi, "a_hi", torch.bfloat16)
        if a_hi.shape[0] != M:
            raise ValueError("a_hi must have as many rows as a_lo")
        k_hi = a_hi.shape[1]
    else:
        ph, ldh, k_hi = None, 0, 0
    pw, ldw = _pitched(w, "w", torch.bfloat16)
    N = w.shape[0]
    if w.shape[1] != k_lo + k_hi:
        raise ValueError(f"w must be (N, {k_lo + k_hi})")
    pb = None
    if bias is not None:
        pb = ops._dev(bias, "bias", torch.float32)
        if bias.numel() != N:
            raise ValueError(f"bias must have {N} elements")
    if out_f32 is None and f32:
        out_f32 = torch.empty((M, N), dtype=torch.float32, device=a_lo.device)
    if out_bf16 is None and bf16:
        out_bf16 = bf16_empty(M, N, a_lo.device)
    pf, ldf = _pitched(out_f32, "out_f32", torch.float32) if out_f32 is not None else (None, 0)
    pbf, ldbf = (_pitched(out_bf16, "out_bf16", torch.bfloat16) if out_bf16 is not None
                 else (None, 0))
    _room(out_f32, "out_f32", M, N)
    _room(out_bf16, "out_bf16", M, N)
    ps = ops._dev(status, "status", torch.int32) if status is not None else None
    ops._check(ops._lib.dlrm_linear_bf16(pa, lda, k_lo, ph, ldh, k_hi, pw, ldw, pb, M, N,
                                         ACTS[act], pf, ldf, pbf, ldbf, ps, ops._stream()),
               "dlrm_linear_bf16")
    return out_f32, out_bf16


def planes_empty(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """A ``(3, rows, cols)`` bf16 view: three planes whose row pitch is ``cols``
    rounded up to 8 (16-byte rows, as the layers' TMA loads require)."""
    return torch.empty((3, rows, _round8(cols)), dtype=torch.bfloat16,
                       device=device)[:, :, :cols]


def _planes(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """(pointer, row pitch, plane stride) in elements of a ``(3, rows, cols)`` bf16 tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda" or t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    if t.dim() != 3 or t.shape[0] != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be (3, rows, cols) with unit column stride")
    ld = t.stride(1) if t.shape[1] > 1 else max(t.stride(1), t.shape[2])
    return t.data_ptr(), ld, t.stride(0)


def split_bf16x3(x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The exact three-plane split of an f32 ``(rows, cols)`` tensor:
    ``x == p[0] + p[1] + p[2]`` with every plane a bf16 value."""
    px, ldx = _pitched(x, "x", torch.float32)
    rows, cols = x.shape
    if out is None:
        out = planes_empty(rows, cols, x.device)
    py, ldy, sp = _planes(out, "out")
    _room(out, "out", rows, cols)
    ops._check(ops._lib.dlrm_split_f32_bf16x3(px, ldx, rows, cols, py, ldy, sp, ops._stream()),
               "dlrm_split_f32_bf16x3")
    return out


def linear_f32a(a_lo: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                act: str = "none", *, a_hi: Optional[torch.Tensor] = None, f32: bool = True,
                planes: bool = False, out_f32: Optional[torch.Tensor] = None,
                out_planes: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None):
    """One layer ``act([a_lo | a_hi] w^T + bias)`` on f32 activations; returns
    ``(y_f32, y_planes)``.

    ``a_lo`` ``(3, M, K_lo)`` and ``a_hi`` ``(3, M, K_hi)`` (optional) are the
    activations' bf16 planes (:func:`split_bf16x3`); ``w`` is bf16 ``(N, K)``
    weights or the ``(3, N, K)`` planes of f32 weights; ``bias`` ``(N,)`` f32 or
    None. The f32 result and/or its planes (the next layer's input) are
    written to ``out_*`` or to new buffers (``f32`` / ``planes`` select which).
    """
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    pa, lda, spa = _planes(a_lo, "a_lo")
    M, k_lo = a_lo.shape[1], a_lo.shape[2]
    if a_hi is not None:
        ph, ldh, sph = _planes(a_hi, "a_hi")
        if a_hi.shape[1] != M:
            raise ValueError("a_hi must have as many rows as a_lo")
        k_hi = a_hi.shape[2]
    else:
        ph, ldh, sph, k_hi = None, 0, 0, 0
    if w.dim() == 3:
        pw, ldw, spw = _planes(w, "w")
        w_planes, N, kw = 3, w.shape[1], w.shape[2]
    else:
        pw, ldw = _pitched(w, "w", torch.bfloat16)
        spw, w_planes, N, kw = 0, 1, w.shape[0], w.shape[1]
    if kw != k_lo + k_hi:
        raise ValueError(f"w must have {k_lo + k_hi} columns")
    pb = None
    if bias is not None:
        pb = ops._dev(bias, "bias", torch.float32)
        if bias.numel() != N:
            raise ValueError(f"bias must have {N} elements")
    if out_f32 is None and f32:
        out_f32 = torch.empty((M, N), dtype=torch.float32, device=a_lo.device)
    if out_planes is None and planes:
        out_planes = planes_empty(M, N, a_lo.device)
    pf, ldf = _pitched(out_f32, "out_f32", torch.float32) if out_f32 is not None else (None, 0)
    pp, ldp, spp = _planes(out_planes, "out_planes") if out_planes is not None else (None, 0, 0)
    _room(out_f32, "out_f32", M, N)
    _room(out_planes, "out_planes", M, N)
    ps = ops._dev(status, "status", torch.int32) if status is not None else None
    ops._check(ops._lib.dlrm_linear_f32a(pa, lda, spa, k_lo, ph, ldh, sph, k_hi, pw, ldw, spw,
                                         w_planes, pb, M, N, ACTS[act], pf, ldf, pp, ldp, spp,
                                         ps, ops._stream()),
               "dlrm_linear_f32a")
    return out_f32, out_planes


class MLP:
    """A stack of layers ``(w, bias, act)``.

    ``w`` is a bf16 ``(N, K)`` tensor (pitched, see :func:`bf16_empty`), or in
    ``"f32"`` mode also the ``(3, N, K)`` planes of f32 weights; ``bias``
    ``(N,)`` f32, ``act`` one of ``"none" | "relu" | "sigmoid"``. In ``"bf16"``
    mode activations between layers are bf16; in ``"f32"`` mode they are f32,
    carried as three exact bf16 planes, and the input is given as planes.

    In ``"int8"`` mode ``w`` is a pair ``(w_q, w_scale)`` (:func:`int8_layers` makes
    them from weights) and the input an f32 or bf16 matrix. The rows in front of
    each layer are rounded to 8 bits (:func:`.int8.quantize_rows`) or, where
    ``norms[i]`` is given (f32 ``(K,)``), normed and rounded
    (:func:`.int8.rms_norm_int8`). Layers with a norm that follow each other at
    one width form a residual stack: the norm in front of layer i reads the sum
    of the sum before it and layer i-1's output. The first sum is the first of
    these layers' input. A stack's last output does not have the sum added.
    Activations between layers, and the sums, are bf16 (an f32 input of a stack is
    rounded as its first sum): what an 8-bit level (2^-8 of its row's maximum) is
    rounded from need not be finer.
    """

    def __init__(self, layers: Sequence[Tuple[torch.Tensor, torch.Tensor, str]],
                 mode: str = "f32", *,
                 norms: Optional[Sequence[Optional[torch.Tensor]]] = None, eps: float = 1e-6):
        if not layers:
            raise ValueError("an MLP needs at least one layer")
        if mode not in ("bf16", "f32", "int8"):
            raise ValueError("mode must be 'bf16', 'f32' or 'int8'")
        if norms is not None and mode != "int8":
            raise ValueError("norms need mode 'int8'")
        if norms is not None and len(norms) != len(layers):
            raise ValueError(f"norms must have {len(layers)} entries")
        if mode == "int8" and any(isinstance(w, torch.Tensor) for w, _, _ in layers):
            raise ValueError("an int8 layer's weights are (w_q, w_scale): see int8_layers")
        self.layers: List[Tuple[torch.Tensor, torch.Tensor, str]] = list(layers)
        self.mode = mode
        self.norms = list(norms) if norms is not None else [None] * len(self.layers)
        self.eps = eps

    @property
    def out_features(self) -> int:
        w = self.layers[-1][0]
        return (w[0] if self.mode == "int8" else w).shape[0]

    def _forward_int8(self, x, last_f32: bool, last_bf16: bool, keep: bool):
        from . import int8

        inputs = []
        h, total = x, None  # total: the residual stack's running sum
        n = len(self.layers)
        for i, ((w_q, w_scale), b, act) in enumerate(self.layers):
            if self.norms[i] is None:
                q, s = int8.quantize_rows(h)
                total = None
            elif total is not None and total.shape == h.shape:
                q, s, total = int8.rms_norm_int8(h, self.norms[i], residual=total, eps=self.eps)
            else:
                q, s, _ = int8.rms_norm_int8(h, self.norms[i], eps=self.eps)
                total = None
                # a stack goes on by widths alone: its sum has the activations' type at once
                if i + 1 < n and self.norms[i + 1] is not None and w_q.shape[0] == h.shape[1]:
                    total = h if h.dtype == torch.bfloat16 else _to_bf16_there(h)
            inputs.append((q, s))
            dtype = torch.float32 if i == n - 1 and last_f32 else torch.bfloat16
            h = int8.linear_int8(q, s, w_q, w_scale, b, act, out_dtype=dtype)
        y32 = h if last_f32 else None
        y_n = None if not last_bf16 else _to_bf16_there(h) if last_f32 else h
        return ((y32, y_n), inputs) if keep else (y32, y_n)

    def forward(self, x: torch.Tensor, *, a_hi: Optional[torch.Tensor] = None,
                last_f32: bool = True, last_bf16: bool = False, keep: bool = False):
        """Run the layers on ``x`` (and ``a_hi`` for the first layer's split form):
        bf16 tensors in ``"bf16"`` mode, three-plane tensors in ``"f32"`` mode.

        Returns ``(y_f32, y_next)`` of the last layer -- ``y_next`` is its bf16
        output (``"bf16"``) or its planes (``"f32"``) when ``last_bf16`` is set
        -- plus the list of every layer's inputs when ``keep`` is set. In
        ``"int8"`` mode ``x`` is an f32 or bf16 matrix, ``a_hi`` is not taken,
        ``y_next`` is bf16 and a layer's input is its ``(q, scale)``.
        """
        if self.mode == "int8":
            if a_hi is not None:
                raise ValueError("int8 layers take one input: a row has one scale")
            return self._forward_int8(x, last_f32, last_bf16, keep)
        inputs = []
        h, hi = x, a_hi
        n = len(self.layers)
        layer = linear_bf16 if self.mode == "bf16" else linear_f32a
        for i, (w, b, act) in enumerate(self.layers):
            inputs.append((h, hi))
            last = i == n - 1
            nxt = (not last) or last_bf16
            if self.mode == "bf16":
                y32, y_n = layer(h, w, b, act, a_hi=hi, f32=last and last_f32, bf16=nxt)
            else:
                y32, y_n = layer(h, w, b, act, a_hi=hi, f32=last and last_f32, planes=nxt)
            h, hi = y_n, None
        return ((y32, y_n), inputs) if keep else (y32, y_n)


def int8_layers(layers: Sequence[Tuple[torch.Tensor, torch.Tensor, str]]):
    """Layers ``(w, bias, act)`` with f32 or bf16 weights ``(N, K)`` as ``"int8"`` layers:
    the weights rounded to 8 bits with one scale for each output channel."""
    from . import int8

    return [(int8.quantize_rows(w), b, act) for w, b, act in layers]


def dlrm_forward(bottom: MLP, top: MLP, dense_x: torch.Tensor, weights: Sequence[torch.Tensor],
                 indices: torch.Tensor, offsets: torch.Tensor, L: int, *, keep: bool = False):
    """DLRMv1 forward: CTR ``(B, 1)`` f32 from the dense features and the tables.

    ``"bf16"`` MLPs: ``dense_x`` is bf16; bottom MLP -> ``dense`` (f32 for the
    interaction, bf16 for the top MLP); sparse stage -> z ``(B, P)`` f32 ->
    bf16; top MLP with ``[dense | z]`` as its split first-layer input.
    ``"f32"`` MLPs: ``dense_x`` is f32 and every activation stays f32: the
    bottom MLP's output goes to the interaction as f32 and to the top MLP as
    its exact planes, and z is split into planes. ``"int8"`` MLPs: ``dense_x`` is
    f32 or bf16, and the sparse stage writes the rows ``[dense | z]`` that the top
    MLP rounds to 8 bits. With ``keep`` it also returns a dict of the
    intermediate tensors.
    """
    if bottom.mode != top.mode:
        raise ValueError("the bottom and top MLPs must use the same mode")
    if bottom.mode == "int8":
        dense32, _ = bottom.forward(dense_x)
        pooled, z = ops.sparse_interact(weights, indices, offsets, dense32, L, concat_dense=True)
        (ctr, _), top_inputs = top.forward(z, keep=True)
        if keep:
            return ctr, dict(dense32=dense32, pooled=pooled, z=z, top_inputs=top_inputs)
        return ctr
    if bottom.mode == "f32":
        x_in = split_bf16x3(dense_x)
        dense32, dense_next = bottom.forward(x_in, last_f32=True, last_bf16=True)
        pooled, z = ops.sparse_interact(weights, indices, offsets, dense32, L)
        z_next = split_bf16x3(z)
    else:
        dense32, dense_next = bottom.forward(dense_x, last_f32=True, last_bf16=True)
        pooled, z = ops.sparse_interact(weights, indices, offsets, dense32, L)
        z_next = to_bf16(z)
    (ctr, _), top_inputs = top.forward(dense_next, a_hi=z_next, keep=True)
    if keep:
        return ctr, dict(dense32=dense32, dense16=dense_next, pooled=pooled, z=z, z16=z_next,
                         top_inputs=top_inputs)
    return ctr
