"""The norms around a block with its gate and residual: the binding of ``w8a8_block_norm``."""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from .binding import _P, _SZ, _check, _need_cuda, lib
from .mx4 import MX4Tensor, _call, _device, _rows_of, mx4_bytes

_KINDS = {"rms": 1, "layer": 2}
_RESIDUAL = {torch.bfloat16: 0, torch.float32: 1}
_I64 = ctypes.c_int64


class Norm(NamedTuple):
    """A norm: ``kind`` "rms" or "layer", bf16 weight and bias [K] (None: 1 and 0)."""
    kind: str
    weight: Optional[torch.Tensor] = None
    bias: Optional[torch.Tensor] = None
    eps: float = 1e-6


class BlockNormOutput(NamedTuple):
    """What was asked for; the rest is None."""
    residual: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    a_scale: Optional[torch.Tensor]
    mx4: Optional[MX4Tensor]


class _NormStruct(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("eps", ctypes.c_float), ("weight", _P), ("bias", _P)]


class _Args(ctypes.Structure):
    _fields_ = [("M", _I64), ("K", _I64), ("x", _P), ("ldx", _I64), ("residual", _P),
                ("residual_out", _P), ("ldr", _I64), ("ldro", _I64), ("residual_dtype", ctypes.c_int),
                ("residual_scale", ctypes.c_float), ("post", _NormStruct), ("pre", _NormStruct),
                ("gate", _P), ("scale", _P), ("shift", _P), ("ld_gate", _I64), ("ld_scale", _I64),
                ("ld_shift", _I64), ("groups", _I64), ("rows_per_group", _I64), ("group_index", _P),
                ("y", _P), ("ldy", _I64), ("q", _P), ("a_scale", _P), ("image", _P),
                ("image_bytes", _SZ)]


def _set_norm(to: _NormStruct, norm: Norm, K: int):
    kind = _KINDS.get(norm.kind)
    if kind is None:
        raise ValueError(f"norm kind must be one of {sorted(_KINDS)}, got {norm.kind!r}")
    to.kind, to.eps = kind, norm.eps
    for name, t in (("weight", norm.weight), ("bias", norm.bias)):
        if t is not None:
            _need_cuda(t, f"norm {name}", torch.bfloat16)
            if t.numel() != K or not t.is_contiguous():
                raise ValueError(f"norm {name} must be contiguous and hold {K} values")
            setattr(to, name, t.data_ptr())


def block_norm(x: torch.Tensor, residual: Optional[torch.Tensor] = None, *, post: Optional[Norm] = None,
               gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
               pre: Optional[Norm] = None, scale: Optional[torch.Tensor] = None,
               shift: Optional[torch.Tensor] = None, rows_per_group: Optional[int] = None,
               group_index: Optional[torch.Tensor] = None, codes: Optional[str] = None,
               y: Optional[bool] = None, residual_out: Optional[torch.Tensor] = None,
               stream=None) -> BlockNormOutput:
    """The step between two blocks, in one kernel:

        u = post(x);  r = residual_scale * residual + gate[g] * u;  y = pre(r) * (1 + scale[g]) + shift[g]

    x: bf16 [..., K], the block's output (without ``residual``: what ``pre`` norms).
    residual: bf16 or fp32 [..., K]; the new stream goes to ``residual_out`` (``residual`` itself
    for an update in place) or to a new tensor.
    gate, scale, shift: bf16 [groups, K] (slices of a wider tensor may be given as they are; [K]
    for one group).  The group of row m is ``group_index[m]`` (int32; a row whose index is
    outside the groups is padding and is left alone), else m // ``rows_per_group`` (default: all
    rows in one group).
    codes: "int8" (``q`` and ``a_scale``, for ``W8A8Linear.apply_codes``) or "mx4" (an ``MX4Tensor``, for
    ``MX4Linear``), equal to the codes of the bf16 output; None: y itself.  ``y=True`` gives y beside codes.
    """
    _need_cuda(x, "x", torch.bfloat16)
    K = x.shape[-1]
    if codes not in (None, "int8", "mx4"):
        raise ValueError(f'codes must be None, "int8" or "mx4", got {codes!r}')
    if pre is None and (codes or y or scale is not None or shift is not None):
        raise ValueError("codes, y, scale and shift need the norm before the next block (pre)")
    if residual is None and (post is not None or gate is not None or residual_out is not None):
        raise ValueError("post, gate and residual_out need a residual")
    if residual is None and pre is None:
        raise ValueError("nothing to compute: give residual, pre or both")
    index = _device(x, residual, gate, scale, shift, group_index, residual_out,
                    *(t for n in (post, pre) if n is not None for t in (n.weight, n.bias)))
    if residual is not None:
        _need_cuda(residual, "residual")
        if residual.dtype not in _RESIDUAL:
            raise ValueError(f"residual must be bf16 or fp32, got {residual.dtype}")
        if residual.shape != x.shape:
            raise ValueError(f"residual must have x's shape {list(x.shape)}, got {list(residual.shape)}")
        if residual_out is not None and (residual_out.dtype != residual.dtype or residual_out.shape != x.shape):
            raise ValueError("residual_out must have the residual's type and shape")
    want_y = pre is not None and (codes is None if y is None else y)
    if pre is not None and codes is None and not want_y:
        raise ValueError("y=False leaves no output for the norm: ask for codes")

    def f(s):
        x2, M, ldx = _rows_of(x)
        a = _Args(M=M, K=K, x=x2.data_ptr(), ldx=ldx, residual_scale=residual_scale)
        if post is not None:
            _set_norm(a.post, post, K)
        if pre is not None:
            _set_norm(a.pre, pre, K)
        new = None
        held = [x2]  # what a copy was made of, until the launch
        if residual is not None:
            r2, _, a.ldr = _rows_of(residual)
            held.append(r2)
            if residual_out is None:
                new, a.ldro = torch.empty(x.shape, dtype=residual.dtype, device=index), K
            else:  # written in place: a view, never a copy
                new = residual_out
                n2 = new.view(-1, K) if new.is_contiguous() else new
                if n2.dim() != 2 or (M and n2.stride(1) != 1):
                    raise ValueError("residual_out must be contiguous, or [rows, K] with unit stride along K")
                a.ldro = n2.stride(0) if M > 1 else K
            a.residual, a.residual_out = r2.data_ptr(), new.data_ptr()
            a.residual_dtype = _RESIDUAL[residual.dtype]

        groups = 0
        for name, t in (("gate", gate), ("scale", scale), ("shift", shift)):
            if t is None:
                continue
            _need_cuda(t, name, torch.bfloat16)
            if t.dim() == 1:
                t = t.view(1, -1)
            if t.dim() != 2 or t.shape[1] != K or (groups and t.shape[0] != groups):
                raise ValueError(f"{name} must be [groups, {K}], with as many groups as the others, "
                                 f"got {list(t.shape)}")
            t, groups, ld = _rows_of(t)
            held.append(t)
            setattr(a, name, t.data_ptr())
            setattr(a, "ld_" + name, ld)
        if group_index is not None:
            _need_cuda(group_index, "group_index", torch.int32)
            if group_index.numel() != M or not group_index.is_contiguous():
                raise ValueError(f"group_index must be contiguous and hold {M} values")
            a.group_index = group_index.data_ptr()
            groups = groups or 1
        if groups:
            a.groups = groups
            a.rows_per_group = (M or 1) if rows_per_group is None else rows_per_group

        out = q = a_scale = image = None
        if want_y:
            out = torch.empty(x.shape, dtype=torch.bfloat16, device=index)
            a.y, a.ldy = out.data_ptr(), K
        if codes == "int8":
            q = torch.empty(x.shape, dtype=torch.int8, device=index)
            a_scale = torch.empty((M,), dtype=torch.float32, device=index)
            a.q, a.a_scale = q.data_ptr(), a_scale.data_ptr()
        elif codes == "mx4":
            a.image_bytes = mx4_bytes(M, K) if M else 0
            image = torch.empty((a.image_bytes,), dtype=torch.uint8, device=index)
            a.image = image.data_ptr()
        if M:
            _check(lib().w8a8_block_norm(ctypes.byref(a), s), "w8a8_block_norm")
        return BlockNormOutput(new, out, q, a_scale,
                               None if image is None else MX4Tensor(image, x.shape[:-1], K))
    return _call(index, stream, f)
