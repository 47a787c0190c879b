"""The norms around a block with its gate and residual: the binding of ``w8a8_block_norm``."""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from .binding import _P, _SZ, _check, _need_cuda, lib
from .mx4 import MX4Tensor, _device, _on, _rows_of, mx4_bytes

_KINDS = {"rms": 1, "layer": 2}
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


def _norm(norm: Optional[Norm], K: int) -> _NormStruct:
    if norm is None:
        return _NormStruct(0, 0.0, None, None)
    if norm.kind not in _KINDS:
        raise ValueError(f"norm kind must be one of {sorted(_KINDS)}, got {norm.kind!r}")
    for name, t in (("weight", norm.weight), ("bias", norm.bias)):
        if t is not None:
            _need_cuda(t, f"norm {name}", torch.bfloat16)
            if t.numel() != K or not t.is_contiguous():
                raise ValueError(f"norm {name} must be contiguous and hold {K} values")
    return _NormStruct(_KINDS[norm.kind], norm.eps, None if norm.weight is None else norm.weight.data_ptr(),
                       None if norm.bias is None else norm.bias.data_ptr())


def _address(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


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
    dev = _device(x, residual, gate, scale, shift, group_index, residual_out,
                  *(t for n in (post, pre) if n is not None for t in (n.weight, n.bias)))
    a = _Args(K=K, post=_norm(post, K), pre=_norm(pre, K), residual_scale=residual_scale)
    with _on(dev, stream) as s:
        x2, a.ldx = _rows_of(x)
        M = a.M = x2.shape[0]
        a.x = x2.data_ptr()

        new = None
        if residual is not None:
            _need_cuda(residual, "residual")
            if residual.dtype not in (torch.bfloat16, torch.float32):
                raise ValueError(f"residual must be bf16 or fp32, got {residual.dtype}")
            if residual.shape != x.shape:
                raise ValueError(f"residual must have x's shape {list(x.shape)}, got {list(residual.shape)}")
            new = torch.empty(x.shape, dtype=residual.dtype, device=dev) if residual_out is None else residual_out
            if new.dtype != residual.dtype or new.shape != x.shape:
                raise ValueError("residual_out must have the residual's type and shape")
            r2, a.ldr = _rows_of(residual)
            # written in place: a view, never a copy
            n2 = new.view(-1, K) if new.is_contiguous() else new
            if n2.dim() != 2 or (M and n2.stride(1) != 1):
                raise ValueError("residual_out must be contiguous, or [rows, K] with unit stride along K")
            a.ldro = n2.stride(0) if M > 1 else K
            a.residual, a.residual_out = r2.data_ptr(), n2.data_ptr()
            a.residual_dtype = 1 if residual.dtype == torch.float32 else 0

        held, groups = [], None
        for name, t in (("gate", gate), ("scale", scale), ("shift", shift)):
            if t is None:
                continue
            _need_cuda(t, name, torch.bfloat16)
            t = t.view(1, -1) if t.dim() == 1 else t
            if t.dim() != 2 or t.shape[1] != K or (groups is not None and t.shape[0] != groups):
                raise ValueError(f"{name} must be [groups, {K}], with as many groups as the others, "
                                 f"got {list(t.shape)}")
            groups = t.shape[0]
            t, ld = _rows_of(t)
            held.append(t)
            setattr(a, name, t.data_ptr())
            setattr(a, "ld_" + name, ld)
        if group_index is not None:
            _need_cuda(group_index, "group_index", torch.int32)
            if group_index.numel() != M or not group_index.is_contiguous():
                raise ValueError(f"group_index must be contiguous and hold {M} values")
            a.group_index = group_index.data_ptr()
            groups = 1 if groups is None else groups
        a.groups = groups or 0
        a.rows_per_group = max(M, 1) if rows_per_group is None else rows_per_group

        want_y = pre is not None and (codes is None if y is None else y)
        if pre is not None and codes is None and not want_y:
            raise ValueError("y=False leaves no output for the norm: ask for codes")
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=dev) if want_y else None
        a.y, a.ldy = _address(out), K
        q = a_scale = image = None
        if codes == "int8":
            q = torch.empty(x.shape, dtype=torch.int8, device=dev)
            a_scale = torch.empty((M,), dtype=torch.float32, device=dev)
            a.q, a.a_scale = _address(q), _address(a_scale)
        elif codes == "mx4":
            a.image_bytes = mx4_bytes(M, K) if M else 0
            image = torch.empty((a.image_bytes,), dtype=torch.uint8, device=dev)
            a.image = image.data_ptr()
        if M:
            _check(lib().w8a8_block_norm(ctypes.byref(a), ctypes.c_void_p(s.cuda_stream)), "w8a8_block_norm")
    return BlockNormOutput(new, out, q, a_scale, None if image is None else MX4Tensor(image, x.shape[:-1], K))
