"""The norms around a block with its gate and residual: the binding of ``w8a8_block_norm``."""
from __future__ import annotations

import struct
from typing import NamedTuple, Optional

import torch

from .binding import _bytes, _check, _device, _elsewhere, _need_cuda, _raw_stream, _rows_of, _there, lib
from .mx4 import MX4Tensor, mx4_bytes

_KINDS = {"rms": 1, "layer": 2}
_RESIDUAL = {torch.bfloat16: 0, torch.float32: 1}


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


#: w8a8_block_norm_args, field by field (native alignment).
_ARGS = struct.Struct("@qq Pq PPqq if ifPP ifPP PPP qqq qq P Pq PP PN".replace(" ", ""))


def _vectors(norm: Optional[Norm], K: int):
    """(kind, eps, weight, bias) of a w8a8_norm."""
    if norm is None:
        return 0, 0.0, 0, 0
    kind, weight, bias, eps = norm
    if kind not in _KINDS:
        raise ValueError(f"norm kind must be one of {sorted(_KINDS)}, got {kind!r}")
    return _KINDS[kind], eps, _vector(weight, "norm weight", K), _vector(bias, "norm bias", K)


def _vector(t: Optional[torch.Tensor], name: str, K: int) -> int:
    if t is None:
        return 0
    _need_cuda(t, name, torch.bfloat16)
    if t.numel() != K or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and hold {K} values")
    return t.data_ptr()


def _per_group(t: torch.Tensor, name: str, K: int, groups: int):
    """(t, or a copy of it, as [groups, K] with rows on 16-byte boundaries, its address, groups, row stride)."""
    _need_cuda(t, name, torch.bfloat16)
    if t.dim() == 1:
        t = t.view(1, -1)
    shape = t.shape
    if len(shape) != 2 or shape[1] != K or not shape[0] or (groups and shape[0] != groups):
        raise ValueError(f"{name} must be [groups, {K}], with as many groups as the others, got {list(shape)}")
    groups = shape[0]
    ld, step = t.stride()
    if step != 1 or t.data_ptr() & 15 or (groups > 1 and (ld % 8 or ld < K)):
        t = t.clone(memory_format=torch.contiguous_format)
        ld = K
    return t, t.data_ptr(), groups, ld if groups > 1 else K


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
    for an update in place; other memory that overlaps neither it nor x) or to a new tensor.
    gate, scale, shift: bf16 [groups, K] (slices of a wider tensor may be given as they are; [K]
    for one group).  The group of row m is ``group_index[m]`` (int32; a row whose index is
    outside the groups, or negative where none of the three is given, is padding: not computed, its
    part of ``residual_out`` left as it was, of the new tensors undefined),
    else m // ``rows_per_group``; one of the two has to be given where there are several groups
    (a single one takes all rows).
    codes: "int8" (``q`` and ``a_scale``, for ``W8A8Linear.apply_codes``) or "mx4" (an ``MX4Tensor``, for
    ``MX4Linear``), equal to the codes of the bf16 output; None: y itself.  ``y=True`` gives y beside codes.
    """
    if rows_per_group is None and group_index is None:
        for t, name in ((gate, "gate"), (scale, "scale"), (shift, "shift")):
            if t is not None and t.dim() > 1 and t.shape[0] > 1:
                raise ValueError(f"{name} holds {t.shape[0]} groups: give rows_per_group or group_index")
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
    if _elsewhere(index, stream):
        with _there(index, stream):
            return block_norm(x, residual, post=post, gate=gate, residual_scale=residual_scale, pre=pre,
                              scale=scale, shift=shift, rows_per_group=rows_per_group,
                              group_index=group_index, codes=codes, y=y, residual_out=residual_out)
    x2, M, ldx = _rows_of(x)
    dense = torch.contiguous_format  # (a single row's stride may be any; the outputs' are those of dense rows)
    r2 = new = None
    ldr = ldro = dtype = 0
    if residual is not None:
        r2, _, ldr = _rows_of(residual)
        dtype, ldro = _RESIDUAL[residual.dtype], K
        if residual_out is None:
            new = torch.empty_like(residual, memory_format=dense)
        else:  # written in place: a view, never a copy
            new = residual_out
            n2 = new.view(-1, K) if new.is_contiguous() else new
            if n2.dim() != 2 or (M and n2.stride(1) != 1):
                raise ValueError("residual_out must be contiguous, or [rows, K] with unit stride along K")
            if M > 1:
                ldro = n2.stride(0)

    groups, held = 0, []
    gate_at = scale_at = shift_at = ld_gate = ld_scale = ld_shift = 0
    if gate is not None:
        gate, gate_at, groups, ld_gate = _per_group(gate, "gate", K, groups)
        held.append(gate)  # what a copy was made of, until the launch
    if scale is not None:
        scale, scale_at, groups, ld_scale = _per_group(scale, "scale", K, groups)
        held.append(scale)
    if shift is not None:
        shift, shift_at, groups, ld_shift = _per_group(shift, "shift", K, groups)
        held.append(shift)
    if group_index is not None:
        _need_cuda(group_index, "group_index", torch.int32)
        if group_index.numel() != M or not group_index.is_contiguous():
            raise ValueError(f"group_index must be contiguous and hold {M} values")
        groups = groups or 0x7FFFFFFF
    if rows_per_group is None:
        rows_per_group = M or 1

    out = q = a_scale = image = None
    if want_y:
        out = torch.empty_like(x, memory_format=dense)
    if codes == "int8":
        q = torch.empty_like(x, dtype=torch.int8, memory_format=dense)
        a_scale = torch.empty_strided((M,), (1,), dtype=torch.float32, device=index)
    elif codes == "mx4":
        image = _bytes(mx4_bytes(M, K) if M else 0, index)
    if M:
        args = _ARGS.pack(
            M, K, x2.data_ptr(), ldx, 0 if r2 is None else r2.data_ptr(), 0 if new is None else new.data_ptr(),
            ldr, ldro, dtype, residual_scale, *_vectors(post, K), *_vectors(pre, K),
            gate_at, scale_at, shift_at, ld_gate, ld_scale, ld_shift, groups, rows_per_group, 0 if group_index is None else group_index.data_ptr(),
            0 if out is None else out.data_ptr(), K, 0 if q is None else q.data_ptr(),
            0 if a_scale is None else a_scale.data_ptr(), 0 if image is None else image.data_ptr(),
            0 if image is None else image.numel())
        _check(lib().w8a8_block_norm(args, _raw_stream(index)), "w8a8_block_norm")
    return BlockNormOutput(new, out, q, a_scale, None if image is None else MX4Tensor(image, x.shape[:-1], K))
