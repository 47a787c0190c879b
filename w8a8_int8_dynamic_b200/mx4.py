"""Microscaled 4-bit (MXFP4) layers: the binding of the ``w8a8_mx4_*`` entry points.

As in ``binding``, argument marshalling only.  Calls run on the device of
their tensors, whichever device is current, on ``stream`` or that device's
current stream; what a call allocates belongs to that stream.  A call with no
rows returns an empty result without a launch.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from .binding import (ACT_NONE, _at, _bytes, _check, _device, _elsewhere, _need_cuda, _new, _raw_stream, _rows_of,
                      _size, _there, lib)


def mx4_bytes(rows: int, K: int) -> int:
    """Bytes of the image of a [rows, K] matrix."""
    return _size("w8a8_mx4_bytes", 0, rows, K)


def mx4_linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return _size("w8a8_mx4_linear_workspace_bytes", torch.cuda.current_device(), M, N, K)


class MX4Tensor:
    """A matrix in the 4-bit image: ``image`` (uint8), of [..., K] values with the
    leading sizes ``lead`` and ``rows`` rows in all."""

    __slots__ = ("image", "lead", "rows", "K")

    def __init__(self, image: torch.Tensor, lead: Tuple[int, ...], K: int):
        self.image, self.lead, self.K = image, tuple(lead), K
        self.rows = math.prod(self.lead)

    @property
    def device(self) -> torch.device:
        return self.image.device

    def dequant(self, stream=None) -> torch.Tensor:
        return mx4_dequant(self, stream=stream)

    def unpack(self, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        return mx4_unpack(self, stream=stream)


def _image(image: Optional[torch.Tensor], rows: int, K: int, index: int) -> torch.Tensor:
    if image is None:
        return _bytes(mx4_bytes(rows, K) if rows else 0, index)
    _need_cuda(image, "image", torch.uint8)
    if not image.is_contiguous():
        raise ValueError("image must be contiguous")
    return image


def _output(out: Optional[torch.Tensor], lead: Tuple[int, ...], N: int, index: int) -> torch.Tensor:
    """A new [*lead, N], or ``out`` seen as one."""
    if out is None:
        return _new(lead, N, torch.bfloat16, index)
    _need_cuda(out, "out", torch.bfloat16)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    return out.view(*lead, N)


def _image_of_x(x2: torch.Tensor, M: int, K: int, ldx: int, out: Optional[torch.Tensor]) -> int:
    """Bytes of workspace that a layer needs: up to 16 rows none, but where the output is in x's place."""
    if M <= 16:
        if out is None:
            return 0
        first, last = x2.data_ptr(), x2.data_ptr() + 2 * ((M - 1) * ldx + K)
        if out.data_ptr() >= last or first >= out.data_ptr() + out.numel() * out.element_size():
            return 0
    return mx4_bytes(M, K)


def _scratch(workspace: Optional[torch.Tensor], need: int, index: int) -> Tuple[Optional[torch.Tensor], int]:
    if workspace is None:
        return (_bytes(need, index), need) if need else (None, 0)
    _need_cuda(workspace, "workspace")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def _whole(t: MX4Tensor):
    """The image holds what its shape says (the library is not told its size)."""
    if t.rows and t.image.numel() < mx4_bytes(t.rows, t.K):
        raise ValueError(f"image of {t.image.numel()} bytes is too small for [{t.rows}, {t.K}]")


def _weight(w: MX4Tensor, bias: Optional[torch.Tensor], K: int):
    _whole(w)
    if w.K != K:
        raise ValueError(f"x has K = {K}, the weight K = {w.K}")
    if bias is not None:
        _need_cuda(bias, "bias", torch.bfloat16)
        if bias.numel() != w.rows or not bias.is_contiguous():
            raise ValueError(f"bias must be contiguous and hold {w.rows} values")


def mx4_quant(x: torch.Tensor, image: Optional[torch.Tensor] = None, stream=None) -> MX4Tensor:
    """bf16 [..., K] -> its 4-bit image (``image``: a uint8 buffer of ``mx4_bytes`` to write)."""
    _need_cuda(x, "x", torch.bfloat16)
    index, K = _device(x, image), x.shape[-1]
    if _elsewhere(index, stream):
        with _there(index, stream):
            return mx4_quant(x, image)
    s = _raw_stream(index)
    x2, M, ldx = _rows_of(x)
    out = _image(image, M, K, index)
    if M:
        _check(lib().w8a8_mx4_quant(x2.data_ptr(), M, K, ldx, out.data_ptr(), out.numel(), s),
               "w8a8_mx4_quant")
    return MX4Tensor(out, x.shape[:-1], K)


def mx4_pack(codes: torch.Tensor, scales: torch.Tensor, image: Optional[torch.Tensor] = None,
             stream=None) -> MX4Tensor:
    """A checkpoint's codes (uint8 [rows, K/2], the lower k in the low half) and scale bytes
    (uint8 [rows, ceil(K/32)]) -> image."""
    _need_cuda(codes, "codes", torch.uint8)
    _need_cuda(scales, "scales", torch.uint8)
    if codes.dim() != 2:
        raise ValueError(f"codes must be [rows, K/2], got {list(codes.shape)}")
    index = _device(codes, scales, image)
    rows, K = codes.shape[0], codes.shape[1] * 2
    if tuple(scales.shape) != (rows, (K + 31) // 32):
        raise ValueError(f"scales must be [{rows}, {(K + 31) // 32}], got {list(scales.shape)}")
    if _elsewhere(index, stream):
        with _there(index, stream):
            return mx4_pack(codes, scales, image)
    s = _raw_stream(index)
    c, e = codes.contiguous(), scales.contiguous()
    if c.data_ptr() & 15:
        c = c.clone()
    out = _image(image, rows, K, index)
    if rows:
        _check(lib().w8a8_mx4_pack(c.data_ptr(), e.data_ptr(), rows, K, out.data_ptr(), out.numel(), s),
               "w8a8_mx4_pack")
    return MX4Tensor(out, (rows,), K)


def mx4_unpack(t: MX4Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """image -> (codes [rows, K/2], scales [rows, ceil(K/32)]), the inverse of ``mx4_pack``."""
    _whole(t)
    index = _device(t.image)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return mx4_unpack(t)
    s = _raw_stream(index)
    codes = torch.empty((t.rows, t.K // 2), dtype=torch.uint8, device=index)
    scales = torch.empty((t.rows, (t.K + 31) // 32), dtype=torch.uint8, device=index)
    if t.rows:
        _check(lib().w8a8_mx4_unpack(t.image.data_ptr(), t.rows, t.K, codes.data_ptr(), scales.data_ptr(),
                                     s), "w8a8_mx4_unpack")
    return codes, scales


def mx4_dequant(t: MX4Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values the image stands for, bf16 [..., K]."""
    _whole(t)
    index = _device(t.image, out)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return mx4_dequant(t, out)
    s = _raw_stream(index)
    x = _output(out, t.lead, t.K, index)
    if t.rows:
        _check(lib().w8a8_mx4_dequant(t.image.data_ptr(), t.rows, t.K, x.data_ptr(), s), "w8a8_mx4_dequant")
    return x


def mx4_scaled_mm(a: MX4Tensor, w: MX4Tensor, bias: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, stream=None, act: int = ACT_NONE) -> torch.Tensor:
    """The product of a [..., K] with a weight [N, K]: y bf16 [..., N] (``act``: epilogue activation)."""
    _whole(a)
    _weight(w, bias, a.K)
    index = _device(a.image, w.image, bias, out)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return mx4_scaled_mm(a, w, bias, out, act=act)
    s = _raw_stream(index)
    M, N, K = a.rows, w.rows, a.K
    y = _output(out, a.lead, N, index)
    if M:
        _check(lib().w8a8_mx4_scaled_mm(a.image.data_ptr(), w.image.data_ptr(), _at(bias), y.data_ptr(), M,
                                        N, K, act, s), "w8a8_mx4_scaled_mm")
    return y


def mx4_scaled_mm_quant(a: MX4Tensor, w: MX4Tensor, bias: Optional[torch.Tensor] = None,
                        image: Optional[torch.Tensor] = None, stream=None,
                        act: int = ACT_NONE) -> MX4Tensor:
    """``mx4_quant(mx4_scaled_mm(...))`` in one kernel: the image of y, the next product's operand."""
    _whole(a)
    _weight(w, bias, a.K)
    index = _device(a.image, w.image, bias, image)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return mx4_scaled_mm_quant(a, w, bias, image, act=act)
    s = _raw_stream(index)
    M, N, K = a.rows, w.rows, a.K
    y = _image(image, M, N, index)
    if M:
        _check(lib().w8a8_mx4_scaled_mm_quant(a.image.data_ptr(), w.image.data_ptr(), _at(bias),
                                              y.data_ptr(), y.numel(), M, N, K, act, s),
               "w8a8_mx4_scaled_mm_quant")
    return MX4Tensor(y, a.lead, N)


def mx4_linear(x: torch.Tensor, w: MX4Tensor, bias: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None, act: int = ACT_NONE) -> torch.Tensor:
    """The whole layer: y[..., N] = x[..., K] quantised, times w (``act``: epilogue activation).
    ``out`` may be x or overlap it."""
    _weight(w, bias, x.shape[-1])
    return _linear(x, w, bias, out, workspace, stream, act)


def _linear(x, w, bias, out, workspace, stream, act):
    """``mx4_linear`` with a weight and bias that have been checked."""
    _need_cuda(x, "x", torch.bfloat16)
    index = _device(x, w.image, bias, out, workspace)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return _linear(x, w, bias, out, workspace, None, act)
    x2, M, ldx = _rows_of(x)
    N, K = w.rows, w.K
    y = _output(out, x.shape[:-1], N, index)
    if M:
        ws, nbytes = _scratch(workspace, _image_of_x(x2, M, K, ldx, out), index)
        _check(lib().w8a8_mx4_linear(x2.data_ptr(), ldx, w.image.data_ptr(), _at(bias), y.data_ptr(), M, N, K,
                                     act, _at(ws), nbytes, _raw_stream(index)), "w8a8_mx4_linear")
    return y


def mx4_linear_quant(x: torch.Tensor, w: MX4Tensor, bias: Optional[torch.Tensor] = None,
                     image: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None, act: int = ACT_NONE) -> MX4Tensor:
    """A layer whose output feeds another 4-bit layer: the image of y, equal to
    ``mx4_quant(mx4_linear(...))``."""
    _weight(w, bias, x.shape[-1])
    return _linear_quant(x, w, bias, image, workspace, stream, act)


def _linear_quant(x, w, bias, image, workspace, stream, act):
    """``mx4_linear_quant`` with a weight and bias that have been checked."""
    _need_cuda(x, "x", torch.bfloat16)
    index = _device(x, w.image, bias, image, workspace)
    if _elsewhere(index, stream):
        with _there(index, stream):
            return _linear_quant(x, w, bias, image, workspace, None, act)
    x2, M, ldx = _rows_of(x)
    N, K = w.rows, w.K
    y = _image(image, M, N, index)
    if M:
        ws, nbytes = _scratch(workspace, _image_of_x(x2, M, K, ldx, image), index)
        _check(lib().w8a8_mx4_linear_quant(x2.data_ptr(), ldx, w.image.data_ptr(), _at(bias), y.data_ptr(),
                                           y.numel(), M, N, K, act, _at(ws), nbytes, _raw_stream(index)),
               "w8a8_mx4_linear_quant")
    return MX4Tensor(y, x.shape[:-1], N)


class MX4Linear:
    """A 4-bit linear layer: a checkpoint's codes and scale bytes (or, with
    :meth:`from_float`, a bf16 weight quantised here) laid out once, then
    applied to bf16 activations or to an ``MX4Tensor`` that an earlier layer
    or norm has formed.  The layer keeps no scratch memory, so one layer may
    be called on several streams and captured in several graphs."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 act: int = ACT_NONE):
        self._set(mx4_pack(codes, scales), bias, act)

    @classmethod
    def from_float(cls, w: torch.Tensor, bias: Optional[torch.Tensor] = None, act: int = ACT_NONE):
        self = cls.__new__(cls)
        self._set(mx4_quant(w), bias, act)
        return self

    def _set(self, w: MX4Tensor, bias, act):
        self.w, self.act = w, act
        self.N, self.K = w.rows, w.K
        self.bias = None if bias is None else bias.to(device=w.device, dtype=torch.bfloat16).contiguous()
        _weight(w, self.bias, self.K)

    def __call__(self, x, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """x: bf16 [..., K] or an MX4Tensor -> y bf16 [..., N]."""
        if isinstance(x, MX4Tensor):
            return mx4_scaled_mm(x, self.w, self.bias, out=out, stream=stream, act=self.act)
        if x.shape[-1] != self.K:
            raise ValueError(f"x has K = {x.shape[-1]}, the weight K = {self.K}")
        return _linear(x, self.w, self.bias, out, None, stream, self.act)

    def quantised(self, x, image: Optional[torch.Tensor] = None, stream=None) -> MX4Tensor:
        """The same output, in the form the next 4-bit layer takes."""
        if isinstance(x, MX4Tensor):
            return mx4_scaled_mm_quant(x, self.w, self.bias, image=image, stream=stream, act=self.act)
        if x.shape[-1] != self.K:
            raise ValueError(f"x has K = {x.shape[-1]}, the weight K = {self.K}")
        return _linear_quant(x, self.w, self.bias, image, None, stream, self.act)
