"""Microscaled 4-bit (MXFP4) layers: the binding of the ``w8a8_mx4_*`` entry points.

As in ``binding``, argument marshalling only.  Calls run on the device of
their tensors, whichever device is current, on ``stream`` or that device's
current stream; what a call allocates belongs to that stream.  A call with no
rows returns an empty result without a launch.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from .binding import ACT_NONE, _SZ, _check, _need_cuda, _ptr, lib


def _device(*tensors: Optional[torch.Tensor]) -> torch.device:
    """The one device that all the tensors given are on."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")
    return dev


@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device)
        else:
            with torch.cuda.stream(stream):  # what the call allocates is this stream's
                yield stream


class _Here:
    """The common case, without a context manager's cost: the tensors' device is current
    and the call goes to its current stream."""

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        return self.stream

    def __exit__(self, *exc):
        return False


def _on(device: torch.device, stream):
    if stream is None and device.index == torch.cuda.current_device():
        return _Here(torch.cuda.current_stream())
    if stream is not None and stream.device != device:
        raise ValueError(f"stream of {stream.device}, tensors on {device}")
    return _switched(device, stream)


def _size(name: str, *shape: int) -> int:
    out = _SZ()
    _check(getattr(lib(), name)(*shape, ctypes.byref(out)), name)
    return out.value


def mx4_bytes(rows: int, K: int) -> int:
    """Bytes of the image of a [rows, K] matrix."""
    return _size("w8a8_mx4_bytes", rows, K)


def mx4_scaled_mm_workspace_bytes(M: int, N: int, K: int) -> int:
    return _size("w8a8_mx4_scaled_mm_workspace_bytes", M, N, K)


def mx4_linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return _size("w8a8_mx4_linear_workspace_bytes", M, N, K)


class MX4Tensor:
    """A matrix in the 4-bit image: ``image`` (uint8), of [..., K] values with the
    leading sizes ``lead`` and ``rows`` rows in all."""

    __slots__ = ("image", "lead", "rows", "K")

    def __init__(self, image: torch.Tensor, lead: Tuple[int, ...], K: int):
        self.image, self.lead, self.K = image, tuple(lead), K
        self.rows = 1
        for n in self.lead:
            self.rows *= n

    @property
    def device(self) -> torch.device:
        return self.image.device

    def dequant(self, stream=None) -> torch.Tensor:
        return mx4_dequant(self, stream=stream)

    def unpack(self, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        return mx4_unpack(self, stream=stream)


def _rows_of(x: torch.Tensor) -> Tuple[torch.Tensor, int]:
    """[..., K] -> ([rows, K] with unit stride along K and rows on 16-byte boundaries, row stride)."""
    K = x.shape[-1]
    x2 = x.reshape(-1, K)
    if x2.stride(1) != 1 or (x2.shape[0] > 1 and (x2.stride(0) % 8 or x2.stride(0) < K)):
        x2 = x2.clone(memory_format=torch.contiguous_format)
    return x2, x2.stride(0) if x2.shape[0] > 1 else K


def _image(image: Optional[torch.Tensor], rows: int, K: int, device) -> torch.Tensor:
    need = mx4_bytes(rows, K) if rows else 0
    if image is None:
        return torch.empty((need,), dtype=torch.uint8, device=device)
    _need_cuda(image, "image", torch.uint8)
    if not image.is_contiguous():
        raise ValueError("image must be contiguous")
    return image


def mx4_quant(x: torch.Tensor, image: Optional[torch.Tensor] = None, stream=None) -> MX4Tensor:
    """bf16 [..., K] -> its 4-bit image (``image``: a uint8 buffer of ``mx4_bytes`` to write)."""
    _need_cuda(x, "x", torch.bfloat16)
    dev = _device(x, image)
    K = x.shape[-1]
    with _on(dev, stream) as s:
        x2, ldx = _rows_of(x)
        M = x2.shape[0]
        out = _image(image, M, K, dev)
        if M:
            _check(lib().w8a8_mx4_quant(_ptr(x2), M, K, ldx, _ptr(out), out.numel(),
                                        ctypes.c_void_p(s.cuda_stream)), "w8a8_mx4_quant")
    return MX4Tensor(out, x.shape[:-1], K)


def mx4_pack(codes: torch.Tensor, scales: torch.Tensor, image: Optional[torch.Tensor] = None,
             stream=None) -> MX4Tensor:
    """A checkpoint's codes (uint8 [rows, K/2], the lower k in the low half) and scale bytes
    (uint8 [rows, ceil(K/32)]) -> image."""
    _need_cuda(codes, "codes", torch.uint8)
    _need_cuda(scales, "scales", torch.uint8)
    dev = _device(codes, scales, image)
    rows, K = codes.shape[0], codes.shape[1] * 2
    if tuple(scales.shape) != (rows, (K + 31) // 32):
        raise ValueError(f"scales must be [{rows}, {(K + 31) // 32}], got {list(scales.shape)}")
    with _on(dev, stream) as s:
        codes, scales = codes.contiguous(), scales.contiguous()
        out = _image(image, rows, K, dev)
        if rows:
            _check(lib().w8a8_mx4_pack(_ptr(codes), _ptr(scales), rows, K, _ptr(out), out.numel(),
                                       ctypes.c_void_p(s.cuda_stream)), "w8a8_mx4_pack")
    return MX4Tensor(out, (rows,), K)


def _whole(t: MX4Tensor):
    """The image holds what its shape says (the library is not told its size)."""
    if t.rows and t.image.numel() < mx4_bytes(t.rows, t.K):
        raise ValueError(f"image of {t.image.numel()} bytes is too small for [{t.rows}, {t.K}]")


def mx4_unpack(t: MX4Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """image -> (codes [rows, K/2], scales [rows, ceil(K/32)]), the inverse of ``mx4_pack``."""
    _whole(t)
    with _on(t.device, stream) as s:
        codes = torch.empty((t.rows, t.K // 2), dtype=torch.uint8, device=t.device)
        scales = torch.empty((t.rows, (t.K + 31) // 32), dtype=torch.uint8, device=t.device)
        if t.rows:
            _check(lib().w8a8_mx4_unpack(_ptr(t.image), t.rows, t.K, _ptr(codes), _ptr(scales),
                                         ctypes.c_void_p(s.cuda_stream)), "w8a8_mx4_unpack")
    return codes, scales


def mx4_dequant(t: MX4Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values the image stands for, bf16 [..., K]."""
    _whole(t)
    _device(t.image, out)
    with _on(t.device, stream) as s:
        out = _output(out, t.rows, t.K, t.device)
        if t.rows:
            _check(lib().w8a8_mx4_dequant(_ptr(t.image), t.rows, t.K, _ptr(out),
                                          ctypes.c_void_p(s.cuda_stream)), "w8a8_mx4_dequant")
    return out.view(*t.lead, t.K)


def _output(out: Optional[torch.Tensor], M: int, N: int, device) -> torch.Tensor:
    if out is None:
        return torch.empty((M, N), dtype=torch.bfloat16, device=device)
    _need_cuda(out, "out", torch.bfloat16)
    if out.numel() != M * N or not out.is_contiguous():
        raise ValueError(f"out must be contiguous and hold [{M}, {N}]")
    return out


def _scratch(workspace: Optional[torch.Tensor], need: int, device) -> Tuple[Optional[torch.Tensor], int]:
    if workspace is None:
        return (torch.empty((need,), dtype=torch.uint8, device=device), need) if need else (None, 0)
    _need_cuda(workspace, "workspace")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def _weight(w: MX4Tensor, bias: Optional[torch.Tensor], K: int):
    _whole(w)
    if w.K != K:
        raise ValueError(f"x has K = {K}, the weight K = {w.K}")
    if bias is not None:
        _need_cuda(bias, "bias", torch.bfloat16)
        if bias.numel() != w.rows or not bias.is_contiguous():
            raise ValueError(f"bias must be contiguous and hold {w.rows} values")


def mx4_scaled_mm(a: MX4Tensor, w: MX4Tensor, bias: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None, act: int = ACT_NONE) -> torch.Tensor:
    """The product of a [..., K] with a weight [N, K]: y bf16 [..., N] (``act``: epilogue activation)."""
    _whole(a)
    _weight(w, bias, a.K)
    dev = _device(a.image, w.image, bias, out, workspace)
    M, N, K = a.rows, w.rows, a.K
    with _on(dev, stream) as s:
        out = _output(out, M, N, dev)
        if M:
            ws, nbytes = _scratch(workspace, mx4_scaled_mm_workspace_bytes(M, N, K), dev)
            _check(lib().w8a8_mx4_scaled_mm(_ptr(a.image), _ptr(w.image), _ptr(bias), _ptr(out), M, N, K,
                                            act, _ptr(ws), nbytes, ctypes.c_void_p(s.cuda_stream)),
                   "w8a8_mx4_scaled_mm")
    return out.view(*a.lead, N)


def mx4_scaled_mm_quant(a: MX4Tensor, w: MX4Tensor, bias: Optional[torch.Tensor] = None,
                        image: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None, act: int = ACT_NONE) -> MX4Tensor:
    """``mx4_quant(mx4_scaled_mm(...))`` in one kernel: the image of y, the next product's operand."""
    _whole(a)
    _weight(w, bias, a.K)
    dev = _device(a.image, w.image, bias, image, workspace)
    M, N, K = a.rows, w.rows, a.K
    with _on(dev, stream) as s:
        out = _image(image, M, N, dev)
        if M:
            ws, nbytes = _scratch(workspace, mx4_scaled_mm_workspace_bytes(M, N, K), dev)
            _check(lib().w8a8_mx4_scaled_mm_quant(_ptr(a.image), _ptr(w.image), _ptr(bias), _ptr(out),
                                                  out.numel(), M, N, K, act, _ptr(ws), nbytes,
                                                  ctypes.c_void_p(s.cuda_stream)),
                   "w8a8_mx4_scaled_mm_quant")
    return MX4Tensor(out, a.lead, N)


def mx4_linear(x: torch.Tensor, w: MX4Tensor, bias: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None, act: int = ACT_NONE) -> torch.Tensor:
    """The whole layer: y[..., N] = x[..., K] quantised, times w (``act``: epilogue activation)."""
    _need_cuda(x, "x", torch.bfloat16)
    _weight(w, bias, x.shape[-1])
    dev = _device(x, w.image, bias, out, workspace)
    with _on(dev, stream) as s:
        x2, ldx = _rows_of(x)
        M, N, K = x2.shape[0], w.rows, w.K
        out = _output(out, M, N, dev)
        if M:
            ws, nbytes = _scratch(workspace, mx4_linear_workspace_bytes(M, N, K), dev)
            _check(lib().w8a8_mx4_linear(_ptr(x2), ldx, _ptr(w.image), _ptr(bias), _ptr(out), M,
                                         N, K, act, _ptr(ws), nbytes, ctypes.c_void_p(s.cuda_stream)),
                   "w8a8_mx4_linear")
    return out.view(*x.shape[:-1], N)


def mx4_linear_quant(x: torch.Tensor, w: MX4Tensor, bias: Optional[torch.Tensor] = None,
                     image: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None, act: int = ACT_NONE) -> MX4Tensor:
    """A layer whose output feeds another 4-bit layer: the image of y, equal to
    ``mx4_quant(mx4_linear(...))``."""
    _need_cuda(x, "x", torch.bfloat16)
    _weight(w, bias, x.shape[-1])
    dev = _device(x, w.image, bias, image, workspace)
    with _on(dev, stream) as s:
        x2, ldx = _rows_of(x)
        M, N, K = x2.shape[0], w.rows, w.K
        out = _image(image, M, N, dev)
        if M:
            ws, nbytes = _scratch(workspace, mx4_linear_workspace_bytes(M, N, K), dev)
            _check(lib().w8a8_mx4_linear_quant(_ptr(x2), ldx, _ptr(w.image), _ptr(bias),
                                               _ptr(out), out.numel(), M, N, K, act, _ptr(ws), nbytes,
                                               ctypes.c_void_p(s.cuda_stream)), "w8a8_mx4_linear_quant")
    return MX4Tensor(out, x.shape[:-1], N)


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

    def __call__(self, x, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """x: bf16 [..., K] or an MX4Tensor -> y bf16 [..., N]."""
        f = mx4_scaled_mm if isinstance(x, MX4Tensor) else mx4_linear
        return f(x, self.w, self.bias, out=out, stream=stream, act=self.act)

    def quantised(self, x, image: Optional[torch.Tensor] = None, stream=None) -> MX4Tensor:
        """The same output, in the form the next 4-bit layer takes."""
        f = mx4_scaled_mm_quant if isinstance(x, MX4Tensor) else mx4_linear_quant
        return f(x, self.w, self.bias, image=image, stream=stream, act=self.act)
