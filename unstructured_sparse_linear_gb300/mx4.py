"""Frozen weights in microscaled 4-bit floating point, and their products.

    mx4_quantize     W as blocks of 32 values: E2M1 codes and one power of two (E8M0) each
    mx4_dequantize   the values again
    mx4_linear       Y = X W^T
    mx4_linear_grad  dX = dY W

RoSA's adapters are trained beside a frozen projection (spops README, "Sparse Operations (spops)"), which takes most
of the memory: 4.25 bits a value instead of 16. Activations are token-major; they may be column slices of a wider
matrix (unit stride inside a row, one row stride).
"""
from __future__ import annotations

import struct

import torch

from torch.autograd.graph import increment_version

from . import _DTYPE, _L, _check, _req
from .lora import _check_writable, _elsewhere, _raw_stream, _rows

__all__ = ["Mx4", "mx4_quantize", "mx4_dequantize", "mx4_linear", "mx4_linear_grad"]

BLOCK = 32
_MAX_COUNT = 0x7fff0000  # SPOPS_MX4_MAX_COUNT
_ARGS = struct.Struct("9q4i").pack  # spops_mx4_args


class Mx4:
    """A weight [rows, cols] in 4 bits. codes: uint8 [rows, 16 * blocks], blocks = ceil(cols / 32), two codes a byte,
    the first in the low four bits (behind the last column: zeros); scales: uint8 [rows, blocks], 2^(b - 127) (255:
    NaN). dtype: the type that ``mx4_dequantize`` gives (that of the weight it was made of); the products use the
    values in the activations' type."""

    __slots__ = ("_codes", "_scales", "_shape", "dtype", "device")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int, dtype: torch.dtype = torch.bfloat16):
        _req(codes, "codes", torch.uint8)
        _req(scales, "scales", torch.uint8, device=codes.device)
        cols = int(cols)
        if dtype not in _DTYPE:
            raise ValueError(f"dtype {dtype} not in {list(_DTYPE)}")
        blocks = -(-cols // BLOCK)
        if codes.dim() != 2 or cols < 0 or codes.shape[1] != 16 * blocks or scales.shape != (codes.shape[0], blocks):
            raise ValueError(f"{cols} columns are {blocks} blocks: codes must be [rows, {16 * blocks}] and scales "
                             f"[rows, {blocks}], got {tuple(codes.shape)} and {tuple(scales.shape)}")
        if codes.shape[0] > _MAX_COUNT or cols > _MAX_COUNT:
            raise ValueError(f"at most {_MAX_COUNT} rows and columns, got {codes.shape[0]} and {cols}")
        self._codes, self._scales, self._shape = codes, scales, (codes.shape[0], cols)
        self.dtype, self.device = dtype, codes.device

    @classmethod
    def _of(cls, codes, scales, shape, dtype, device):  # (of a conversion: nothing to check)
        W = object.__new__(cls)
        W._codes, W._scales, W._shape, W.dtype, W.device = codes, scales, shape, dtype, device
        return W

    def __setstate__(self, state):  # (one from a file is where its arrays were brought to)
        for part in state:
            for name, value in (part or {}).items():
                setattr(self, name, value)
        self.device = self._codes.device

    @property
    def codes(self) -> torch.Tensor:
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        return self._scales

    @property
    def shape(self):
        return self._shape

    def __repr__(self):
        return f"Mx4({self._shape[0]} x {self._shape[1]}, {self.dtype}, {self.device})"


def _given(out, name, rows, cols, dtype, device):
    """(address, row stride) of an output that the caller gave."""
    at = _rows(out, name, rows, cols, dtype, device)
    if out.requires_grad:
        _check_writable(out, name)
    return at


def _weight(W):
    if type(W) is not Mx4 and not isinstance(W, Mx4):
        raise TypeError(f"W must be an Mx4, got {type(W).__name__}")
    if W.device.index is None:  # (loaded without its device)
        raise ValueError(f"W is on {W.device}: it must be on a CUDA device")
    return W


def mx4_quantize(X: torch.Tensor) -> Mx4:
    """The rows of X (fp32, fp16 or bf16, [rows, cols]) in 4 bits: a block's scale is the power of two of its largest
    magnitude's exponent less two, its values are rounded to the nearest code (ties to the even one, beyond the last to
    the last). A block that holds an infinity or a NaN is NaN as a whole."""
    if not isinstance(X, torch.Tensor):
        raise TypeError("X must be a torch.Tensor")
    dev, dt = X.device, X.dtype
    if dev.type != "cuda":
        raise ValueError("X must be a CUDA tensor")
    code = _DTYPE.get(dt)
    if code is None:
        raise ValueError(f"X dtype {dt} not in {list(_DTYPE)}")
    if X.dim() != 2:
        raise ValueError(f"X must be 2-D, got {tuple(X.shape)}")
    rows, cols = X.shape
    if rows > _MAX_COUNT or cols > _MAX_COUNT:
        raise ValueError(f"at most {_MAX_COUNT} rows and columns, got {rows} and {cols}")
    if _elsewhere(dev.index):
        with torch.cuda.device(dev):
            return mx4_quantize(X)
    x, ldx = _rows(X, "X", rows, cols, dt, dev)
    blocks = -(-cols // BLOCK)
    codes = torch.empty((rows, 16 * blocks), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, blocks), dtype=torch.uint8, device=dev)
    st = _L().spops_mx4_quantize(x, ldx, code, rows, cols, codes.data_ptr(), scales.data_ptr(),
                                 _raw_stream(dev.index))
    if st:
        _check(st, "mx4_quantize")
    return Mx4._of(codes, scales, (rows, cols), dt, dev)


def mx4_dequantize(W: Mx4, dtype: torch.dtype | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """W's values as a dense [rows, cols] matrix of `dtype` (default: W's): exact, but where they leave its range."""
    rows, cols = _weight(W).shape
    if dtype is None:
        dtype = getattr(out, "dtype", W.dtype)
    if dtype not in _DTYPE:
        raise ValueError(f"dtype {dtype} not in {list(_DTYPE)}")
    dev, given = W.device, out is not None
    if _elsewhere(dev.index):
        with torch.cuda.device(dev):
            return mx4_dequantize(W, dtype, out)
    if given:
        y, ldy = _given(out, "out", rows, cols, dtype, dev)
    else:
        out = torch.empty((rows, cols), dtype=dtype, device=dev)
        y, ldy = out.data_ptr(), cols
    st = _L().spops_mx4_dequantize(W._codes.data_ptr(), W._scales.data_ptr(), rows, cols, y, ldy, _DTYPE[dtype],
                                   _raw_stream(dev.index))
    if st:
        _check(st, "mx4_dequantize")
    if given:
        increment_version(out)
    return out


def _product(X, W, out, back, name):
    rows, cols = _weight(W)._shape
    n_in, n_out = (rows, cols) if back else (cols, rows)
    dev = W.device
    if not isinstance(X, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dt = X.dtype
    code = _DTYPE.get(dt)
    if code is None:
        raise ValueError(f"{name} dtype {dt} not in {list(_DTYPE)}")
    if X.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(X.shape)}")
    tokens = X.shape[0]
    if tokens > _MAX_COUNT:
        raise ValueError(f"at most {_MAX_COUNT} tokens, got {tokens}")
    index = dev.index
    if _elsewhere(index):
        with torch.cuda.device(dev):
            return _product(X, W, out, back, name)
    x, ldx = _rows(X, name, tokens, n_in, dt, dev)
    given = out is not None
    if given:
        y, ldy = _given(out, "out", tokens, n_out, dt, dev)
    else:
        out = torch.empty((tokens, n_out), dtype=dt, device=dev)
        y, ldy = out.data_ptr(), n_out
    lib = _L()
    ws, size = 0, 0
    # the parts of fp32, and rows that the tensor cores' kernel gets copies of
    if dt is torch.float32 or (x | y | 2 * ldx | 2 * ldy) & 15 or (n_in | n_out) & 7:
        size = lib.spops_mx4_workspace_size(tokens, n_in, n_out, code)
        scratch = torch.empty(size, dtype=torch.uint8, device=dev)
        ws = scratch.data_ptr()
    st = (lib.spops_mx4_linear_grad if back else lib.spops_mx4_linear)(_ARGS(
        x, ldx, W._codes.data_ptr(), W._scales.data_ptr(), y, ldy, ws, size, _raw_stream(index), code, tokens,
        rows, cols))
    if st:
        _check(st, "mx4_linear_grad" if back else "mx4_linear")
    if given:  # (what autograd saved of it is no longer there)
        increment_version(out)
    return out


def mx4_linear(X: torch.Tensor, W: Mx4, out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X W^T for X [tokens, cols] (on the tensor cores; fp32 as three bf16 parts: all 24 bits, below 2^-110 to the
    nearest multiple of 2^-133), W's values in X's type, fp32 sums. Autograd records nothing of it (RosaLinear is the form
    that it differentiates): an out that belongs to an autograd graph is refused."""
    return _product(X, W, out, False, "X")


def mx4_linear_grad(dY: torch.Tensor, W: Mx4, out: torch.Tensor | None = None) -> torch.Tensor:
    """dX = dY W, the input gradient of ``mx4_linear`` for the output gradient dY [tokens, rows]."""
    return _product(dY, W, out, True, "dY")
