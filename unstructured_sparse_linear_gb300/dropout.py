"""Dropout from a counter-based generator, without a stored mask.

    Y = base + keep X / (1 - p)

The mask is a function of the state (a seed and a call number) and of the place in the matrix: the same state gives the
same mask whatever the type, the strides or the launch, so the backward pass forms it again. RosaLinear uses it in front
of the low-rank factors.
"""
from __future__ import annotations

import struct

import torch

from torch.autograd.graph import increment_version

from . import _DTYPE, _L, _check, _req
from .lora import _check_writable, _elsewhere, _raw_stream, _rows

__all__ = ["dropout"]

_MAX_COUNT = 0x7fffffff
_ARGS = struct.Struct("7q2QQd3i").pack  # spops_dropout_args


def dropout(X: torch.Tensor, p: float, state, base: torch.Tensor | None = None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = base + keep X / (1 - p) for X [rows, cols] (fp32, fp16 or bf16; rows may lie one stride apart), base None:
    zeros. state: (seed, call), two numbers of 64 bits, or a contiguous int64 CUDA tensor of the two, which a captured
    graph's replays read anew. p is taken in steps of 2^-16 (the factor too, so that the mean stays); the number of each
    place is that of Philox4x32-7, eight columns a step (see the C header). Dropped values are zero whatever they were.
    The gradient is the same call on the output's. out=X or out=base: in place. Autograd records nothing of it
    (RosaLinear(dropout=p) is differentiable): an out that belongs to an autograd graph is refused."""
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
    index = dev.index
    if _elsewhere(index):
        with torch.cuda.device(dev):
            return dropout(X, p, state, base, out)
    rows, cols = X.shape
    if rows > _MAX_COUNT or cols > _MAX_COUNT:
        raise ValueError(f"at most {_MAX_COUNT} rows and columns, got {rows} and {cols}")
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must lie in [0, 1], got {p}")
    at = seed = call = 0
    if isinstance(state, torch.Tensor):
        if not (state.dtype is torch.int64 and state.device == dev and state.numel() == 2 and state.is_contiguous()):
            _req(state, "state", torch.int64, device=dev)
            raise ValueError(f"state must hold a seed and a call number, got {tuple(state.shape)}")
        at = state.data_ptr()
    else:
        seed, call = (int(v) for v in state)
        if not (0 <= seed < 2 ** 64 and 0 <= call < 2 ** 64):
            raise ValueError(f"seed and call must lie in [0, 2^64), got {seed} and {call}")
    ldx, step = X.stride()
    x = X.data_ptr()
    if step != 1 or ldx < cols:  # (one column or row, or what is wrong)
        x, ldx = _rows(X, "X", rows, cols, dt, dev)
    b, ldb = _rows(base, "base", rows, cols, dt, dev) if base is not None else (0, cols)
    given = out is not None
    if given:
        y, ldy = _rows(out, "out", rows, cols, dt, dev)
        if out.requires_grad:
            _check_writable(out, "out")
    else:
        out = torch.empty_like(X) if ldx == cols and step == 1 and type(X) is torch.Tensor else \
            torch.empty((rows, cols), dtype=dt, device=dev)
        y, ldy = out.data_ptr(), cols
    st = _L().spops_dropout(_ARGS(x, ldx, b, ldb, y, ldy, at, seed, call, _raw_stream(index), p, code, rows, cols))
    if st:
        _check(st, "dropout")
    if given:
        increment_version(out)
    return out
