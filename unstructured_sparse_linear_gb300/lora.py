"""Low-rank adapters: the product beside a shared projection, for many requests at once, and
its gradients.

RoSA adds a low-rank and a sparse update to one frozen projection (spops README, "Sparse
Operations (spops)"). The sparse half is csr_add / spmm / sddmm; this is the low-rank half:

    lora_add    Y = base + s_i (X A_i^T) B_i^T, adapter i chosen per token
    lora_grad   dX = dX_base + s_i (dY B_i) A_i,  dA_i = s_i (dY B_i)^T X,  dB_i = s_i dY^T (X A_i^T)

A is [adapters, rank, in], B [adapters, out, rank], X token-major [tokens, in]. The batch's
plan (``lora_plan``: its tokens sorted by adapter) is built once and serves every projection of
every layer. Activations may be column slices of a wider matrix (a fused projection): their
rows need unit stride inside and one row stride; everything else is contiguous.
"""
from __future__ import annotations

import struct
import threading

import torch

from torch.autograd.graph import increment_version

from . import _DTYPE, _L, _check, _req

__all__ = ["LoraPlan", "lora_plan", "lora_add", "lora_grad"]


_MAX_COUNT = 0x7fff0000  # SPOPS_LORA_MAX_COUNT

# spops_lora_add_args and spops_lora_grad_args
_ADD_ARGS = struct.Struct("12qf6i").pack
_GRAD_ARGS = struct.Struct("18qf6i").pack


def _raw_stream(index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index)


def _rows(t, name, rows, cols, dtype, device):
    """Checks a row-strided [rows, cols] operand; returns (address, row stride). The launch of a
    small call takes longer than its kernel, so the common case is a handful of tests."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == (rows, cols) and t.device == device:
        ld, step = t.stride()
        if step == 1 and ld >= cols:
            return t.data_ptr(), ld
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() != 2 or t.size(0) != rows or t.size(1) != cols:
        raise ValueError(f"{name} must be {rows} x {cols}, got {tuple(t.shape)}")
    ld, step = t.stride()
    if rows > 0 and ((step != 1 and cols > 1) or (ld < cols and rows > 1)):
        raise ValueError(f"{name} must have contiguous rows at least {cols} elements apart, got strides {(ld, step)}")
    return t.data_ptr(), ld


def _check_writable(t, name):
    """For a caller's tensor that requires a gradient: autograd believes to know its values, and the kernels write
    through its address."""
    if torch.is_grad_enabled():
        raise RuntimeError(f"{name} is part of an autograd graph, which would not see that it is written (RosaLinear is "
                           "the differentiable form; under torch.no_grad() it may be written)")


class Built:
    """A device table that is written on one stream and may be read on others. Kernels follow the
    addresses and indices in it, so a stream other than the one that wrote it waits for the writing
    before its first use (in a graph capture the table has to be complete: nothing can be waited
    for there that is not captured too), and the memory is kept until that stream is done with it."""

    def __init__(self, buf: torch.Tensor):
        self.device = buf.device
        self._buf = buf
        self._ptr = buf.data_ptr()
        self._streams = {_raw_stream(buf.device.index)}
        self._written = torch.cuda.Event()
        self._written.record(torch.cuda.current_stream(buf.device))

    def __reduce_ex__(self, protocol):  # (a copy's kernels would follow the original's addresses)
        raise TypeError(f"a {type(self).__name__} cannot be copied or pickled: it holds device addresses; make a new one")

    def _on_stream(self, stream: int) -> int:
        """The table's address, usable by work that is queued on `stream` from now on."""
        if stream not in self._streams and not torch.cuda.is_current_stream_capturing():
            s = torch.cuda.current_stream(self.device)
            s.wait_event(self._written)
            self._buf.record_stream(s)
            self._streams.add(stream)
        return self._ptr


class LoraPlan(Built):
    """Which tokens of a batch use which adapter, sorted; built by ``lora_plan``. A captured graph holds the
    plan's address and not the plan: keep it as long as the graph is replayed."""

    def __init__(self, buf: torch.Tensor, tokens: int, n_adapters: int):
        super().__init__(buf)
        self.buf, self.tokens, self.n_adapters = buf, tokens, n_adapters
        self._scratch = {}

    def _grad_scratch(self, rank: int, stream: int):
        """(buffer, address, bytes) of lora_grad's workspace on the current stream. It is kept for the calls
        of one thread on one stream, which come one after the other (allocating and freeing one took
        2 of a small call's 29 us); a graph capture has its own, as replays may run beside those."""
        capturing = torch._C._cuda_isCurrentStreamCapturing()
        key = (rank, stream, threading.get_ident())
        ws = None if capturing else self._scratch.get(key)
        if ws is None:
            size = int(_L().spops_lora_grad_workspace_size(self.tokens, rank))
            buf = torch.empty(size, dtype=torch.uint8, device=self.device)
            ws = (buf, buf.data_ptr(), size)
            if not capturing:
                self._scratch[key] = ws
        return ws

    def order(self) -> torch.Tensor:
        """The tokens sorted by adapter (stable; those without an adapter last), int32."""
        return self.buf[64:64 + 4 * self.tokens].view(torch.int32)


def lora_plan(adapter_ids: torch.Tensor | None, n_adapters: int, tokens: int | None = None,
              device=None) -> LoraPlan:
    """The plan of a batch (asynchronous on the current stream). adapter_ids: int32 [tokens], the
    adapter of each token in any order; an id outside 0 .. n_adapters - 1 (-1) means none.
    adapter_ids=None with tokens (and device): every token uses adapter 0, as in training."""
    if adapter_ids is None:
        if tokens is None:
            raise ValueError("lora_plan needs adapter_ids or tokens")
        dev = torch.device(device if device is not None else "cuda")
        if dev.type != "cuda":
            raise ValueError(f"device must be a CUDA device, got {dev}")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        ids = 0
    else:
        _req(adapter_ids, "adapter_ids", torch.int32)
        if adapter_ids.dim() != 1 or (tokens is not None and tokens != adapter_ids.numel()):
            raise ValueError(f"adapter_ids must be a vector with one id per token, got {tuple(adapter_ids.shape)}")
        tokens, dev, ids = adapter_ids.numel(), adapter_ids.device, adapter_ids.data_ptr()
    tokens, n_adapters = int(tokens), int(n_adapters)
    if not (0 <= tokens <= _MAX_COUNT and 1 <= n_adapters <= _MAX_COUNT):
        raise ValueError(f"need tokens >= 0 and n_adapters >= 1, at most {_MAX_COUNT} of each, got {tokens}, {n_adapters}")
    lib = _L()
    size = lib.spops_lora_plan_size(tokens, n_adapters)
    with torch.cuda.device(dev):
        buf = torch.empty(size, dtype=torch.uint8, device=dev)
        _check(lib.spops_lora_plan_build(ids, tokens, n_adapters, buf.data_ptr(), size, _raw_stream(dev.index)),
               "lora_plan_build")
        return LoraPlan(buf, tokens, n_adapters)


def _weights(X, A, B, plan, scale):
    """Checks shared by both calls; returns (device, dtype, in, out, rank, n, scale address, factor)."""
    if not isinstance(plan, LoraPlan):
        raise TypeError("plan must be a LoraPlan")
    dev = plan.device
    if not isinstance(X, torch.Tensor):
        raise TypeError("X must be a torch.Tensor")
    dt = X.dtype
    if X.device != dev:
        if not X.is_cuda:
            raise ValueError("X must be a CUDA tensor")
        raise ValueError(f"X is on {X.device} and the plan on {dev}")
    if dt not in _DTYPE:
        raise ValueError(f"X dtype {dt} not in {list(_DTYPE)}")
    if not (type(A) is torch.Tensor and A.dtype is dt and A.device == dev and A.is_contiguous()):
        _req(A, "A", dt, device=dev)  # (a Parameter, or what is wrong)
    if not (type(B) is torch.Tensor and B.dtype is dt and B.device == dev and B.is_contiguous()):
        _req(B, "B", dt, device=dev)
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be [adapters, rank, in] and B [adapters, out, rank]")
    n, rank, k = A.shape
    nb, n_out, rb = B.shape
    if nb != n or rb != rank:
        raise ValueError(f"A {tuple(A.shape)} and B {tuple(B.shape)} differ in adapters or rank")
    if plan.n_adapters != n:
        raise ValueError(f"plan was built for {plan.n_adapters} adapters, not {n}")
    if scale is None:
        return dev, dt, k, n_out, rank, n, 0, 1.0
    if isinstance(scale, torch.Tensor):
        _req(scale, "scale", torch.float32, device=dev)
        if scale.numel() != n:
            raise ValueError(f"scale must have one factor per adapter ({n}), got {scale.numel()}")
        return dev, dt, k, n_out, rank, n, scale.data_ptr(), 1.0
    return dev, dt, k, n_out, rank, n, 0, float(scale)


def _elsewhere(index: int) -> bool:
    """Whether another device than this one is current. (The calls then make it current and call
    themselves: a context entered by every call takes 0.6 us.)"""
    return torch._C._cuda_getDevice() != index


def lora_add(X, A, B, plan: LoraPlan, base=None, scale=None, out=None, return_h: bool = False):
    """Y = base + s_i (X A_i^T) B_i^T with the adapter i of each token (tokens without one: base).
    base: the shared projection's output (None: zeros); out=base adds in place. scale: a float,
    or an fp32 tensor with one factor per adapter. return_h: also return X A_i^T (fp32
    [tokens, rank]), which lora_grad takes. Autograd records nothing of it (RosaLinear is the form
    that it differentiates): an out that belongs to an autograd graph is refused."""
    dev, dt, k, n_out, rank, n, s_ptr, s_all = _weights(X, A, B, plan, scale)
    if _elsewhere(dev.index):
        with torch.cuda.device(dev):
            return lora_add(X, A, B, plan, base, scale, out, return_h)
    T = plan.tokens
    x, ldx = _rows(X, "X", T, k, dt, dev)
    b, ldb = _rows(base, "base", T, n_out, dt, dev) if base is not None else (0, n_out)
    lib = _L()
    given = False
    if out is None:
        out = torch.empty((T, n_out), dtype=dt, device=dev)
        y, ldy = out.data_ptr(), n_out
    else:
        y, ldy = _rows(out, "out", T, n_out, dt, dev)
        if out.requires_grad:
            _check_writable(out, "out")
        given = True
    h = torch.empty((T, rank), dtype=torch.float32, device=dev) if return_h else None
    stream = _raw_stream(dev.index)
    st = lib.spops_lora_add_block(_ADD_ARGS(
        x, ldx, A.data_ptr(), B.data_ptr(), s_ptr, b, ldb, y, ldy, h.data_ptr() if return_h else 0,
        plan._on_stream(stream), stream, s_all, _DTYPE[dt], T, k, n_out, rank, n))
    if st:
        _check(st, "lora_add")
    if given:  # (what autograd saved of it is no longer there)
        increment_version(out)
    return (out, h) if return_h else out


def _like(t, w, name):
    _req(t, name, w.dtype, device=w.device)
    if t.shape != w.shape:
        raise ValueError(f"{name} must be {tuple(w.shape)}, got {tuple(t.shape)}")
    return t


def lora_grad(dY, X, A, B, plan: LoraPlan, scale=None, h=None, dX_base=None, dX_out=None, dA_out=None, dB_out=None,
              need=(True, True, True)):
    """(dX, dA, dB) of lora_add for the output gradient dY. dX = dX_base + s_i (dY B_i) A_i, so the
    shared projection's own input gradient goes in as dX_base (dX_out=dX_base: in place). h: the
    one lora_add returned for this X (None: formed here). need: which of the three to compute;
    the others come back as None. dA_out, dB_out: buffers for the weights' gradients (such as those of
    a GradSet), overwritten; as dX_out, they may not belong to an autograd graph."""
    dev, dt, k, n_out, rank, n, s_ptr, s_all = _weights(X, A, B, plan, scale)
    if _elsewhere(dev.index):
        with torch.cuda.device(dev):
            return lora_grad(dY, X, A, B, plan, scale, h, dX_base, dX_out, dA_out, dB_out, need)
    T = plan.tokens
    x, ldx = _rows(X, "X", T, k, dt, dev)
    dy, lddy = _rows(dY, "dY", T, n_out, dt, dev)
    hp = 0
    if h is not None:
        hp, ldh = _rows(h, "h", T, rank, torch.float32, dev)
        if ldh != rank and T > 1:
            raise ValueError(f"h must be contiguous, got strides {h.stride()}")
    b, ldb = _rows(dX_base, "dX_base", T, k, dt, dev) if dX_base is not None else (0, k)
    lib = _L()
    dX = dA = dB = None
    dx, lddx = 0, k
    if need[0]:
        if dX_out is None:
            dX = torch.empty_like(X) if ldx == k and type(X) is torch.Tensor else torch.empty((T, k), dtype=dt, device=dev)
            dx = dX.data_ptr()
        else:
            dX = dX_out
            dx, lddx = _rows(dX, "dX_out", T, k, dt, dev)
    if need[1]:
        dA = _like(dA_out, A, "dA_out") if dA_out is not None else torch.empty_like(A)
    if need[2]:
        dB = _like(dB_out, B, "dB_out") if dB_out is not None else torch.empty_like(B)
    given = [t for t, use in ((dX_out, need[0]), (dA_out, need[1]), (dB_out, need[2])) if use and t is not None] \
        if dX_out is not None or dA_out is not None or dB_out is not None else ()
    for t in given:
        if t.requires_grad:
            _check_writable(t, "dX_out" if t is dX_out else "dA_out" if t is dA_out else "dB_out")
    stream = _raw_stream(dev.index)
    ws, ws_ptr, size = plan._grad_scratch(rank, stream)
    st = lib.spops_lora_grad_block(_GRAD_ARGS(
        dy, lddy, x, ldx, A.data_ptr(), B.data_ptr(), s_ptr, hp, b, ldb, dx, lddx,
        dA.data_ptr() if need[1] else 0, dB.data_ptr() if need[2] else 0, plan._on_stream(stream), ws_ptr, size,
        stream, s_all, _DTYPE[dt], T, k, n_out, rank, n))
    if st:
        _check(st, "lora_grad")
    for t in given:
        increment_version(t)
    return dX, dA, dB
