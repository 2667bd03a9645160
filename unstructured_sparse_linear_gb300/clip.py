"""The global 2-norm of many gradients, and clipping by it.

    norm = sqrt(sum of g^2 over every gradient),  g <- g min(1, max_norm / (norm + 1e-6))

The step between an adapter's gradients (sddmm, lora_grad) and masked_adam. One kernel launch
whatever the number of tensors (two for the norm alone), and nothing is read back to the host: the norm stays on the
device. A training loop whose gradient buffers stay where they are keeps a ``GradSet`` of them.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.graph import increment_version

from . import _DTYPE, _L, _check, _req
from .lora import Built, _elsewhere, _raw_stream

__all__ = ["GradSet", "grad_norm", "clip_grads"]


class GradSet(Built):
    """Gradients that are clipped together (fp32, fp16 and bf16 mixed; contiguous; on one
    device). Holds the tensors and a device table of their addresses, so it serves every step
    that writes its gradients into the same buffers; new buffers need a new set (0.85 ms for 672
    tensors). A captured graph holds its address: keep it as long as the graph is replayed. out: tensors
    of the same sizes and types that receive the clipped gradients (default: in place). The set
    keeps the calls' partial sums, so calls on one set run one after the other (on one stream, or on
    streams that wait for each other)."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError(f"{len(self.grads)} gradients and {len(self.out)} outputs")
        n = len(self.grads)
        if n:
            _req(self.grads[0], "gradient 0", dtypes=_DTYPE)
        dev = self.grads[0].device if n else torch.device("cuda", torch.cuda.current_device())
        ins, outs, counts, dtypes = [], [], [], []
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            # (an address, a size and a type each; what is wrong is found out where something is)
            if not (type(g) is torch.Tensor and g.dtype in _DTYPE and g.device == dev and g.is_contiguous()):
                _req(g, f"gradient {i}", dtypes=_DTYPE, device=dev)
            count, dt = g.numel(), g.dtype
            ins.append(g.data_ptr())
            counts.append(count)
            dtypes.append(_DTYPE[dt])
            if o is g:
                outs.append(ins[-1])
                continue
            if not (type(o) is torch.Tensor and o.dtype is dt and o.device == dev and o.is_contiguous()):
                _req(o, f"output {i}", dtype=dt, device=dev)
            if o.numel() != count:
                raise ValueError(f"gradient {i} has {count} elements and its output {o.numel()}")
            outs.append(o.data_ptr())
        lib = _L()
        size = lib.spops_grad_set_size(n)
        self._n, self._ws = n, int(lib.spops_grad_norm_workspace_size())
        chunks, in_place = ctypes.c_int64(0), ctypes.c_int32(0)
        with torch.cuda.device(dev):
            # the table, then the calls' partial sums
            at = (size + 255) // 256 * 256
            table = torch.empty(at + self._ws, dtype=torch.uint8, device=dev)
            _check(lib.spops_grad_set_build(
                (ctypes.c_void_p * n)(*ins), (ctypes.c_void_p * n)(*outs), (ctypes.c_int64 * n)(*counts),
                (ctypes.c_int32 * n)(*dtypes), n, table.data_ptr(), size, ctypes.byref(chunks), ctypes.byref(in_place),
                _raw_stream(dev.index)), "grad_set_build")
            super().__init__(table)
        self._chunks, self._in_place = chunks.value, in_place.value
        self._partial_ptr = self._ptr + at
        # what autograd counts the writes of: views of one buffer share its count
        owners = [o if o.is_inference() or o._base is None else o._base for o in self.out]
        self._owners = list({id(o): o for o in owners}.values())

    def __len__(self):
        return self._n


def _set(grads) -> GradSet:
    return grads if isinstance(grads, GradSet) else GradSet(grads)


def grad_norm(grads) -> torch.Tensor:
    """The 2-norm of all gradients together: an fp32 scalar on the device. grads: a GradSet or
    a list of tensors."""
    s = _set(grads)
    dev = s.device
    if _elsewhere(dev.index):
        with torch.cuda.device(dev):
            return grad_norm(s)
    norm = torch.empty((), dtype=torch.float32, device=dev)
    stream = _raw_stream(dev.index)
    st = _L().spops_grad_norm(s._on_stream(stream), s._n, s._chunks, norm.data_ptr(), s._partial_ptr, s._ws, stream)
    if st:
        _check(st, "grad_norm")
    return norm


def clip_grads(grads, max_norm: float) -> torch.Tensor:
    """Scales every gradient by min(1, max_norm / (norm + 1e-6)), in place or into the set's
    outputs, and returns the norm before clipping (an fp32 scalar on the device). An infinite
    norm scales by 0 and a NaN one by NaN, as the formula says: check the returned norm where
    that matters. max_norm = inf clips nothing, whatever the norm. grads: a GradSet or a list of tensors."""
    s = _set(grads)
    dev = s.device
    if _elsewhere(dev.index):
        with torch.cuda.device(dev):
            return clip_grads(s, max_norm)
    norm = torch.empty((), dtype=torch.float32, device=dev)
    stream = _raw_stream(dev.index)
    st = _L().spops_clip_grads(s._on_stream(stream), s._n, s._chunks, s._in_place, float(max_norm), norm.data_ptr(),
                               s._partial_ptr, s._ws, stream)
    if st:
        _check(st, "clip_grads")
    increment_version(s._owners)  # (a backward pass that saved one of the outputs raises)
    return norm
