"""A sparse linear layer on a fixed CSR mask, forward and backward on this package's kernels.

HazyResearch/fly issue "Pure torch implementaton of pixelfly": a pixelfly layer is a
linear layer whose weight keeps only a butterfly pattern of dense blocks; the issue times
its forward and backward against nn.Linear. spops README ("Sparse Operations (spops)"):
SpMM is the forward product, SDDMM the weight gradient on the mask, and csr_transpose
gives the input gradient (torchsparsegradutils README, "Basic Sparse Matrix
Multiplication": both gradients of a sparse product keep the sparsity).

Activations are feature-major (features x tokens), the layout in which every product is
one call with no transposed copies:
    forward   Y^T  = W X^T                 spmm
    dW        dW   = (dY^T X) on the mask  sddmm(A = dY^T, BT = X^T)
    dX        dX^T = W^T dY^T              spmm of the cached transpose of W
The row permutation, the mask plan and the transpose's structure are built once per mask.
"""
from __future__ import annotations

import functools

import torch

from . import csr_add, csr_transpose, permute_values, plan_build, sddmm, sort_rows, spmm
from .lora import lora_add, lora_grad, lora_plan


class _Refuse(torch.autograd.Function):
    """The first `count` of its tensors, as results of all of them that cannot be differentiated."""

    @staticmethod
    def forward(ctx, count, *tensors):
        return tensors[:count]

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the gradients of this layer cannot be differentiated again: its kernels compute first "
                           "derivatives only, so they cannot be taken twice")


def first_derivatives_only(backward):
    """A backward pass on the kernels, whose results carry no graph. Under create_graph=True the gradients
    come back tied to the output's gradient and to what the forward pass saved, so that a second derivative raises
    instead of missing them. (torch's once_differentiable ties them to the output's gradient alone.)"""

    @functools.wraps(backward)
    def wrapped(ctx, dY):
        with torch.no_grad():
            grads = backward(ctx, dY)
        return _Refuse.apply(len(grads), *grads, dY, *ctx.saved_tensors) if torch.is_grad_enabled() else grads

    return wrapped


def _tensors(x):
    """The tensors of one that a layer derives from its mask: a tensor, a Plan or a Transpose."""
    if isinstance(x, torch.Tensor):
        return [x]
    return [x.buf] if hasattr(x, "buf") else [x.row_offsets, x.col_idx, x.perm]


class _MaskedLayer(torch.nn.Module):
    """A layer on a CSR mask, its buffers row_offsets and col_idx. What the kernels need of the mask beside it
    is derived from them (``_derive``, a dict of attributes), and derived again once the buffers hold another mask or
    have moved, as after load_state_dict or to: a plan leads the kernels to rows and columns, so one of another
    mask would lead them out of range."""

    _mask = None  # (row_offsets, its version, col_idx, its version) that the derived ones are of

    def _derive(self) -> dict:
        raise NotImplementedError

    def _follow_mask(self):
        """Brings the derived ones up to date; returns what tells this mask from others."""
        now = []
        for t in (self.row_offsets, self.col_idx):
            now += [t, None if t.is_inference() else t._version]
        then = self._mask
        if then is not None and now[0] is then[0] and now[1] == then[1] and now[2] is then[2] and now[3] == then[3]:
            return then
        if then is not None and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the mask of this layer has changed: call the layer once before it is captured in a graph")
        for name, new in self._derive().items():
            old = self.__dict__.get(name)
            if old is not None and all(o.device == n.device and o.shape == n.shape
                                       for o, n in zip(_tensors(old), _tensors(new))):
                for o, n in zip(_tensors(old), _tensors(new)):  # (graphs that were captured read them where they are)
                    o.copy_(n)
            else:
                setattr(self, name, new)
        self._mask = tuple(now)
        return self._mask

    def _check_mask(self, then):
        """For a backward pass, with what _follow_mask returned in the forward one."""
        if then is not None and self._follow_mask() is not then:
            raise RuntimeError("the mask of this layer has changed since the forward pass")

    def __getstate__(self):  # copies and pickles derive their own
        made = set(self._derived_names) | {"_mask"}
        return {k: v for k, v in super().__getstate__().items() if k not in made}

    def __setstate__(self, state):
        super().__setstate__(state)
        if "row_offsets" in self._buffers and self.row_offsets.is_cuda:
            self._follow_mask()


class SparseLinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, values, Xt, layer):
        ctx.mask = layer._follow_mask()
        Yt = spmm(values, layer.row_offsets, layer.row_idx, layer.col_idx, Xt, layer.out_features, plan=layer.plan)
        ctx.save_for_backward(values, Xt)
        ctx.layer = layer
        return Yt

    @staticmethod
    @first_derivatives_only
    def backward(ctx, dYt):
        values, Xt = ctx.saved_tensors
        L = ctx.layer
        L._check_mask(ctx.mask)
        dYt = dYt.contiguous()
        d_values = d_Xt = None
        if ctx.needs_input_grad[0]:
            d_values = sddmm(L.row_offsets, L.row_idx, L.col_idx, dYt, Xt, plan=L.plan)
        if ctx.needs_input_grad[1]:
            vt = permute_values(values, L.transpose)
            d_Xt = spmm(vt, L.transpose.row_offsets, L.row_idx_t, L.transpose.col_idx, dYt, L.in_features,
                        plan=L.plan_t)
        return d_values, d_Xt, None


class SparseLinear(_MaskedLayer):
    """Y^T = W X^T with W (out_features x in_features) stored as the values of a fixed CSR
    mask (row_offsets int32, col_idx int16/int32); inputs and outputs are feature-major
    (features x tokens), fp16 or bf16 (fp32 runs the general kernels). Gradients are first
    derivatives: differentiating them again raises."""

    def __init__(self, row_offsets: torch.Tensor, col_idx: torch.Tensor, values: torch.Tensor, in_features: int):
        super().__init__()
        self.out_features = row_offsets.numel() - 1
        self.in_features = int(in_features)
        self.register_buffer("row_offsets", row_offsets)
        self.register_buffer("col_idx", col_idx)
        self.values = torch.nn.Parameter(values)
        self._follow_mask()

    _derived_names = ("row_idx", "plan", "transpose", "row_idx_t", "plan_t")

    def _derive(self):
        ro, col = self.row_offsets, self.col_idx
        row_idx = sort_rows(ro, nnz=col.numel(), index_dtype=col.dtype)
        t = csr_transpose(None, ro, col, self.in_features)
        row_idx_t = sort_rows(t.row_offsets, nnz=col.numel(), index_dtype=col.dtype)
        return dict(row_idx=row_idx, plan=plan_build(ro, row_idx, col, self.in_features), transpose=t,
                    row_idx_t=row_idx_t, plan_t=plan_build(t.row_offsets, row_idx_t, t.col_idx, self.out_features))

    def forward(self, Xt: torch.Tensor) -> torch.Tensor:
        return SparseLinearFunction.apply(self.values, Xt.contiguous(), self)


class RosaLinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, values, A, B, layer, plan):
        weight, scale = layer.weight, layer.scale
        Y = X @ layer.merged(values).t()
        ctx.mask = layer._mask if values is not None else None
        Y, h = lora_add(X, A, B, plan, base=Y, scale=scale, out=Y, return_h=True)
        factors = scale if isinstance(scale, torch.Tensor) else None
        ctx.save_for_backward(X, values, A, B, h, weight, factors)
        ctx.layer, ctx.plan, ctx.scale = layer, plan, scale if factors is None else None
        return Y

    @staticmethod
    @first_derivatives_only
    def backward(ctx, dY):
        X, values, A, B, h, weight, factors = ctx.saved_tensors
        L, scale = ctx.layer, ctx.scale if factors is None else factors
        L._check_mask(ctx.mask)
        dY = dY.contiguous()
        need_x, need_v, need_a, need_b = ctx.needs_input_grad[:4]
        # The merged weight is formed again: less time than its memory is worth in a deep model.
        base = dY @ L.merged(values, weight) if need_x else None
        dX, dA, dB = lora_grad(dY, X, A, B, ctx.plan, scale=scale, h=h, dX_base=base, dX_out=base,
                               need=(need_x, need_a, need_b))
        dV = None
        if need_v and values is not None:
            dV = sddmm(L.row_offsets, L.row_idx, L.col_idx, dY.t().contiguous(), X.t().contiguous(), plan=L.plan)
        return dX, dV, dA, dB, None, None


class RosaLinear(_MaskedLayer):
    """A frozen projection with a RoSA adapter, a sparse and a low-rank update (spops README,
    "Sparse Operations (spops)": RoSA's sparse part is added to the weight with csr_add, and its
    gradient is an SDDMM on the mask):

        Y = X (W + S)^T + s_i (X A_i^T) B_i^T

    weight: W [out, in], fp16 or bf16 (fp32 runs the general kernels), not trained. row_offsets,
    col_idx, values: S on a fixed CSR mask, shared by all tokens (None: no sparse part). n_adapters
    low-rank adapters of one rank, their factor `scale` a number or an fp32 tensor with one per
    adapter (then part of the layer's state); A starts at random and B at zero, so that the adapters start as no change. X is
    token-major [..., in]; adapter_ids (int32, one per token) or a plan of them choose each token's
    adapter, by default adapter 0 for all. Gradients are first derivatives: differentiating them again
    raises."""

    def __init__(self, weight: torch.Tensor, rank: int, n_adapters: int = 1, scale=1.0, row_offsets=None, col_idx=None,
                 values=None):
        super().__init__()
        self.out_features, self.in_features = weight.shape
        self.n_adapters = int(n_adapters)
        self.register_buffer("factors", None)
        RosaLinear.scale.fset(self, scale)  # (a Parameter would be registered under that name)
        self.register_buffer("weight", weight)
        dev, dt = weight.device, weight.dtype
        self.A = torch.nn.Parameter(torch.randn(self.n_adapters, rank, self.in_features, device=dev, dtype=torch.float32)
                                    .mul_(self.in_features ** -0.5).to(dt))
        self.B = torch.nn.Parameter(torch.zeros(self.n_adapters, self.out_features, rank, device=dev, dtype=dt))
        if values is None:
            self.values = None
        else:
            self.register_buffer("row_offsets", row_offsets)
            self.register_buffer("col_idx", col_idx)
            self.values = torch.nn.Parameter(values)
            self._follow_mask()
        self._plans = {}  # by number of tokens: every token uses adapter 0
        self._captured = {}  # those of them that a graph's replays read, kept as long as the layer

    @property
    def scale(self):
        """The adapters' factors: a number, or the fp32 tensor of one per adapter, which is part of the state
        (``factors``) and moves with the layer."""
        return self._factor if self.factors is None else self.factors

    @scale.setter
    def scale(self, value):
        tensor = isinstance(value, torch.Tensor)
        if tensor and value.requires_grad:
            raise ValueError("scale requires a gradient, but the factors are not trained: they would get none")
        self.factors, self._factor = (value, None) if tensor else (None, value)

    def _apply(self, *args, **kwargs):
        factors = self.factors
        super()._apply(*args, **kwargs)
        if factors is not None and self.factors.dtype != factors.dtype:  # 32 bits, whatever type the layer is brought to
            self.factors = factors.to(self.factors.device)
        return self

    _derived_names = ("row_idx", "plan")

    def _derive(self):
        row_idx = sort_rows(self.row_offsets, nnz=self.col_idx.numel(), index_dtype=self.col_idx.dtype)
        return dict(row_idx=row_idx, plan=plan_build(self.row_offsets, row_idx, self.col_idx, self.in_features))

    def __getstate__(self):  # a copy or a pickle of the layer makes its own plans
        return {**super().__getstate__(), "_plans": {}, "_captured": {}}

    def merged(self, values, weight=None):
        """W + S (of another weight than the layer's, where one is given)."""
        weight = self.weight if weight is None else weight
        if values is None:
            return weight
        self._follow_mask()
        return csr_add(values, self.row_offsets, self.row_idx, self.col_idx, weight)

    def _one_adapter_plan(self, tokens, device):
        capturing = torch.cuda.is_current_stream_capturing()
        plan = self._captured.get((tokens, device)) or self._plans.get(tokens)
        if plan is None or plan.device != device:  # (the layer may have moved)
            plan = lora_plan(None, self.n_adapters, tokens=tokens, device=device)
            if capturing:  # (written by the graph's replays: not for calls outside it)
                return plan
            if len(self._plans) >= 64:  # (lengths that come and go)
                self._plans.clear()
            self._plans[tokens] = plan
        if capturing:  # the graph holds the plan's address and nothing else holds the plan
            self._captured[tokens, device] = plan
        return plan

    def forward(self, X: torch.Tensor, adapter_ids: torch.Tensor | None = None, plan=None) -> torch.Tensor:
        X2 = X.reshape(-1, self.in_features)
        if plan is None and adapter_ids is not None:
            plan = lora_plan(adapter_ids.reshape(-1), self.n_adapters)
        if plan is None:
            plan = self._one_adapter_plan(X2.shape[0], X2.device)
        Y = RosaLinearFunction.apply(X2.contiguous(), self.values, self.A, self.B, self, plan)
        return Y.reshape(*X.shape[:-1], self.out_features)
