"""RosaLinear's own bookkeeping, with stand-ins for the calls that need a GPU."""
import copy
import gc
import pickle
import weakref

import pytest
import torch

import unstructured_sparse_linear_gb300 as sp
from unstructured_sparse_linear_gb300 import layer as layer_module


class FakePlan:
    def __init__(self, tokens, device):
        self.tokens, self.device = tokens, device


@pytest.fixture
def fake(monkeypatch):
    """A layer whose plans are counted and whose forward pass returns the plan that it was given."""
    state = {"capturing": False, "made": [], "used": None}

    def lora_plan(ids, n, tokens=None, device=None):
        state["made"].append(tokens)
        return FakePlan(tokens, device)

    def apply(X, values, A, B, layer, plan):
        state["used"] = plan
        return X.new_zeros(X.shape[0], layer.out_features)

    monkeypatch.setattr(layer_module, "lora_plan", lora_plan)
    monkeypatch.setattr(layer_module.RosaLinearFunction, "apply", apply)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    state["layer"] = sp.RosaLinear(torch.zeros(6, 4), 2)
    return state


def use(fake, tokens, capturing=False):
    fake["capturing"] = capturing
    fake["layer"](torch.zeros(tokens, 4))
    fake["capturing"] = False
    plan, fake["used"] = fake["used"], None
    return plan


def test_a_plan_that_a_graph_captured_outlives_the_cache(fake):
    """Warm-up, capture of the same length, then more other lengths than the cache holds: the graph's
    replays still read the captured plan, which nothing but the layer owns."""
    use(fake, 5)
    captured = weakref.ref(use(fake, 5, capturing=True))
    passing = weakref.ref(use(fake, 6))
    for tokens in range(100, 230):
        use(fake, tokens)
    gc.collect()
    assert passing() is None  # (the cache did drop plans)
    assert captured() is not None
    assert use(fake, 5) is captured() and fake["made"].count(5) == 1  # and it serves the length again
    use(fake, 200)
    again = weakref.ref(use(fake, 200, capturing=True))  # a second graph, beside the first
    for tokens in range(300, 430):
        use(fake, tokens)
    gc.collect()
    assert captured() is not None and again() is not None


def test_a_plan_made_in_a_capture_is_not_kept(fake):
    use(fake, 5, capturing=True)
    assert fake["layer"]._plans == {}
    use(fake, 5)
    assert fake["made"] == [5, 5]


@pytest.fixture
def plain(monkeypatch):
    """The two low-rank calls as the kernels do them: on the values, outside autograd."""
    def lora_add(X, A, B, plan, base=None, scale=1.0, out=None, return_h=False):
        h = X.detach() @ A.detach()[0].t()
        out.data.add_(scale * (h @ B.detach()[0].t()))
        return out, h

    def lora_grad(dY, X, A, B, plan, scale=1.0, h=None, dX_base=None, dX_out=None, need=(True,) * 3, **kw):
        dY, X, A, B, h = (t.detach() for t in (dY, X, A, B, h))
        dP = scale * (dY @ B[0])
        if need[0]:
            dX_out.data.add_(dP @ A[0])
        return dX_out if need[0] else None, (dP.t() @ X)[None], scale * (dY.t() @ h)[None]

    monkeypatch.setattr(layer_module, "lora_add", lora_add)
    monkeypatch.setattr(layer_module, "lora_grad", lora_grad)
    layer = sp.RosaLinear(torch.randn(6, 4, dtype=torch.float64), 2, scale=0.5)
    layer.B.data.normal_()
    return layer


@pytest.mark.parametrize("own_dy", [True, False])
def test_second_derivatives_are_refused(plain, own_dy):
    X = torch.randn(5, 4, dtype=torch.float64, requires_grad=True)
    dY = torch.randn(5, 6, dtype=torch.float64, requires_grad=own_dy)
    Y = plain(X, plan=object())
    dX, dA, dB = torch.autograd.grad(Y, (X, plain.A, plain.B), dY, create_graph=True)
    assert torch.allclose(dX, dY @ (plain.weight + 0.5 * plain.B[0] @ plain.A[0]))
    assert torch.allclose(dB[0], 0.5 * dY.t() @ X @ plain.A[0].t())
    for first in (dX, dA, dB):
        with pytest.raises(RuntimeError, match="twice"):
            (Y.sum() + first.square().sum()).backward(retain_graph=True)
        for one in (dY, X, plain.A, plain.B) if own_dy else (X, plain.A, plain.B):
            with pytest.raises(RuntimeError, match="twice"):
                torch.autograd.grad(first.sum(), one, retain_graph=True)


def test_sparse_linear_refuses_second_derivatives(monkeypatch):
    """As the kernels' results carry no graph, a penalty on a gradient would be left out of a loss in silence."""
    W = torch.randn(6, 4, dtype=torch.float64)
    monkeypatch.setattr(layer_module, "spmm", lambda v, ro, ri, ci, X, m, plan=None: v.detach().reshape(ci) @ X.detach())
    monkeypatch.setattr(layer_module, "sddmm", lambda ro, ri, ci, dY, X, plan=None: (dY @ X.t()).detach().reshape(-1))
    monkeypatch.setattr(layer_module, "permute_values", lambda v, t: v.detach().reshape(6, 4).t().contiguous())

    class Layer:
        row_offsets = row_idx = row_idx_t = plan = plan_t = None
        col_idx, out_features, in_features = (6, 4), 6, 4
        _follow_mask = _check_mask = staticmethod(lambda *mask: None)

        class transpose:
            row_offsets, col_idx = None, (4, 6)

    values = W.reshape(-1).clone().requires_grad_()
    X = torch.randn(4, 5, dtype=torch.float64, requires_grad=True)
    Y = layer_module.SparseLinearFunction.apply(values, X, Layer)
    dX, dV = torch.autograd.grad(Y.sum(), (X, values), create_graph=True)
    assert torch.allclose(dX, W.t() @ torch.ones(6, 5, dtype=torch.float64))
    for first in (dX, dV):
        with pytest.raises(RuntimeError, match="twice"):
            (Y.sum() + first.square().sum()).backward(retain_graph=True)


def test_backward_uses_what_the_output_was_computed_with(plain):
    X = torch.randn(5, 4, dtype=torch.float64)
    dY = torch.randn(5, 6, dtype=torch.float64)
    Y = plain(X, plan=object())
    plain.scale = 3.0
    (dB,) = torch.autograd.grad(Y, plain.B, dY)
    assert torch.allclose(dB[0], 0.5 * dY.t() @ X @ plain.A.detach()[0].t())
    plain.scale = torch.tensor([0.25], dtype=torch.float64)
    Y = plain(X, plan=object())
    plain.scale.fill_(2.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(Y, plain.B, dY)
    Y = plain(X.requires_grad_(), plan=object())
    W = plain.weight
    plain.weight = torch.zeros_like(W)
    want = dY @ (W + 2.0 * plain.B.detach()[0] @ plain.A.detach()[0])
    assert torch.allclose(torch.autograd.grad(Y, X, dY)[0], want)
    Y = plain(X, plan=object())
    plain.weight.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(Y, X, dY)


class Rows:
    """What is derived of a mask, as tensors that tell it from another one's."""
    def __init__(self, row_offsets, col_idx):
        self.buf = torch.cat([row_offsets.long(), col_idx.long()])

    def of(self, layer):
        return torch.equal(self.buf, torch.cat([layer.row_offsets.long(), layer.col_idx.long()]))


class Turned:
    def __init__(self, row_offsets, col_idx):
        self.row_offsets, self.col_idx, self.perm = row_offsets + 100, col_idx + 100, col_idx + 200


@pytest.fixture
def masks(monkeypatch, plain):
    used = {"spmm": [], "sddmm": [], "csr_add": []}

    def note(name, result):
        def call(*a, plan=None, **kw):
            used[name].append((a, plan))
            return result(*a)
        return call

    monkeypatch.setattr(layer_module, "sort_rows", lambda ro, nnz=None, index_dtype=None: (ro[:-1] * 7).clone())
    monkeypatch.setattr(layer_module, "plan_build", lambda ro, row_idx, col, n: Rows(ro, col))
    monkeypatch.setattr(layer_module, "csr_transpose", lambda v, ro, col, n: Turned(ro, col))
    monkeypatch.setattr(layer_module, "permute_values", lambda v, t: v)
    monkeypatch.setattr(layer_module, "csr_add", note("csr_add", lambda v, ro, ri, ci, W: W.clone()))
    monkeypatch.setattr(layer_module, "spmm", note("spmm", lambda v, ro, ri, ci, X, m: X.new_zeros(m, X.shape[1])))
    monkeypatch.setattr(layer_module, "sddmm", note("sddmm", lambda ro, ri, ci, a, b: a.new_zeros(ci.numel())))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: used.get("capturing", False))
    return used


MASK_A = torch.tensor([0, 1, 2, 2, 3, 3, 4], dtype=torch.int32), torch.tensor([0, 3, 1, 2], dtype=torch.int16)
MASK_B = torch.tensor([0, 0, 0, 3, 3, 4, 4], dtype=torch.int32), torch.tensor([0, 1, 2, 3], dtype=torch.int16)


def masked(kind, mask):
    ro, col = (t.clone() for t in mask)
    values = torch.zeros(4, dtype=torch.float64)
    if kind == "sparse":
        return sp.SparseLinear(ro, col, values, 4)
    return sp.RosaLinear(torch.zeros(6, 4, dtype=torch.float64), 2, row_offsets=ro, col_idx=col, values=values)


def step(layer):
    kind = isinstance(layer, sp.SparseLinear)
    X = torch.zeros(*((4, 5) if kind else (5, 4)), dtype=torch.float64, requires_grad=True)
    return layer(X) if kind else layer(X, plan=object())


@pytest.mark.parametrize("kind", ["sparse", "rosa"])
def test_what_is_derived_of_the_mask_follows_it(masks, kind):
    layer = masked(kind, MASK_A)
    step(layer).sum().backward()
    plan, row_idx = layer.plan, layer.row_idx
    assert plan.of(layer) and masks["sddmm"][-1][1] is plan
    layer.load_state_dict(masked(kind, MASK_B).state_dict())
    assert torch.equal(layer.col_idx, MASK_B[1])
    step(layer).sum().backward()
    a, used = masks["sddmm"][-1]
    assert used.of(layer) and torch.equal(a[1], MASK_B[0][:-1] * 7)
    assert used is plan and a[1] is row_idx  # (written where captured graphs read them)
    if kind == "rosa":
        assert torch.equal(masks["csr_add"][-1][0][2], MASK_B[0][:-1] * 7)
    else:
        assert torch.equal(layer.transpose.perm, MASK_B[1] + 200) and layer.plan_t.buf[0] == 100
        assert masks["spmm"][-2][1].of(layer)
    # buffers that another layer shares, replaced ones, and moved ones
    layer.col_idx.copy_(MASK_A[1])
    layer.row_offsets.copy_(MASK_A[0])
    step(layer)
    assert layer.plan.of(layer)
    other = masked(kind, MASK_B)
    layer.load_state_dict({k: v.clone() for k, v in other.state_dict().items()}, assign=True)
    step(layer)
    assert layer.plan.of(layer)


@pytest.mark.parametrize("kind", ["sparse", "rosa"])
def test_a_mask_that_changes_between_the_passes_or_in_a_capture(masks, kind):
    layer = masked(kind, MASK_A)
    Y = step(layer)
    layer.col_idx.copy_(MASK_B[1])
    layer.row_offsets.copy_(MASK_B[0])
    with pytest.raises(RuntimeError, match="mask of this layer has changed"):
        Y.sum().backward()
    step(layer).sum().backward()
    layer.row_offsets.copy_(MASK_A[0])
    masks["capturing"] = True
    with pytest.raises(RuntimeError, match="before it is captured"):
        step(layer)
    masks["capturing"] = False
    step(layer)
    masks["capturing"] = True
    step(layer)


@pytest.mark.parametrize("kind", ["sparse", "rosa"])
def test_copies_derive_their_own(masks, kind):
    layer = masked(kind, MASK_A)
    for twin in (copy.deepcopy(layer), pickle.loads(pickle.dumps(layer))):
        step(twin)
        assert twin.plan is not layer.plan and twin.plan.of(twin)
        assert layer.plan.of(layer)


def test_plans_of_a_length_belong_to_a_device(fake, monkeypatch):
    """A layer that moved makes plans where it is; captured ones of both places stay."""
    layer = fake["layer"]
    here, there = torch.device("cuda", 0), torch.device("cuda", 1)

    def on(device, capturing=False):
        fake["capturing"] = capturing
        plan = layer._one_adapter_plan(5, device)
        fake["capturing"] = False
        return plan

    first = on(here)
    assert on(here, capturing=True) is first
    second = on(there)
    assert (first.device, second.device) == (here, there)
    assert on(there, capturing=True) is second
    layer._plans.clear()
    assert on(here) is first and on(there) is second


def test_factors_per_adapter_are_state():
    W, factors = torch.randn(6, 4), torch.tensor([0.5, 1.7, 0.3])
    layer = sp.RosaLinear(W.clone(), 2, n_adapters=3, scale=factors.clone())
    assert torch.equal(layer.scale, factors)
    other = sp.RosaLinear(W.clone(), 2, n_adapters=3, scale=torch.ones(3))
    other.load_state_dict(layer.state_dict())
    assert torch.equal(other.scale, factors) and torch.equal(other.A, layer.A)
    for narrow in (torch.float16, torch.bfloat16):  # the factors stay in 32 bits, to the last of them
        twin = copy.deepcopy(layer).to(narrow)
        assert twin.A.dtype == narrow and twin.scale.dtype == torch.float32 and torch.equal(twin.scale, factors)
    assert copy.deepcopy(layer).to("meta").scale.device.type == "meta"
    twin = pickle.loads(pickle.dumps(layer))
    assert torch.equal(twin.scale, factors)
    with pytest.raises(RuntimeError, match="size mismatch"):
        sp.RosaLinear(W.clone(), 2, n_adapters=2, scale=torch.ones(2)).load_state_dict(layer.state_dict())


def test_a_factor_may_be_a_number_or_a_tensor_at_any_time():
    layer = sp.RosaLinear(torch.randn(6, 4), 2, n_adapters=3, scale=2.0)
    assert layer.scale == 2.0 and set(layer.state_dict()) == {"weight", "A", "B"}
    layer.scale = torch.ones(3)
    assert "factors" in layer.state_dict() and torch.equal(layer.scale, torch.ones(3))
    layer.scale = 0.5
    assert layer.scale == 0.5 and set(layer.state_dict()) == {"weight", "A", "B"}
    layer.scale = torch.ones(3)
    assert layer.to("meta").to_empty(device="cpu").scale.shape == (3,)


def test_an_empty_batch_takes_any_strides(plain):
    """Autograd's gradient of a sum is a broadcast number, which without a token counts as contiguous."""
    from unstructured_sparse_linear_gb300.lora import _rows
    cpu = torch.device("cpu")
    for t in (torch.ones(()).expand(0, 96), torch.ones(96).expand(0, 96), torch.empty(96, 0).t()):
        assert t.is_contiguous()
        _rows(t, "dY", 0, 96, torch.float32, cpu)
    with pytest.raises(ValueError, match="contiguous rows"):
        _rows(torch.ones(96).expand(2, 96), "dY", 2, 96, torch.float32, cpu)


def test_factors_that_require_a_gradient_are_refused():
    """They would get none."""
    W = torch.randn(6, 4)
    for factors in (torch.ones(3, requires_grad=True), torch.nn.Parameter(torch.ones(3))):
        with pytest.raises(ValueError, match="not trained"):
            sp.RosaLinear(W, 2, n_adapters=3, scale=factors)
    layer = sp.RosaLinear(W, 2, n_adapters=3, scale=torch.ones(3))
    with pytest.raises(ValueError, match="not trained"):
        layer.scale = torch.ones(3, requires_grad=True)
    layer.requires_grad_(True)  # (parameters only)
    assert not layer.scale.requires_grad and torch.equal(layer.scale, torch.ones(3))
