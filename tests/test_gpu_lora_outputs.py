"""lora_add and lora_grad into the caller's tensors, and what autograd learns of that."""
import pytest
import torch

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
T, K, N, R, ADAPTERS = 300, 64, 96, 8, 3


def operands(dtype=torch.bfloat16, tokens=T):
    torch.manual_seed(7)

    def randn(*shape):
        return torch.randn(*shape, device=DEV).mul_(0.3).to(dtype)

    ids = (torch.arange(tokens, device=DEV) % (ADAPTERS + 1) - 1).to(torch.int32)
    return dict(X=randn(tokens, K), A=randn(ADAPTERS, R, K), B=randn(ADAPTERS, N, R), W=randn(N, K), dY=randn(tokens, N),
                dX=randn(tokens, K), plan=sp.lora_plan(ids, ADAPTERS))


def test_out_of_a_graph_is_refused():
    d = operands()
    args = d["A"].requires_grad_(), d["B"].requires_grad_(), d["plan"]
    X = d["X"].requires_grad_()
    Y = X @ d["W"].t()
    before = Y.detach().clone()
    with pytest.raises(RuntimeError, match="out is part of an autograd graph"):
        sp.lora_add(X, *args, base=Y, out=Y)
    leaf = before.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="out is part"):
        sp.lora_add(X, *args, out=leaf)
    assert torch.equal(Y, before) and torch.equal(leaf, before)
    want = sp.lora_add(X, *args, base=before)  # (a result of its own is no part of a graph)
    assert not want.requires_grad
    with torch.no_grad():
        sp.lora_add(X, *args, base=Y, out=Y)
    assert torch.equal(Y, want)


def test_gradients_into_a_graph_are_refused():
    d = operands()
    args = d["dY"], d["X"], d["A"], d["B"], d["plan"]
    want = sp.lora_grad(*args)
    for i, name in enumerate(("dX_out", "dA_out", "dB_out")):
        leaf = torch.zeros_like(want[i]).requires_grad_()
        for out in (leaf, leaf * 1):
            with pytest.raises(RuntimeError, match=f"{name} is part"):
                sp.lora_grad(*args, **{name: out})
        assert not leaf.any()
        sp.lora_grad(*args, **{name: leaf}, need=tuple(j != i for j in range(3)))  # (not asked for: not written)
        assert not leaf.any()
        with torch.no_grad():
            sp.lora_grad(*args, **{name: leaf})
        assert torch.equal(leaf, want[i])


def test_a_saved_tensor_that_was_written_is_noticed():
    d = operands()
    w = torch.ones(N, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    Y = d["X"] @ d["W"].t()
    loss = (Y * w).sum()  # saves Y
    sp.lora_add(d["X"], d["A"], d["B"], d["plan"], base=Y, out=Y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    for name, like in (("dX_out", "X"), ("dA_out", "A"), ("dB_out", "B")):
        out = torch.ones_like(d[like])
        v = torch.ones_like(out).requires_grad_()
        loss = (out * v).sum()
        sp.lora_grad(d["dY"], d["X"], d["A"], d["B"], d["plan"], **{name: out})
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens", [5, 300, 700])
def test_outputs_given_hold_the_same_bits(dtype, tokens):
    d = operands(dtype, tokens)
    Y = sp.lora_add(d["X"], d["A"], d["B"], d["plan"], base=d["dY"])
    out = torch.full_like(Y, float("nan"))
    assert sp.lora_add(d["X"], d["A"], d["B"], d["plan"], base=d["dY"], out=out) is out and torch.equal(out, Y)
    args = d["dY"], d["X"], d["A"], d["B"], d["plan"]
    want = sp.lora_grad(*args, dX_base=d["dX"])
    outs = [torch.full_like(t, float("nan")) for t in want]
    got = sp.lora_grad(*args, dX_base=d["dX"], dX_out=outs[0], dA_out=outs[1], dB_out=outs[2])
    for w, o, g in zip(want, outs, got):
        assert g is o and torch.equal(o, w)
    # buffers of a set that is clipped
    flat = torch.full((outs[1].numel() + outs[2].numel(),), float("nan"), dtype=dtype, device=DEV)
    dA, dB = flat[:outs[1].numel()].view_as(outs[1]), flat[outs[1].numel():].view_as(outs[2])
    s = sp.GradSet([dA, dB])
    sp.lora_grad(*args, dA_out=dA, dB_out=dB, need=(False, True, True))
    assert torch.equal(dA, want[1]) and torch.equal(dB, want[2])
    sp.clip_grads(s, 1e-3)
    assert abs(float(torch.linalg.vector_norm(flat.float())) - 1e-3) < 1e-4


def test_inference_tensors_are_written():
    d = operands()
    want = sp.lora_add(d["X"], d["A"], d["B"], d["plan"])
    with torch.inference_mode():
        out = torch.empty_like(want)
        sp.lora_add(d["X"], d["A"], d["B"], d["plan"], out=out)
    assert torch.equal(out, want)
    sp.lora_add(d["X"], d["A"], d["B"], d["plan"], out=out)
    assert torch.equal(out, want)


def test_refusals_of_outputs():
    d = operands()
    args = d["dY"], d["X"], d["A"], d["B"], d["plan"]
    with pytest.raises(ValueError, match="dA_out must be"):
        sp.lora_grad(*args, dA_out=torch.empty(ADAPTERS, R, K + 8, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dtype"):
        sp.lora_grad(*args, dB_out=torch.empty(ADAPTERS, N, R, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        sp.lora_grad(*args, dB_out=torch.empty(ADAPTERS, R, N, device=DEV, dtype=torch.bfloat16).transpose(1, 2))
    with pytest.raises(ValueError, match="overlap"):
        sp.lora_grad(*args, dA_out=d["A"])
