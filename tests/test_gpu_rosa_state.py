"""What a RosaLinear keeps between calls and what autograd is told of it."""
import copy
import gc
import pickle
import weakref

import pytest
import torch

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def layer_of(k=48, out=72, rank=4, **kw):
    torch.manual_seed(3)
    layer = sp.RosaLinear(torch.randn(out, k, device=DEV, dtype=BF16).mul_(k ** -0.5), rank, **kw)
    layer.B.data.normal_(0, 0.1)
    return layer


def test_plan_of_a_captured_length_stays_while_other_lengths_pass():
    layer = layer_of()
    X = torch.randn(300, 48, device=DEV, dtype=BF16)
    with torch.no_grad():
        want = layer(X)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            Y = layer(X)
        plan = layer._plans[300]
        address, keeps = plan.buf.data_ptr(), weakref.ref(plan)
        del plan
        for tokens in range(1, 66):
            layer(X[:tokens])
        gc.collect()
        assert 300 not in layer._plans and keeps() is not None and keeps().buf.data_ptr() == address
        graph.replay()
        assert torch.equal(Y, want) and torch.equal(layer(X), want)


@pytest.mark.parametrize("own_dy", [True, False])
def test_gradients_with_a_graph_match_and_refuse_second_derivatives(own_dy):
    layer = layer_of()
    X = torch.randn(200, 48, device=DEV, dtype=BF16, requires_grad=True)
    dY = torch.randn(200, 72, device=DEV, dtype=BF16, requires_grad=own_dy)
    inputs = (X, layer.A, layer.B)
    want = torch.autograd.grad(layer(X), inputs, dY.detach())
    got = torch.autograd.grad(layer(X), inputs, dY, create_graph=True)
    for w, g in zip(want, got):
        assert torch.equal(w, g)
        with pytest.raises(RuntimeError, match="twice"):
            g.float().square().sum().backward(retain_graph=True)


def masked_layer(kind, seed, m=256, k=192, dtype=BF16):
    """A layer on a block mask: columns in blocks of 32, two or three of six per row of blocks."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for b in range(m // 64):
        blocks = torch.randperm(k // 32, generator=g)[:3].sort().values
        cols = (blocks[:, None] * 32 + torch.arange(32)).reshape(-1)
        rows += [cols] * 64
    ro = torch.arange(m + 1, dtype=torch.int32, device=DEV) * 96
    col = torch.cat(rows).to(torch.int16).to(DEV)
    values = torch.randn(col.numel(), generator=g).mul_(0.1).to(dtype).to(DEV)
    if kind == "sparse":
        return sp.SparseLinear(ro, col, values, k)
    W = torch.randn(m, k, generator=g).mul_(k ** -0.5).to(dtype).to(DEV)
    layer = sp.RosaLinear(W, 4, row_offsets=ro, col_idx=col, values=values)
    layer.A.data.copy_(torch.randn(1, 4, k, generator=g).mul_(k ** -0.5))
    layer.B.data.copy_(torch.randn(1, m, 4, generator=g).mul_(0.1))
    return layer


def both_passes(layer):
    g = torch.Generator().manual_seed(9)
    shape = (192, 160) if isinstance(layer, sp.SparseLinear) else (160, 192)
    X = torch.randn(shape, generator=g).to(BF16).to(DEV).requires_grad_()
    Y = layer(X)
    dY = torch.randn(Y.shape, generator=g).to(BF16).to(DEV)
    return (Y.detach(), *torch.autograd.grad(Y, [X, *layer.parameters()], dY))


@pytest.mark.parametrize("kind", ["sparse", "rosa"])
def test_another_mask_of_the_same_size_is_loaded(kind):
    layer, other = masked_layer(kind, 1), masked_layer(kind, 2)
    first, want = both_passes(layer), both_passes(other)
    assert not torch.equal(layer.col_idx, other.col_idx)
    graph = torch.cuda.CUDAGraph()
    X = torch.randn((192, 160) if kind == "sparse" else (160, 192), device=DEV, dtype=BF16)
    with torch.no_grad():
        layer(X)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            Y = layer(X)
    layer.load_state_dict({k: v.clone() for k, v in other.state_dict().items()})
    for a, b in zip(both_passes(layer), want):
        assert torch.equal(a, b)
    with torch.no_grad():
        graph.replay()  # (what it reads was written where it reads it)
        assert torch.equal(Y, other(X))
    back = masked_layer(kind, 1)
    layer.load_state_dict(back.state_dict(), assign=True)
    for a, b in zip(both_passes(layer), first):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["sparse", "rosa"])
def test_copies_and_moves_give_the_same_bits(kind):
    layer = masked_layer(kind, 3)
    want = both_passes(layer)
    for twin in (copy.deepcopy(layer), pickle.loads(pickle.dumps(layer)), copy.deepcopy(layer).cpu().to(DEV)):
        for a, b in zip(both_passes(twin), want):
            assert torch.equal(a, b)
    layer.cpu().to(DEV)
    for a, b in zip(both_passes(layer), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["sparse", "rosa", "low rank"])
def test_an_empty_batch_trains(kind):
    layer = layer_of() if kind == "low rank" else masked_layer(kind, 1)
    k = 48 if kind == "low rank" else 192
    X = torch.empty((k, 0) if kind == "sparse" else (0, k), device=DEV, dtype=BF16, requires_grad=True)
    layer(X).sum().backward()
    assert X.grad.shape == X.shape
    for p in layer.parameters():
        assert p.grad.shape == p.shape and not p.grad.any()
