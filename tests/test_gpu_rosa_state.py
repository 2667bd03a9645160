"""What a RosaLinear keeps between calls and what autograd is told of it."""
import gc
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
