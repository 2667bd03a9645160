"""RosaLinear (sparse + low-rank adapter beside a frozen projection) against a dense 64-bit model,
and the example that trains and serves it.

Tolerance: the merged weight, the projection and the two products each round to the storage type
once or twice; relative Frobenius errors stay within three of its half-ulps per stage: 2^-8 * 6 for
bf16, 2^-11 * 6 for fp16, and 1e-5 in fp32."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import workloads as wl
from helpers import as_f64, rel_fro

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
REL = {torch.float32: 1e-5, torch.float16: 6 * 2.0 ** -11, torch.bfloat16: 6 * 2.0 ** -8}


@pytest.mark.parametrize("dtype", list(REL))
@pytest.mark.parametrize("n,sparse", [(1, True), (3, True), (2, False)])
def test_forward_and_gradients_against_dense(dtype, n, sparse):
    torch.manual_seed(n)
    k, out, r, T = 264, 392, 8, 300
    W = torch.randn(out, k, device=DEV).mul_(k ** -0.5).to(dtype)
    kw = {}
    if sparse:
        ro, col = wl.uniform_mask(5, out, k, 0.05)
        kw = dict(row_offsets=torch.from_numpy(ro).to(DEV), col_idx=torch.from_numpy(col).to(torch.int16).to(DEV),
                  values=torch.randn(col.size, device=DEV).mul_(0.1).to(dtype))
    scale = torch.rand(n, device=DEV) + 0.5
    layer = sp.RosaLinear(W, r, n_adapters=n, scale=scale, **kw)
    layer.B.data.normal_(0, 0.1)
    X = torch.randn(3, T // 3, k, device=DEV).to(dtype).requires_grad_()
    ids = torch.randint(-1, n, (3, T // 3), dtype=torch.int32, device=DEV) if n > 1 else None
    Y = layer(X, adapter_ids=ids)
    G = torch.randn(T, out, device=DEV).to(dtype).reshape(Y.shape)
    Y.backward(G)

    d = {x: torch.from_numpy(as_f64(t)).requires_grad_() for x, t in (("X", X), ("A", layer.A), ("B", layer.B))}
    Wd, vals = torch.from_numpy(as_f64(W)), None
    if sparse:
        vals = torch.from_numpy(as_f64(layer.values)).requires_grad_()
        rows = np.repeat(np.arange(out), np.diff(ro))
        Wd = Wd.index_put((torch.from_numpy(rows), torch.from_numpy(col.astype(np.int64))), vals, accumulate=True)
    flat, which = d["X"].reshape(-1, k), (ids.reshape(-1).cpu() if ids is not None else torch.zeros(T, dtype=torch.int32))
    want = flat @ Wd.t()
    for a in range(n):
        own = (which == a).double()[:, None]
        want = want + own * float(scale[a]) * (flat @ d["A"][a].t() @ d["B"][a].t())
    want.backward(torch.from_numpy(as_f64(G)).reshape(T, out))

    def close(got, ref, what):
        e = rel_fro(as_f64(got).reshape(ref.shape), ref.detach().numpy())
        assert e <= REL[dtype], (what, e)

    close(Y, want, "Y")
    close(X.grad, d["X"].grad.reshape(X.shape), "dX")
    close(layer.A.grad, d["A"].grad, "dA")
    close(layer.B.grad, d["B"].grad, "dB")
    if sparse:
        close(layer.values.grad, vals.grad, "dvalues")


def test_only_the_gradients_that_are_asked_for():
    W = torch.randn(64, 48, device=DEV, dtype=torch.bfloat16)
    layer = sp.RosaLinear(W, 4)
    layer.A.requires_grad_(False)
    X = torch.randn(70, 48, device=DEV, dtype=torch.bfloat16)
    layer(X).sum().backward()  # the sum's gradient is one broadcast number
    assert layer.A.grad is None and layer.B.grad is not None and layer.weight.grad is None
    want = as_f64(X) @ as_f64(layer.A)[0].T
    assert rel_fro(as_f64(layer.B.grad)[0], np.tile(want.sum(0), (64, 1))) <= REL[torch.bfloat16]


def test_first_call_of_a_length_in_a_graph_capture():
    """The plan of a length that is first seen in a capture belongs to the graph: calls outside make their own."""
    torch.manual_seed(2)
    W = torch.randn(72, 48, device=DEV, dtype=torch.bfloat16).mul_(48 ** -0.5)
    layer = sp.RosaLinear(W, 4)
    layer.B.data.normal_(0, 0.1)
    X = torch.randn(300, 48, device=DEV, dtype=torch.bfloat16)
    with torch.no_grad():
        layer(X[:7])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            Y = layer(X)
        assert list(layer._plans) == [7]
        own = layer(X)
        graph.replay()
        assert list(layer._plans) == [7, 300] and torch.equal(Y, own)
    want = as_f64(X) @ (as_f64(W) + as_f64(layer.B)[0] @ as_f64(layer.A)[0]).T
    assert rel_fro(as_f64(own), want) <= REL[torch.bfloat16]


def test_example_trains_and_serves():
    spec = importlib.util.spec_from_file_location("rosa_example", os.path.join(ROOT, "examples",
                                                                              "rosa_finetune_and_serve.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, norms = ex.train(steps=12)
    assert losses[-1] < 0.9 * losses[0] and all(np.isfinite(losses)) and all(x > 0 for x in norms)
    got = ex.serve()
    W, A, B = (as_f64(got[x]) for x in ("W", "A", "B"))
    for s in got["steps"]:
        X, ids = as_f64(s["X"]), s["ids"].cpu().numpy()
        want = X @ W.T
        for a in range(A.shape[0]):
            own = ids == a
            want[own] += got["scale"] * (X[own] @ A[a].T @ B[a].T)
        assert rel_fro(as_f64(s["Y"]), want) <= REL[torch.bfloat16]
