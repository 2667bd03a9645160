"""RosaLinear on a 4-bit frozen weight and with dropout in front of its low-rank factors, against a dense 64-bit model with
the mask of the same numbers.

Tolerance, fixed before any run: as for the dense layer, each stage rounds to the storage type once or twice, dropout adds one
rounding to what the factors see and one to its gradient: relative Frobenius errors within eight half-ulps (2^-8 for bf16,
2^-11 for fp16), 1e-5 in fp32. The 4-bit values themselves are exact."""
import copy
import importlib.util
import os

import numpy as np
import pytest
import torch

import mx4_reference as ref
import workloads as wl
from helpers import as_f64, rel_fro

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
REL = {torch.float32: 1e-5, torch.float16: 8 * 2.0 ** -11, torch.bfloat16: 8 * 2.0 ** -8}
SEED = 1234


def make(dtype, k=264, out=392, n=1, sparse=False, bits4=True, dropout=0.0):
    torch.manual_seed(3)
    W = torch.randn(out, k, device=DEV).mul_(k ** -0.5).to(dtype)
    kw = {}
    if sparse:
        ro, col = wl.uniform_mask(5, out, k, 0.05)
        kw = dict(row_offsets=torch.from_numpy(ro).to(DEV), col_idx=torch.from_numpy(col).to(torch.int16).to(DEV),
                  values=torch.randn(col.size, device=DEV).mul_(0.1).to(dtype))
    scale = torch.rand(n, device=DEV) + 0.5 if n > 1 else 1.5
    layer = sp.RosaLinear(sp.mx4_quantize(W) if bits4 else W, 8, n_adapters=n, scale=scale, dropout=dropout, **kw)
    layer.B.data.normal_(0, 0.1)
    W64 = ref.values(*ref.quantize(as_f64(W)), k) if bits4 else as_f64(W)
    return layer, W64


def drawn_state():
    torch.manual_seed(SEED)
    return [int(v) for v in torch.randint(0, 2 ** 63 - 1, (2,), dtype=torch.int64, device=DEV).cpu()]


def factor_mask(shape, p):
    seed, call = drawn_state()
    return ref.dropout(np.ones(shape), p, seed, call)


@pytest.mark.parametrize("dtype", list(REL))
@pytest.mark.parametrize("tokens", [1, 6, 300])
@pytest.mark.parametrize("n,sparse,bits4,p", [(1, False, True, 0.0), (3, True, True, 0.25), (1, False, True, 0.1),
                                              (2, False, False, 0.5), (1, True, False, 0.0)])
def test_forward_and_gradients(dtype, tokens, n, sparse, bits4, p):
    layer, W64 = make(dtype, n=n, sparse=sparse, bits4=bits4, dropout=p)
    out, k = W64.shape
    X = torch.randn(tokens, k, device=DEV).to(dtype).requires_grad_()
    ids = torch.randint(-1, n, (tokens,), dtype=torch.int32, device=DEV) if n > 1 else None
    G = torch.randn(tokens, out, device=DEV).to(dtype)
    torch.manual_seed(SEED)
    Y = layer(X, adapter_ids=ids)
    Y.backward(G)

    d = {x: torch.from_numpy(as_f64(t)).requires_grad_() for x, t in (("X", X), ("A", layer.A), ("B", layer.B))}
    Wd, vals = torch.from_numpy(W64), None
    if sparse:
        vals = torch.from_numpy(as_f64(layer.values)).requires_grad_()
        rows = np.repeat(np.arange(out), np.diff(layer.row_offsets.cpu().numpy()))
        at = torch.from_numpy(rows), layer.col_idx.cpu().long()
        Wd = Wd.index_put(at, vals, accumulate=True)
    seen = d["X"] if p == 0 else d["X"] * torch.from_numpy(factor_mask((tokens, k), p))
    which = ids.cpu() if ids is not None else torch.zeros(tokens, dtype=torch.int32)
    want = d["X"] @ Wd.t()
    for a in range(n):
        own = (which == a).double()[:, None]
        s = float(layer.scale[a]) if n > 1 else layer.scale
        want = want + own * s * (seen @ d["A"][a].t() @ d["B"][a].t())
    want.backward(torch.from_numpy(as_f64(G)))

    def close(got, wanted, what):
        wanted = wanted.detach().numpy()
        e = rel_fro(as_f64(got).reshape(wanted.shape), wanted)
        assert e <= REL[dtype], (what, e)

    close(Y, want, "Y")
    close(X.grad, d["X"].grad, "dX")
    close(layer.A.grad, d["A"].grad, "dA")
    close(layer.B.grad, d["B"].grad, "dB")
    if sparse:
        close(layer.values.grad, vals.grad, "dvalues")


def test_gradients_against_differences():
    """fp32, one mask: the loss's change along a direction is the gradients' product with it."""
    layer, _ = make(torch.float32, k=64, out=96, dropout=0.3)
    X = torch.randn(40, 64, device=DEV, requires_grad=True)
    G = torch.randn(40, 96, device=DEV)

    def loss():
        torch.manual_seed(SEED)
        return (layer(X).double() * G).sum()

    loss().backward()
    eps = 2.0 ** -7  # (the loss is a polynomial of third degree in all of them; its middle difference is off by eps^2)
    dirs = {id(t): torch.randn_like(t) * 0.5 for t in (X, layer.A, layer.B)}
    want = sum(float((t.grad.double() * dirs[id(t)]).sum()) for t in (X, layer.A, layer.B))
    values = []
    with torch.no_grad():
        keep = {id(t): t.detach().clone() for t in (X, layer.A, layer.B)}
        for sign in (1, -1):
            for t in (X, layer.A, layer.B):
                t.copy_(keep[id(t)] + sign * eps * dirs[id(t)])
            values.append(float(loss()))
        # the cubic term, exactly: s (dir_X keep) dir_A^T dir_B^T G
        seen = torch.from_numpy(factor_mask((40, 64), 0.3)).to(DEV)
        third = float(((dirs[id(X)].double() * seen) @ dirs[id(layer.A)][0].double().t() @ dirs[id(layer.B)][0].double().t() * G).sum()) * 1.5
    got = (values[0] - values[1]) / (2 * eps) - eps ** 2 * third
    # 64 * 96 * 40 products of about 1 rounded to 2^-24 each way, divided by 2 eps
    assert abs(got - want) <= 2e-4 * abs(want) + 0.05


def test_evaluation_and_masks():
    layer, W64 = make(torch.bfloat16, dropout=0.5)
    X = torch.randn(200, 264, device=DEV, dtype=torch.bfloat16)
    with torch.no_grad():
        torch.manual_seed(1)
        a, b = layer(X), layer(X)
        torch.manual_seed(1)
        c = layer(X)
        assert not torch.equal(a, b) and torch.equal(a, c)  # a mask for each pass, the generator's
        layer.eval()
        d = layer(X)
        assert torch.equal(d, layer(X))
        plain, _ = make(torch.bfloat16)
        assert torch.equal(d, plain(X))


def test_state_moves_and_copies():
    layer, W64 = make(torch.bfloat16, sparse=True)
    assert set(layer.state_dict()) == {"codes", "scales", "A", "B", "row_offsets", "col_idx", "values"}
    X = torch.randn(100, 264, device=DEV, dtype=torch.bfloat16)
    Y = layer(X)
    twin = copy.deepcopy(layer)
    assert twin._quantized is None and torch.equal(twin(X), Y)
    other, _ = make(torch.bfloat16, sparse=True)
    with torch.no_grad():
        other.codes.zero_()
    assert not torch.equal(other(X), Y)
    other.load_state_dict(layer.state_dict())
    assert torch.equal(other(X), Y)
    back = layer.to("cpu").to(DEV)
    assert torch.equal(back(X), Y)
    half, _ = make(torch.bfloat16)
    half = half.to(torch.float16)
    want = as_f64(X.half()) @ (W64 + 1.5 * as_f64(half.B)[0] @ as_f64(half.A)[0]).T
    assert half.quantized.dtype == torch.float16 and rel_fro(as_f64(half(X.half())), want) <= REL[torch.float16]


def test_a_weight_that_changes_between_the_passes_is_noticed():
    layer, _ = make(torch.bfloat16)
    X = torch.randn(30, 264, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    Y = layer(X)
    layer.scales.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        Y.sum().backward()


def test_captured_training_step():
    """Forward and backward in one graph: every replay has a mask of its own, and its gradients go with it."""
    layer, _ = make(torch.bfloat16, k=128, out=256, dropout=0.4)
    X = torch.randn(90, 128, device=DEV, dtype=torch.bfloat16)
    G = torch.randn(90, 256, device=DEV, dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            layer.zero_grad()
            layer(X).backward(G)
    torch.cuda.current_stream().wait_stream(side)
    layer.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = layer(X)
        Y.backward(G)
    seen = []
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        seen.append((Y.detach().clone(), layer.A.grad.clone(), layer.B.grad.clone()))
    assert not torch.equal(seen[0][0], seen[1][0]) and not torch.equal(seen[1][0], seen[2][0])
    # dB = s G^T (D A^T) with Y = base + s (D A^T) B^T: what the factors added and its gradient share D
    A, B, G64 = as_f64(layer.A)[0], as_f64(layer.B)[0], as_f64(G)
    for Yv, dA, dB in seen:
        layer.eval()
        keep = layer.B.data.clone()
        layer.B.data.zero_()
        base = as_f64(layer(X))
        layer.B.data.copy_(keep)
        h = np.linalg.lstsq(1.5 * B, (as_f64(Yv) - base).T, rcond=None)[0].T  # [tokens, rank]
        # (Y's rounding reaches h through B's pseudo-inverse: well conditioned, 256 x 8 normal values)
        assert rel_fro(as_f64(dB)[0], 1.5 * G64.T @ h) <= 0.05


def test_refusals():
    W = sp.mx4_quantize(torch.randn(64, 48, device=DEV, dtype=torch.bfloat16))
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(ValueError, match="dropout must lie"):
            sp.RosaLinear(W, 4, dropout=p)
    layer = sp.RosaLinear(W, 4)
    with pytest.raises(ValueError, match="dtype"):
        layer(torch.randn(5, 48, device=DEV))
    X = torch.randn(5, 48, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    (g,) = torch.autograd.grad(layer(X).sum(), X, create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        g.sum().backward()


def test_adapter_training_and_serving_run():
    """As they are used together: a weight converted once, trained with dropout, clipped and stepped; then evaluated for a
    batch of prompts and token by token, where the results agree."""
    torch.manual_seed(0)
    k = 256
    W = torch.randn(k, k, device=DEV).mul_(k ** -0.5).to(torch.bfloat16)
    layer = sp.RosaLinear(sp.mx4_quantize(W), 16, scale=2.0, dropout=0.1)
    X = torch.randn(500, k, device=DEV, dtype=torch.bfloat16)
    params = list(layer.parameters())
    for q in params:
        q.grad = torch.zeros_like(q)
    grads = sp.GradSet([q.grad for q in params])
    master = [q.detach().float().reshape(-1).clone() for q in params]
    moments = [(torch.zeros_like(m), torch.zeros_like(m)) for m in master]
    before = [q.detach().clone() for q in params]
    for step in range(1, 5):
        (layer(X) - X).float().square().mean().backward()
        norm = float(sp.clip_grads(grads, 1.0))
        assert np.isfinite(norm) and norm > 0
        for q, m, (a, b) in zip(params, master, moments):
            sp.masked_adam(m, a, b, q.grad.reshape(-1), step, lr=1e-2)
            q.data.copy_(m.reshape(q.shape))
            q.grad.zero_()
    assert all(not torch.equal(q, old) for q, old in zip(params, before))
    layer.eval()
    with torch.no_grad():
        whole = layer(X)
        want = as_f64(X) @ (ref.values(*ref.quantize(as_f64(W)), k) + 2.0 * as_f64(layer.B)[0] @ as_f64(layer.A)[0]).T
        assert rel_fro(as_f64(whole), want) <= REL[torch.bfloat16]
        for t in (0, 3, 499):
            assert rel_fro(as_f64(layer(X[t:t + 1]))[0], want[t]) <= REL[torch.bfloat16]


def test_example_with_four_bits():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "rosa_finetune_and_serve.py")
    spec = importlib.util.spec_from_file_location("rosa_example_4bit", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, norms = ex.train(steps=4, four_bits=True, dropout=0.1)
    assert np.isfinite(losses).all() and all(x > 0 for x in norms)
