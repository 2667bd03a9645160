"""A weight that kernels of the same stream write again and again is read as the last of them left it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("tokens", [1, 4, 40, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(256, 384), (1000, 264), (4096, 512)])
def test_weights_converted_in_turn(rows, cols, dtype, tokens):
    """Two weights whose conversions land in the same memory, and every reader of them: nothing of the one before is seen."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    dense = [torch.randn(rows, cols, device=DEV, generator=g, dtype=torch.float32).to(dtype).mul_(s) for s in (1, 2.0 ** -9)]
    X = torch.randn(tokens, cols, device=DEV, generator=g).to(dtype)
    dY = torch.randn(tokens, rows, device=DEV, generator=g).to(dtype)
    Y, dX = torch.empty_like(dY), torch.empty_like(X)
    back = torch.empty_like(dense[0])

    def run(d, reader):
        W = sp.mx4_quantize(d)
        out = {"linear": lambda: sp.mx4_linear(X, W, out=Y), "grad": lambda: sp.mx4_linear_grad(dY, W, out=dX),
               "values": lambda: sp.mx4_dequantize(W, out=back)}[reader]()
        return out, W.codes.data_ptr()

    for reader in ("linear", "grad", "values"):
        want = []
        for d in dense:
            want.append(run(d, reader)[0].clone())
            torch.cuda.synchronize()
        at = set()
        for i in range(60):
            out, codes = run(dense[i % 2], reader)
            got = out.clone()
            at.add(codes)
            assert torch.equal(got, want[i % 2])
        assert len(at) <= 20  # (the same memory again and again, or this test tests nothing)


@pytest.mark.parametrize("tokens", [1, 4, 40])
def test_weight_written_in_place(tokens):
    """Codes and scales copied over by kernels queued just before the product, in a captured graph too."""
    g = torch.Generator(device=DEV).manual_seed(tokens)
    both = [sp.mx4_quantize(torch.randn(520, 512, device=DEV, generator=g).mul_(s)) for s in (1, 0.01)]
    X = torch.randn(tokens, 512, device=DEV, generator=g).bfloat16()
    want = [sp.mx4_linear(X, W) for W in both]
    W = sp.Mx4(torch.zeros_like(both[0].codes), torch.zeros_like(both[0].scales), 512)

    def turn():
        out = []
        for V in both:
            W.codes.copy_(V.codes)
            W.scales.copy_(V.scales)
            out.append(sp.mx4_linear(X, W))
        return out

    for _ in range(40):
        assert all(torch.equal(a, b) for a, b in zip(turn(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [y for _ in range(4) for y in turn()]
    for _ in range(10):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(out))
