"""Where a product with a 4-bit weight is written has no part in its bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("back", [False, True], ids=["linear", "grad"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,rows,cols", [(1, 300, 260), (3, 64, 96), (8, 513, 640), (40, 192, 320), (140, 333, 129), (300, 256, 264)])
def test_columns_of_a_wider_matrix(tokens, rows, cols, dtype, back):
    g = torch.Generator(device=DEV).manual_seed(tokens)
    W = sp.mx4_quantize(torch.randn(rows, cols, device=DEV, generator=g))
    n_in, n_out = (rows, cols) if back else (cols, rows)
    call = sp.mx4_linear_grad if back else sp.mx4_linear
    X = torch.randn(tokens, n_in, device=DEV, generator=g).to(dtype)
    Y = call(X, W)
    for left, right in ((8, 8), (3, 5), (1, 8), (16, 0)):
        wide = torch.empty(tokens, n_in + left + right, dtype=dtype, device=DEV)
        x = wide[:, left:left + n_in]
        x.copy_(X)
        out = torch.zeros(tokens, n_out + left + right, dtype=dtype, device=DEV)[:, left:left + n_out]
        assert torch.equal(call(x, W), Y) and torch.equal(call(X, W, out=out), Y) and torch.equal(call(x, W, out=out), Y)
