"""Dropout that drops nothing, or everything, of values that are no numbers."""
import pytest
import torch

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("cols", [64, 33])
def test_the_ends_of_the_range(dtype, cols):
    X = torch.randn(96, cols, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(dtype)
    X[::3], X[1::3, ::2] = float("inf"), float("nan")
    X[3] = -float("inf")
    assert torch.equal(torch.isnan(X).any(), torch.tensor(True, device=DEV))
    same = dict(rtol=0, atol=0, equal_nan=True)
    torch.testing.assert_close(sp.dropout(X, 0.0, (1, 2)), X, **same)
    torch.testing.assert_close(sp.dropout(X, 2.0 ** -18, (1, 2)), X, **same)  # (rounds to 0 of 65536)
    base = torch.randn(96, cols, device=DEV).to(dtype)
    torch.testing.assert_close(sp.dropout(X, 0.0, (1, 2), base=base), base + X, **same)
    assert torch.equal(sp.dropout(X, 1.0, (1, 2), base=base), base) and not sp.dropout(X, 1.0, (1, 2)).any()
