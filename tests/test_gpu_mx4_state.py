"""4-bit weights that come back from a file."""
import io

import pytest
import torch

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")


def test_a_weight_from_a_file():
    W = sp.mx4_quantize(torch.randn(96, 130, device=DEV).bfloat16())
    X = torch.randn(7, 130, device=DEV).bfloat16()
    f = io.BytesIO()
    torch.save(W, f)
    f.seek(0)
    V = torch.load(f, weights_only=False)
    assert V.device == W.device and V.dtype is W.dtype and torch.equal(sp.mx4_linear(X, V), sp.mx4_linear(X, W))
    f.seek(0)
    away = torch.load(f, map_location="cpu", weights_only=False)
    with pytest.raises(ValueError, match="W is on cpu"):
        sp.mx4_linear(X, away)
    back = sp.Mx4(away.codes.to(DEV), away.scales.to(DEV), away.shape[1], away.dtype)
    assert torch.equal(sp.mx4_linear(X, back), sp.mx4_linear(X, W))
