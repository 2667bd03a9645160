"""Infinities and values of very different magnitudes in the low-rank products, on both kernels."""
import numpy as np
import pytest
import torch

from helpers import ACC_UNIT, as_f64, ulp

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
K, N = 72, 136


def operands(fmt, tokens, rank, seed=0, k=K, n=N):
    rng = np.random.default_rng([seed, tokens, rank])

    def rand(*shape):
        return torch.from_numpy(rng.standard_normal(shape)).to(DTYPES[fmt]).to(DEV)

    return dict(X=rand(tokens, k), A=rand(1, rank, k).abs() * 0.125, B=rand(1, n, rank).abs() * 0.25, base=rand(tokens, n),
                dY=rand(tokens, n), dX_base=rand(tokens, k), plan=sp.lora_plan(None, 1, tokens=tokens, device=DEV))


# on both sides of the choice between the kernels
SIZES = [(5, 1), (11000, 1), (2600, 5), (40, 24), (700, 24), (700, 33), (300, 100)]


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens,rank", SIZES)
def test_an_infinity_in_a_row_gives_the_formulas_infinity(fmt, tokens, rank):
    """With A, B > 0 a row of X with an infinity has P = inf in every column, Y = inf; the gradients likewise."""
    d = operands(fmt, tokens, rank)
    args = d["A"], d["B"], d["plan"]
    clean = sp.lora_add(d["X"], *args, base=d["base"])
    clean_dX = sp.lora_grad(d["dY"], d["X"], *args, dX_base=d["dX_base"], need=(True, False, False))[0]
    hit = tokens // 2
    X, dY = d["X"].clone(), d["dY"].clone()
    X[hit, 3], dY[hit, 2] = float("inf"), float("inf")
    Y, h = sp.lora_add(X, *args, base=d["base"], return_h=True)
    dX, dA, _ = sp.lora_grad(dY, d["X"], *args, dX_base=d["dX_base"])
    torch.cuda.synchronize()
    keep = torch.arange(tokens, device=DEV) != hit
    assert torch.equal(Y[keep], clean[keep]) and torch.equal(dX[keep], clean_dX[keep])
    assert (Y[hit] == float("inf")).all() and (h[hit] == float("inf")).all() and (dX[hit] == float("inf")).all()
    want = torch.full((rank, K), float("inf"), device=DEV) * d["X"][hit].float()
    assert torch.equal(dA[0].float(), want)
